"""Plain forms in 64 bits of the short convolution, the selective scan and draft verification, and
the inputs of their tests.  Token by token and row by row from the formulas; CPU tensors in, CPU
tensors out."""
import torch


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def conv(x, weight, bias, lens, held, silu, used=None):
    """(o, held rows after the used tokens), all float64; held [n, W - 1, D]."""
    x, weight, held = x.double(), weight.double(), held.double().clone()
    W = weight.shape[1]
    o = torch.zeros_like(x)
    for b, (at, n) in enumerate(zip(offsets(lens), lens)):
        rows = torch.cat([held[b], x[at:at + n]])
        n = n if used is None else used[b]
        for t in range(n):
            y = (weight.t() * rows[t:t + W]).sum(0) + (0 if bias is None else bias.double())
            o[at + t] = y / (1 + torch.exp(-y)) if silu else y
        held[b] = rows[n:n + W - 1]
    return o, held


def ssm(x, dt, A, B, C, lens, S, D=None, z=None, dt_bias=None, dt_softplus=True, used=None):
    """(o, states, size of o's terms, size of the states' terms): the recurrence, and the same
    with the absolute values of everything that is summed."""
    x, A, B, C, S = (v.double() for v in (x, A, B, C, S))
    total, H, P = x.shape
    per = H // B.shape[1]
    S, Sa = S.clone(), S.abs()
    o, oa = torch.zeros_like(x), torch.zeros_like(x)
    raw = dt.double() + (0 if dt_bias is None else dt_bias.double())
    step = torch.logaddexp(raw, torch.zeros_like(raw)) if dt_softplus else raw
    B, C = B.repeat_interleave(per, 1), C.repeat_interleave(per, 1)
    gate = torch.ones_like(x) if z is None else z.double() / (1 + torch.exp(-z.double()))
    skip = torch.zeros(H, dtype=torch.float64) if D is None else D.double()
    for b, (at, n) in enumerate(zip(offsets(lens), lens)):
        for t in range(at, at + (n if used is None else used[b])):
            a = torch.exp(step[t] * A)[:, None, None]
            add = B[t][:, :, None] * (step[t][:, None] * x[t])[:, None, :]
            S[b] = a * S[b] + add
            Sa[b] = a * Sa[b] + add.abs()
            y = (C[t][:, :, None] * S[b]).sum(1) + skip[:, None] * x[t]
            ya = (C[t].abs()[:, :, None] * Sa[b]).sum(1) + (skip[:, None] * x[t]).abs()
            o[t], oa[t] = y * gate[t], ya * gate[t].abs()
    return o, S, oa, Sa


def verify(target, tokens, u, lens, draft=None):
    """(out_tokens, n_out) as lists."""
    p, u = target.double(), u.double()
    q = None if draft is None else draft.double()
    out, count = [], []
    for b, (at, n) in enumerate(zip(offsets(lens), lens)):
        got = []
        for j in range(n):
            w = p[at + j].clone()
            if j < n - 1:
                x = int(tokens[at + j + 1])
                qx = 1.0 if q is None else q[at - b + j, x]
                if u[at + j] * qx < p[at + j, x]:
                    got.append(x)
                    continue
                if q is None:
                    w[x] = 0
                else:
                    w = (w - q[at - b + j]).clamp(min=0)
                if w.sum() == 0:
                    w = p[at + j].clone()
            cdf = w.cumsum(0)
            got.append(int((cdf <= u[at + n - 1] * cdf[-1]).sum()))
            break
        out += got + [-1] * (n - len(got))
        count.append(len(got))
    return out, count


def ssm_inputs(total, H, P, G, N, seed, wide=0):
    """x, dt, A, B, C, D, z, dt_bias on the CPU; steps around 0.001 to 0.1, rates 1 to 16.  With
    `wide`, x, B and C are slices of one buffer of wider rows, z and dt of another."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    xbc = torch.nn.functional.silu(rnd(total, H * P + 2 * G * N + wide)).bfloat16()
    zdt = rnd(total, (H * P + H + 7) // 8 * 8 + wide).bfloat16()
    step = torch.exp(torch.rand(H, generator=g) * 4.6 - 6.9)
    return dict(x=xbc[:, :H * P].view(total, H, P), B=xbc[:, H * P:H * P + G * N].view(total, G, N),
                C=xbc[:, H * P + G * N:H * P + 2 * G * N].view(total, G, N),
                z=zdt[:, :H * P].view(total, H, P), dt=zdt[:, H * P:H * P + H],
                A=-(1 + 15 * torch.rand(H, generator=g)), D=1 + 0.1 * rnd(H),
                dt_bias=step + torch.log(-torch.expm1(-step)))


def draft_inputs(lens, V, seed, half=False, near=0.5):
    """target, draft, tokens, u: drafts drawn from a distribution near the target's."""
    g = torch.Generator().manual_seed(seed)
    total, n = sum(lens), len(lens)
    logits = 2 * torch.randn(total, V, generator=g)
    target = torch.softmax(logits, 1)
    judged = [at + j for at, L in zip(offsets(lens), lens) for j in range(L - 1)]
    draft = torch.softmax(logits[judged] + near * torch.randn(total - n, V, generator=g), 1)
    tokens = torch.randint(0, V, (total,), generator=g, dtype=torch.int32)
    if judged:
        tokens[torch.tensor(judged) + 1] = torch.multinomial(draft, 1, generator=g)[:, 0].int()
    u = torch.rand(total, generator=g)
    t = torch.bfloat16 if half else torch.float32
    return target.to(t), draft.to(t), tokens, u
