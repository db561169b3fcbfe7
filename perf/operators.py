"""Cases of the state space layer's operators and of draft verification: what they take, their
plain forms in elementary torch operations, and their values from the definitions in 64 bits.

Five operators: the short causal convolution over packed prompts (`conv_fwd`) and over single
tokens or short runs on a pool of last inputs (`conv_tokens`); the selective state space scan over
packed prompts (`ssm_fwd`) and over single tokens or short runs on a pool of states
(`ssm_tokens`); and the verification of drafted tokens (`verify_draft`).
"""
import math

import torch

own = False

# Packed lengths of a mixed batch: long and short prompts, one of a single token, odd sizes.
PACKED = "9000,4096,12001,1,7000,670"
SHORT = "1,77,250"


def listed():
    return [
        # short prompts of one scheduler step, where latency counts
        dict(name="conv_prompt_short", kind="conv_fwd", lengths=SHORT, D=2304, W=4, silu=True, state=True),
        # a mixed batch of prompts: the convolution in front of 64 heads of 64 and one B/C group
        dict(name="conv_prompt_packed", kind="conv_fwd", lengths=PACKED, D=4352, W=4, silu=True, state=True),
        # one decode step of 512 sequences
        dict(name="conv_token", kind="conv_tokens", n=512, run=1, D=4352, W=4, silu=True, commit=True, used=False),
        # the accepted part of ragged drafted runs goes into the pool
        dict(name="conv_run_commit", kind="conv_tokens", n=256, run=5, D=2304, W=4, silu=True, commit=True, used=True),
        # short prompts of one scheduler step
        dict(name="ssm_prompt_short", kind="ssm_fwd", lengths=SHORT, H=32, P=64, G=1, N=128, z=True, state=True),
        # a mixed batch of prompts, 64 heads of 64
        dict(name="ssm_prompt_packed", kind="ssm_fwd", lengths=PACKED, H=64, P=64, G=1, N=128, z=True, state=True),
        # one long prompt with few heads: the scan's length is what there is to split
        dict(name="ssm_prompt_long", kind="ssm_fwd", lengths="131072", H=16, P=128, G=1, N=128, z=False, state=False),
        # a decode step of a handful of sequences
        dict(name="ssm_token_few", kind="ssm_tokens", n=3, run=1, H=16, P=64, G=2, N=128, z=True, commit=True, used=False),
        # a decode step of 512 sequences with 32 heads of 128
        dict(name="ssm_token_many", kind="ssm_tokens", n=512, run=1, H=32, P=128, G=4, N=128, z=False, commit=True, used=False),
        # ragged drafted runs on resident states, without commit
        dict(name="ssm_run_verify", kind="ssm_tokens", n=256, run=5, H=32, P=64, G=1, N=128, z=True, commit=False, used=False),
        # drafts of a few sequences, small vocabulary, bf16 probabilities
        dict(name="draft_few", kind="verify", n=4, run=5, V=32000, half=True, draft=True),
        # drafts of a large batch over a large vocabulary
        dict(name="draft_many", kind="verify", n=256, run=6, V=131072, half=False, draft=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lengths(rng, most, n_most=8):
    n = rng.randint(1, n_most)
    got = [_log(rng, 1, max(2, most // n)) for _ in range(n)]
    if n > 2 and rng.random() < 0.3:
        got[rng.randrange(n)] = 0
    return ",".join(map(str, got if any(got) else [1]))


def draw(rng):
    kind = rng.choice(["conv_fwd", "conv_tokens", "ssm_fwd", "ssm_fwd", "ssm_tokens", "ssm_tokens", "verify"])
    if kind == "conv_fwd":
        return dict(kind=kind, lengths=_lengths(rng, 32768), D=_log(rng, 64, 4352), W=rng.choice([2, 3, 4, 4]),
                    silu=rng.random() < 0.8, state=rng.random() < 0.6)
    if kind == "conv_tokens":
        run = rng.choice([1, 1, 2, 3, 5, 8])
        return dict(kind=kind, n=_log(rng, 1, 512), run=run, D=_log(rng, 64, 4352), W=rng.choice([2, 3, 4, 4]),
                    silu=rng.random() < 0.8, commit=rng.random() < 0.8, used=run > 1 and rng.random() < 0.5)
    if kind in ("ssm_fwd", "ssm_tokens"):
        G = rng.choice([1, 1, 2, 4, 8])
        c = dict(kind=kind, H=G * rng.randint(1, 32 // G), P=rng.choice([64, 128]), G=G, N=rng.choice([64, 128]),
                 z=rng.random() < 0.5)
        if kind == "ssm_fwd":
            # tokens x head columns at most those of the mixed batch
            most = min(65536, 32768 * 4096 // (c["H"] * c["P"]))
            return dict(c, lengths=_lengths(rng, most), state=rng.random() < 0.5)
        run = rng.choice([1, 1, 2, 3, 5, 8])
        return dict(c, n=_log(rng, 1, 512 // (2 if run > 1 else 1)), run=run, commit=rng.random() < 0.7,
                    used=run > 1 and rng.random() < 0.5)
    V = _log(rng, 1000, 131072)
    run = rng.randint(1, 8)
    return dict(kind=kind, n=max(1, _log(rng, 1, 256) * 6 // max(6, run)), run=run, V=V,
                half=rng.random() < 0.5, draft=rng.random() < 0.8)


def _lens(case):
    """Tokens of every sequence: the case's list, or ragged runs of 1 to `run` tokens."""
    if "lengths" in case:
        return [int(v) for v in case["lengths"].split(",")]
    return [1 + (7919 * b + case["run"] - 1) % case["run"] for b in range(case["n"])]


def _cu(lens, dev):
    cu = [0]
    for v in lens:
        cu.append(cu[-1] + v)
    return torch.tensor(cu, dtype=torch.int32, device=dev)


def _wide(total, width, used, gen, dev):
    """A projection's output [total, width]: N(0, 1) in bf16, rows padded to 16 bytes, `used` columns of it taken."""
    return torch.randn(total, (width + 7) // 8 * 8, generator=gen, device=dev).bfloat16()[:, used:]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=gen, device=dev)  # noqa: E731
    kind, lens = case["kind"], _lens(case)
    n, total = len(lens), sum(lens)
    s = dict(case=case, kind=kind, n=n, total=total, lens=lens, cu=_cu(lens, dev), longest=max(lens))
    if kind in ("conv_tokens", "ssm_tokens"):
        # the pool has more slots than the batch, taken in no order; single tokens come without offsets
        s["slots"] = torch.randperm(n + n // 4 + 1, generator=gen, device=dev)[:n].int()
        s["n_slots"] = n + n // 4 + 1
        s["used"] = (uni(n) * (s["cu"][1:] - s["cu"][:-1] + 1)).int() if case["used"] else None
        s["cu_arg"] = s["cu"] if case["run"] > 1 else None
    if kind in ("conv_fwd", "conv_tokens"):
        D, W = case["D"], case["W"]
        # x is the middle of a projection's rows, as the layer slices it
        s["x"] = _wide(total, D + 128, 64, gen, dev)[:, :D]
        s["weight"] = (rnd(D, W) / math.sqrt(W)).bfloat16()
        s["bias"] = (0.1 * rnd(D)).bfloat16()
        if kind == "conv_tokens":
            s["pool"] = rnd(s["n_slots"], W - 1, D).bfloat16()
        else:
            s["conv0"] = rnd(n, W - 1, D).bfloat16() if case["state"] else None
            s["conv_final"] = torch.empty(n, W - 1, D, dtype=torch.bfloat16, device=dev)
        return s
    if kind in ("ssm_fwd", "ssm_tokens"):
        H, P, G, N = (case[k] for k in "HPGN")
        # x, B, C: slices of the convolution's output after silu; z, dt: slices of the projection
        v = torch.nn.functional.silu(rnd(total, H * P + 2 * G * N)).bfloat16()
        s["x"] = v[:, :H * P].view(total, H, P)
        s["B"] = v[:, H * P:H * P + G * N].view(total, G, N)
        s["C"] = v[:, H * P + G * N:].view(total, G, N)
        w = _wide(total, H * P + H, 0, gen, dev)
        s["z"] = w[:, :H * P].view(total, H, P) if case["z"] else None
        s["dt"] = w[:, H * P:H * P + H]
        # rates from 1 to 16, steps around 0.001 to 0.1: memories of one to a thousand tokens
        s["A"] = -(1 + 15 * uni(H))
        step = torch.exp(uni(H) * math.log(100.0) + math.log(0.001))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["D"] = 1 + 0.1 * rnd(H)
        if kind == "ssm_tokens":
            s["pool"] = 0.1 * rnd(s["n_slots"], H, N, P)
        else:
            s["S0"] = 0.1 * rnd(n, H, N, P) if case["state"] else None
            s["S_final"] = torch.empty(n, H, N, P, device=dev)
        return s
    # verification: the draft model's distribution is near the target's, its tokens are drawn from it
    V, dt = case["V"], torch.bfloat16 if case["half"] else torch.float32
    s["target"] = torch.empty(total, V, dtype=dt, device=dev)
    s["draft"] = torch.empty(total - n, V, dtype=dt, device=dev) if case["draft"] else None
    s["tokens"] = torch.randint(0, V, (total,), generator=gen, device=dev).int()
    rows = torch.tensor([c for b, L in enumerate(lens) for c in [b] * (L - 1)], dtype=torch.int64, device=dev)
    at = torch.arange(total - n, device=dev) + rows  # the run's row that judges drafted token i
    last = s["cu"][1:].long() - 1
    for k in range(0, total - n, 256):
        i = at[k:k + 256]
        logits = 2.5 * rnd(len(i), V)
        near = logits + 0.5 * rnd(len(i), V)
        q = torch.softmax(near, 1)
        s["target"][i] = torch.softmax(logits, 1).to(dt)
        if s["draft"] is not None:
            s["draft"][k:k + 256] = q.to(dt)
        s["tokens"][i + 1] = (near - torch.log(-torch.log(uni(len(i), V)))).argmax(1).int()
    for k in range(0, n, 256):
        s["target"][last[k:k + 256]] = torch.softmax(2.5 * rnd(len(last[k:k + 256]), V), 1).to(dt)
    s["u"] = uni(total)
    return s


def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    import linear_attention_serving_chunk_gb300 as kda
    c = s["case"]
    if s["kind"] == "conv_fwd":
        o = kda.conv_fwd(s["x"], s["weight"], s["bias"], cu_seqlens=s["cu"], conv0=s["conv0"],
                         conv_final=s["conv_final"], silu=c["silu"])
        return o, s["conv_final"]
    if s["kind"] == "conv_tokens":
        o = kda.conv_tokens(s["x"], s["weight"], s["bias"], s["pool"], slots=s["slots"], cu_seqlens=s["cu_arg"],
                            used=s["used"], commit=c["commit"], silu=c["silu"])
        return o, s["pool"]
    if s["kind"] == "ssm_fwd":
        o = kda.ssm_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                        cu_seqlens=s["cu"], S0=s["S0"], S_final=s["S_final"])
        return o, s["S_final"]
    if s["kind"] == "ssm_tokens":
        o = kda.ssm_tokens(s["x"], s["dt"], s["A"], s["B"], s["C"], s["pool"], slots=s["slots"],
                           cu_seqlens=s["cu_arg"], used=s["used"], commit=c["commit"], D=s["D"], z=s["z"],
                           dt_bias=s["dt_bias"])
        return o, s["pool"]
    return kda.verify_draft(s["target"], s["tokens"], s["u"], s["cu"], draft=s["draft"])


def _sequence_of(s):
    """(sequence, position in it) of every token."""
    t = torch.arange(s["total"], device=s["cu"].device)
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return b, t - s["cu"].long()[b]


def _plain(s):
    return {"conv_fwd": _plain_conv, "conv_tokens": _plain_conv, "ssm_fwd": _plain_ssm, "ssm_tokens": _plain_ssm,
            "verify": _plain_verify}[s["kind"]](s)


def _plain_conv(s):
    c, x, W = s["case"], s["x"], s["case"]["W"]
    b, pos = _sequence_of(s)
    held = s["pool"][s["slots"].long()] if s["kind"] == "conv_tokens" else s["conv0"]
    if held is None:
        held = torch.zeros(s["n"], W - 1, c["D"], dtype=x.dtype, device=x.device)
    # rows of [x ; held rows of every sequence]: tap w of token t is W - 1 - w tokens back
    rows = torch.cat([x, held.reshape(-1, c["D"])])
    tap = torch.arange(W, device=x.device)
    back = (pos[:, None] + tap - (W - 1))
    t = torch.arange(s["total"], device=x.device)
    i = torch.where(back >= 0, t[:, None] + tap - (W - 1), s["total"] + b[:, None] * (W - 1) + back + W - 1)
    o = (rows[i].float() * s["weight"].float().t()).sum(1) + s["bias"].float()
    o = (o * torch.sigmoid(o) if c["silu"] else o).to(x.dtype)
    cu = s["cu"].long()
    L = cu[1:] - cu[:-1]
    if s.get("used") is not None:
        # tokens beyond the used ones are not taken: their rows of o stay zero
        L = s["used"].long()
        o = o * (pos < L[b])[:, None]
    back = L[:, None] + tap[:W - 1] - (W - 1)
    first = s["total"] + torch.arange(s["n"], device=x.device)[:, None] * (W - 1)
    i = torch.where(back >= 0, cu[:-1, None] + back, first + back + W - 1)
    if s["kind"] == "conv_fwd":
        s["conv_final"].copy_(rows[i])
        return o, s["conv_final"]
    if c["commit"]:
        s["pool"][s["slots"].long()] = rows[i]
    return o, s["pool"]


def _plain_ssm(s):
    """Padded to [sequence, chunk, token]: in a chunk by the matrix of decayed products, between
    chunks by the matrix of decays.  Sums of log decays in 64 bits, the products in 32."""
    c, dev = s["case"], s["x"].device
    H, P, G, N = (c[k] for k in "HPGN")
    n, total = s["n"], s["total"]
    Q = 256 if s["longest"] > 1024 else min(64, s["longest"])
    nc = -(-s["longest"] // Q)
    b, pos = _sequence_of(s)
    L = (s["cu"][1:] - s["cu"][:-1]).long()
    if s.get("used") is not None:
        L = s["used"].long()
    where = b * (nc * Q) + pos

    def padded(v, *shape):
        out = torch.zeros(n * nc * Q, v[0].numel() if total else 1, device=dev, dtype=torch.float32)
        out[where] = v.reshape(total, -1).float()
        return out.view(n, nc, Q, *shape)

    live = (pos < L[b])[:, None]
    raw = s["dt"].double() + s["dt_bias"].double()
    dt = torch.where(live, torch.logaddexp(raw, torch.zeros_like(raw)), 0.0)
    g = torch.zeros(n * nc * Q, H, dtype=torch.float64, device=dev)
    g[where] = dt * s["A"].double()
    l = g.view(n, nc, Q, H).cumsum(2)  # log decay from the chunk's start, that token's included
    X = padded(s["x"], G, H // G, P)
    Bm, Cm = padded(s["B"], G, N), padded(s["C"], G, N)
    dtp = padded(dt, G, H // G)
    xd = X * dtp[..., None]
    S0 = s["pool"][s["slots"].long()] if s["kind"] == "ssm_tokens" else s["S0"]
    S0 = torch.zeros(n, H, N, P, device=dev) if S0 is None else S0
    S0 = S0.view(n, G, H // G, N, P)
    lh = l.permute(0, 1, 3, 2)  # n, chunk, head, token
    future = torch.ones(Q, Q, dtype=torch.bool, device=dev).triu(1)
    E = torch.exp((lh[..., :, None] - lh[..., None, :]).float().masked_fill_(future, -math.inf))
    E = E.view(n, nc, G, H // G, Q, Q)
    E *= torch.matmul(Cm.transpose(2, 3), Bm.permute(0, 1, 3, 4, 2))[:, :, :, None]
    o = torch.matmul(E, xd.permute(0, 1, 3, 4, 2, 5))  # n, chunk, G, head, token, P
    del E
    # what each chunk adds to the state, and the state that each chunk starts from
    w = torch.exp((lh[..., -1:] - lh).float()).view(n, nc, G, H // G, Q)
    xw = xd.permute(0, 1, 3, 4, 2, 5) * w[..., None]
    add = torch.matmul(Bm.permute(0, 1, 3, 4, 2)[:, :, :, None], xw)  # n, chunk, G, head, N, P
    whole = torch.cat([torch.zeros(n, 1, H, dtype=torch.float64, device=dev), l[:, :, -1]], 1).cumsum(1)
    whole = whole.permute(0, 2, 1)  # n, head, boundary
    between = whole[..., :, None] - whole[..., None, :]
    between = torch.exp(between.float().masked_fill_(
        torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=dev).triu(1), -math.inf))
    parts = torch.cat([S0[:, None], add], 1).permute(0, 2, 3, 1, 4, 5).reshape(n, H, nc + 1, N * P)
    S = torch.matmul(between, parts).view(n, G, H // G, nc + 1, N, P)
    into = torch.exp(lh.float()).view(n, nc, G, H // G, Q)
    o += into[..., None] * torch.matmul(Cm.permute(0, 1, 3, 2, 4)[:, :, :, None],
                                        S[:, :, :, :-1].permute(0, 3, 1, 2, 4, 5))
    o = o.permute(0, 1, 4, 2, 3, 5).reshape(n * nc * Q, H, P)[where]
    o = o + s["D"][:, None] * s["x"].float()
    if s["z"] is not None:
        z = s["z"].float()
        o = o * (z * torch.sigmoid(z))
    o = o.to(s["x"].dtype)
    last = S[:, :, :, -1].reshape(n, H, N, P)
    if s["kind"] == "ssm_fwd":
        s["S_final"].copy_(last)
        return o, s["S_final"]
    if s["used"] is not None:
        o = o * live[:, :, None]
    if c["commit"]:
        s["pool"][s["slots"].long()] = last
    return o, s["pool"]


def _plain_verify(s):
    p, q, u, V, n = s["target"], s["draft"], s["u"].double(), s["case"]["V"], s["n"]
    dev = p.device
    b, pos = _sequence_of(s)
    cu = s["cu"].long()
    k = cu[1:] - cu[:-1] - 1
    t = torch.arange(s["total"], device=dev)
    drafted = pos < k[b]  # rows that judge a drafted token
    x = s["tokens"].long()[(t + 1).clamp(max=s["total"] - 1)]
    px = p[t, x].double()
    qx = torch.ones_like(px)
    if q is not None and len(q):
        qx = q[(t - b).clamp(max=len(q) - 1), x].double()
    refused = drafted & ~(u * qx < px)
    first = torch.where(refused, pos, k[b])
    got = torch.full((n,), 1 << 30, dtype=torch.int64, device=dev).scatter_reduce(0, b, first, "amin")  # accepted
    row = cu[:-1] + got
    r = p[row].double()
    cut = got < k
    if q is not None and len(q):
        r = torch.where(cut[:, None], r - q[(row - torch.arange(n, device=dev)).clamp(max=len(q) - 1)].double(), r)
    elif q is None:
        r = torch.where(cut[:, None] & (torch.arange(V, device=dev) == x[row][:, None]), 0.0, r)
    r = r.clamp(min=0)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, p[row].double())
    cdf = r.cumsum(1)
    token = (cdf <= (u[cu[1:] - 1] * cdf[:, -1])[:, None]).sum(1)
    out = torch.where(pos < got[b], x, torch.where(pos == got[b], token[b], -1))
    return out.int(), (got + 1).int()


def work(case):
    lens = _lens(case)
    n, total = len(lens), sum(lens)
    kind = case["kind"]
    if kind in ("conv_fwd", "conv_tokens"):
        D, W = case["D"], case["W"]
        held = 2 * n * (W - 1) * D
        states = held * (2 if kind == "conv_tokens" and case["commit"] or case.get("state") else 1)
        return {"bytes": 4 * total * D + states + 2 * D * (W + 1), "flops": (2 * W + 4) * total * D}
    if kind in ("ssm_fwd", "ssm_tokens"):
        H, P, G, N = (case[k] for k in "HPGN")
        both = case["commit"] if kind == "ssm_tokens" else case["state"]
        states = 4 * n * H * N * P * (2 if both else 1)
        rows = 2 * total * (H * P * (3 if case["z"] else 2) + 2 * G * N + H)
        # the recurrence: decay and update of the state, and its product with C
        return {"bytes": states + rows, "flops": 5 * total * H * N * P}
    V, size = case["V"], 2 if case["half"] else 4
    # one row of each distribution for every sequence: about half of the runs end in a refusal
    return {"bytes": n * V * size * (1.5 if case["draft"] else 1) + 12 * total, "flops": 3 * n * V}


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] in ("conv_fwd", "conv_tokens"):
        return _exact_conv(s)
    if s["kind"] in ("ssm_fwd", "ssm_tokens"):
        return _exact_ssm(s)
    return None  # whole numbers


def _exact_conv(s):
    """Tap by tap over each sequence with its held rows in front."""
    c, W = s["case"], s["case"]["W"]
    tokens = s["kind"] == "conv_tokens"
    weight, bias = s["weight"].double(), s["bias"].double()
    out, held = [], s["pool"].double().clone() if tokens else s["conv_final"].double().zero_()
    at, used = 0, None if s.get("used") is None else s["used"].tolist()
    slots = s["slots"].tolist() if tokens else list(range(s["n"]))
    for b, L in enumerate(s["lens"]):
        x = s["x"][at:at + L].double()
        at += L
        before = held[slots[b]].clone() if tokens else (
            s["conv0"][b].double() if s["conv0"] is not None else torch.zeros_like(held[b]))
        x = torch.cat([before, x])
        o = bias + sum(weight[:, w] * x[w:w + L] for w in range(W))
        o = o / (1 + torch.exp(-o)) if c["silu"] else o
        take = L if used is None else used[b]
        o[take:] = 0
        out.append(o)
        if not tokens or c["commit"]:
            held[slots[b]] = x[take:take + W - 1]
    return torch.cat(out), held


def _exact_ssm(s):
    """The recurrence token by token, all sequences that still have tokens at once."""
    c, dev = s["case"], s["x"].device
    H, P, G, N = (c[k] for k in "HPGN")
    tokens = s["kind"] == "ssm_tokens"
    steps = s["longest"]
    if steps * (60e-6 + s["n"] * H * N * P * 1e-11) > 15:
        return None
    raw = s["dt"].double() + s["dt_bias"].double()
    dt = torch.where(raw > 30, raw, torch.log1p(torch.exp(raw.clamp(max=30))))
    a = torch.exp(dt * s["A"].double())
    order = sorted(range(s["n"]), key=lambda b: -s["lens"][b])
    used = s["lens"] if s.get("used") is None else s["used"].tolist()
    S = torch.zeros(s["n"], H, N, P, dtype=torch.float64, device=dev)
    if tokens:
        S += s["pool"][s["slots"].long()]
    elif s["S0"] is not None:
        S += s["S0"]
    first = [sum(s["lens"][:b]) for b in range(s["n"])]
    S = S[order]
    begin = torch.tensor([first[b] for b in order], dtype=torch.int64, device=dev)
    length = sorted((s["lens"][b] for b in order), reverse=True)
    limit = torch.tensor([used[b] for b in order], device=dev)
    y = torch.zeros(s["total"], H, P, dtype=torch.float64, device=dev)
    ragged = s.get("used") is not None
    active = s["n"]
    for t in range(steps):
        while active and length[active - 1] <= t:
            active -= 1
        i = begin[:active] + t
        Bt = s["B"][i].double().repeat_interleave(H // G, 1)
        Ct = s["C"][i].double().repeat_interleave(H // G, 1)
        xt = dt[i][:, :, None] * s["x"][i].double()
        new = S[:active] if not ragged else S[:active].clone()
        new.mul_(a[i][:, :, None, None]).addcmul_(Bt[..., None], xt[:, :, None, :])
        if ragged:
            S[:active] = torch.where((limit[:active] > t)[:, None, None, None], new, S[:active])
        y[i] = (Ct[:, :, None, :] @ new)[:, :, 0]
    y += s["D"].double()[:, None] * s["x"].double()
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z / (1 + torch.exp(-z))
    if ragged:
        b, pos = _sequence_of(s)
        y = y * (pos < s["used"].long()[b])[:, None, None]
    back = torch.empty_like(S)
    back[order] = S
    if not tokens:
        return y, back
    pool = s["pool"].double()
    if c["commit"]:
        pool[s["slots"].long()] = back
    return y, pool
