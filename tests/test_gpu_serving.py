"""Short convolution, selective scan and draft verification on the GPU against their plain forms in
64 bits (tests/serving_ref.py)."""
import pytest
import torch

import linear_attention_serving_chunk_gb300 as kda
import serving_ref as ref

pytestmark = pytest.mark.gpu

HALF_STEP = 2.0 ** -8       # a rounding to bf16, relative to the value
SUM32 = 2.0 ** -19          # fp32 sums and exponentials, relative to the size of their terms


@pytest.fixture(autouse=True)
def clean_status():
    kda.device_status()
    yield
    torch.cuda.synchronize()


def cuda(t):
    return None if t is None else t.cuda()


def wide_cuda(t, wide):
    """`t` on the GPU as the middle columns of a buffer of wider rows."""
    rows = t.shape[0]
    buf = torch.full((rows, t[0].numel() + 2 * wide), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[:, wide:buf.shape[1] - wide]
    view.copy_(t.reshape(rows, -1))
    return view.view(t.shape) if t.dim() == 2 else view.unflatten(1, t.shape[1:])


def cu_of(lens):
    return torch.tensor(ref.offsets(lens), dtype=torch.int32, device="cuda")


def within(got, want, size, relative=HALF_STEP):
    """|got - want| within one rounding of the result and the sums' error."""
    err = (got.double().cpu() - want).abs()
    worst = (err - relative * want.abs() - size).max() if err.numel() else torch.tensor(-1.0)
    assert not torch.isnan(err).any() and float(worst) <= 0, float(worst)


LENS = [[5], [1, 77, 250], [0, 1, 2, 3, 0, 31, 32, 33, 0], [64, 0, 127, 128, 129], [300, 1]]


# ---- short convolution -------------------------------------------------------------------------

@pytest.mark.parametrize("D,wide", [(8, 0), (64, 8), (136, 16), (70, 3), (547, 0), (1, 0), (1100, 4)])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lens", LENS)
def test_conv_fwd(D, wide, W, lens):
    g = torch.Generator().manual_seed(D + W)
    total, n = sum(lens), len(lens)
    silu, state = (D + W) % 2 == 0, len(lens) % 2 == 1
    x = torch.randn(total, D, generator=g).bfloat16()
    weight, bias = torch.randn(D, W, generator=g).bfloat16(), torch.randn(D, generator=g).bfloat16()
    bias = bias if W != 3 else None
    held = torch.randn(n, W - 1, D, generator=g).bfloat16() if state else torch.zeros(n, W - 1, D)
    want, last = ref.conv(x, weight, bias, lens, held, silu)
    size, _ = ref.conv(x.abs(), weight.abs(), bias if bias is None else bias.abs(), lens, held.abs(), False)
    xs, o = wide_cuda(x, wide), wide_cuda(torch.zeros(total, D, dtype=torch.bfloat16), wide)
    final = torch.full((n, W - 1, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = kda.conv_fwd(xs, cuda(weight), cuda(bias), cu_seqlens=cu_of(lens),
                       conv0=cuda(held) if state else None, conv_final=final, silu=silu, o=o)
    assert got is o
    # exp and the division of the activation: under 2^-19 of the value for |y| below 90
    within(got, want, 2 * SUM32 * (1 + size))
    assert torch.equal(final.double().cpu(), last)
    assert kda.device_status() == 0
    if wide and total:  # nothing beside the columns is written
        rest = o._base[:, list(range(wide)) + list(range(wide + D, 2 * wide + D))]
        assert torch.isnan(rest).all()


def test_conv_fwd_equal_lengths_and_no_state():
    g = torch.Generator().manual_seed(0)
    x, weight = torch.randn(3 * 40, 64, generator=g).bfloat16(), torch.randn(64, 4, generator=g).bfloat16()
    want, _ = ref.conv(x, weight, None, [40] * 3, torch.zeros(3, 3, 64), True)
    got = kda.conv_fwd(cuda(x), cuda(weight), n_seq=3)
    within(got, want, 2 * SUM32 * 40)


@pytest.mark.parametrize("D", [64, 75])
def test_conv_nan_of_one_sequence_stays_there(D):
    lens = [33, 40, 7]
    x = torch.randn(80, D).bfloat16()
    w = torch.randn(D, 4).bfloat16()
    want = kda.conv_fwd(cuda(x), cuda(w), cu_seqlens=cu_of(lens))
    x[33:73] = float("nan")
    got = kda.conv_fwd(cuda(x), cuda(w), cu_seqlens=cu_of(lens))
    assert torch.equal(got[:33], want[:33]) and torch.equal(got[73:], want[73:])
    assert torch.isnan(got[33:73]).all()


def test_conv_fwd_malformed_offsets_are_recorded():
    x, w = torch.ones(40, 64, dtype=torch.bfloat16).cuda(), torch.ones(64, 4, dtype=torch.bfloat16).cuda()
    for bad in ([0, 50, 40], [-3, 10, 40], [0, 30, 20], [0, 2 ** 30, 40]):
        final = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")
        kda.conv_fwd(x, w, cu_seqlens=torch.tensor(bad, dtype=torch.int32, device="cuda"), conv_final=final)
        assert kda.device_status() == kda.KDA_ERR_SHAPE, bad


@pytest.mark.parametrize("D,W", [(64, 4), (70, 4), (1100, 3), (9, 2)])
@pytest.mark.parametrize("lens", [[1] * 7, [1, 3, 5, 2], [2, 0, 4]])
@pytest.mark.parametrize("mode", ["plain", "used", "keep", "advance"])
def test_conv_tokens(D, W, lens, mode):
    g = torch.Generator().manual_seed(D)
    n, total = len(lens), sum(lens)
    x = torch.randn(total, D, generator=g).bfloat16()
    weight, bias = torch.randn(D, W, generator=g).bfloat16(), torch.randn(D, generator=g).bfloat16()
    pool = torch.randn(n + 3, W - 1, D, generator=g).bfloat16()
    slots = torch.randperm(n + 3, generator=g)[:n]
    used = [(b * 2 + 1) % (L + 1) for b, L in enumerate(lens)] if mode in ("used", "advance") else None
    held = pool[slots]
    want, last = ref.conv(x, weight, bias, lens, held, True, used)
    size, _ = ref.conv(x.abs(), weight.abs(), bias.abs(), lens, held.abs(), False)
    p = cuda(pool)
    got = kda.conv_tokens(cuda(x), cuda(weight), cuda(bias), p, slots=cuda(slots.int()),
                          cu_seqlens=None if lens == [1] * 7 else cu_of(lens),
                          used=None if used is None else torch.tensor(used, dtype=torch.int32, device="cuda"),
                          commit=mode != "keep", o=False if mode == "advance" else None)
    if mode == "advance":
        assert got is None
    else:
        within(got, want, 2 * SUM32 * (1 + size))
    after = pool.double()
    if mode != "keep":
        after[slots] = last
    assert torch.equal(p.double().cpu(), after)
    assert kda.device_status() == 0


def test_token_forms_skip_bad_slots_and_bad_used():
    n, D, H, P, N = 5, 64, 2, 64, 64
    slots = torch.tensor([0, 9, -1, 3, 4], dtype=torch.int32, device="cuda")
    used = torch.tensor([1, 1, 1, 2, -1], dtype=torch.int32, device="cuda")
    x, w = torch.randn(n, D).bfloat16().cuda(), torch.randn(D, 4).bfloat16().cuda()
    pool = torch.randn(6, 3, D).bfloat16().cuda()
    before = pool.clone()
    o = torch.full((n, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.conv_tokens(x, w, None, pool, slots=slots, used=used, o=o)
    assert kda.device_status() == kda.KDA_ERR_SHAPE
    assert torch.equal(pool[1:], before[1:]) and not torch.equal(pool[0], before[0])
    assert (o[1:] == 7).all()
    i = {k: cuda(v) for k, v in ref.ssm_inputs(n, H, P, 1, N, 3).items()}
    states = torch.randn(6, H, N, P, device="cuda")
    before = states.clone()
    o = torch.full((n, H, P), 7.0, dtype=torch.bfloat16, device="cuda")
    kda.ssm_tokens(state_pool=states, slots=slots, used=used, o=o, **i)
    assert kda.device_status() == kda.KDA_ERR_SHAPE
    assert torch.equal(states[1:], before[1:]) and not torch.equal(states[0], before[0])
    assert (o[1:] == 7).all()


# ---- selective scan ----------------------------------------------------------------------------

def scan_case(lens, H, P, G, N, seed, wide=0, state=True, drop=(), softplus=True):
    i = ref.ssm_inputs(sum(lens), H, P, G, N, seed, wide)
    for k in drop:
        i[k] = None
    if not softplus:
        i["dt"] = (0.05 * i["dt"].float().abs()).bfloat16()
        i["dt_bias"] = None
    S0 = torch.randn(len(lens), H, N, P, generator=torch.Generator().manual_seed(seed + 1))
    return i, S0 if state else torch.zeros(len(lens), H, N, P)


def check_states(got, want, size):
    within(got, want, SUM32 * size, relative=0.0)


SCANS = [  # H, P, G, N, wide, dropped inputs, softplus
    (2, 64, 1, 64, 0, (), True), (2, 64, 1, 128, 8, ("z",), True), (3, 64, 1, 128, 0, ("D",), True),
    (2, 128, 2, 128, 0, ("z", "dt_bias"), True), (1, 128, 1, 64, 16, (), False),
    (6, 64, 2, 64, 0, ("z", "D"), True), (5, 64, 5, 128, 0, (), True)]


@pytest.mark.parametrize("H,P,G,N,wide,drop,softplus", SCANS)
@pytest.mark.parametrize("lens", LENS)
def test_ssm_fwd(H, P, G, N, wide, drop, softplus, lens):
    state = len(lens) % 2 == 1
    i, S0 = scan_case(lens, H, P, G, N, seed=H + len(lens), wide=wide, state=state, drop=drop, softplus=softplus)
    want, last, size, size_s = ref.ssm(lens=lens, S=S0, dt_softplus=softplus, **i)
    final = torch.full((len(lens), H, N, P), float("nan"), device="cuda")
    d = {k: cuda(v) for k, v in i.items()}
    if wide:
        d["x"], d["B"], d["C"] = (wide_cuda(i[k], wide) for k in "xBC")
    got = kda.ssm_fwd(cu_seqlens=cu_of(lens), S0=cuda(S0) if state else None, S_final=final,
                      dt_softplus=softplus, **d)
    # two roundings to bf16: the weights of a chunk's tokens, and the result
    within(got, want, HALF_STEP * size)
    rms = (got.double().cpu() - want).norm() / want.norm()
    assert float(rms) <= 2 ** 0.5 * HALF_STEP / 3 ** 0.5
    check_states(final, last, size_s)
    assert kda.device_status() == 0


@pytest.mark.parametrize("T,n,H,P,N", [(1500, 1, 2, 64, 128), (2111, 1, 2, 128, 64), (1024, 2, 1, 128, 128)])
def test_ssm_fwd_long(T, n, H, P, N):
    """Longer sequences, without offsets, and a state that is kept for all of them."""
    lens = [T] * n
    i, S0 = scan_case(lens, H, P, 1, N, seed=T)
    i["A"], i["dt_bias"] = i["A"] * 0 - 0.05, i["dt_bias"] * 0 - 3.0
    want, last, size, size_s = ref.ssm(lens=lens, S=S0, **i)
    final = torch.empty(n, H, N, P, device="cuda")
    got = kda.ssm_fwd(n_seq=n, S0=cuda(S0), S_final=final, **{k: cuda(v) for k, v in i.items()})
    within(got, want, HALF_STEP * size)
    check_states(final, last, size_s)
    # the states of a prefix continue to the same end
    half = torch.empty(n, H, N, P, device="cuda")
    cut = [t * T + u for t in range(n) for u in range(700)]
    rest = [t * T + u for t in range(n) for u in range(700, T)]
    part = {k: (v[cut] if k in ("x", "dt", "B", "C", "z") else v) for k, v in i.items()}
    kda.ssm_fwd(n_seq=n, S0=cuda(S0), S_final=half, **{k: cuda(v) for k, v in part.items()})
    part = {k: (v[rest] if k in ("x", "dt", "B", "C", "z") else v) for k, v in i.items()}
    kda.ssm_fwd(n_seq=n, S0=half, S_final=final, **{k: cuda(v) for k, v in part.items()})
    check_states(final, last, size_s)


def test_ssm_decays_to_nothing_and_keeps_everything():
    """exp(dt A) of 0 forgets what was there; dt of 0 leaves the state as it is, bit by bit."""
    lens, H, P, N = [300], 2, 64, 128
    i, S0 = scan_case(lens, H, P, 1, N, seed=5, drop=("dt_bias",), softplus=False)
    i["dt_bias"] = None
    i["dt"] = torch.zeros(300, H, dtype=torch.bfloat16)
    i["dt"][:, 1] = 2.0
    i["A"] = torch.tensor([-1.0, -3000.0])
    want, last, size, size_s = ref.ssm(lens=lens, S=S0, dt_softplus=False, **i)
    final = torch.empty(1, H, N, P, device="cuda")
    got = kda.ssm_fwd(S0=cuda(S0), S_final=final, dt_softplus=False, **{k: cuda(v) for k, v in i.items()})
    within(got, want, HALF_STEP * size)
    check_states(final, last, size_s)
    assert torch.equal(final[0, 0].cpu(), S0[0, 0])


@pytest.mark.parametrize("lens,bad", [([100, 130, 7], 1), ([128, 200, 300], 1), ([60, 0, 1, 300], 2)])
def test_ssm_nan_of_one_sequence_stays_there(lens, bad):
    H, P, G, N = 2, 64, 1, 128
    i, S0 = scan_case(lens, H, P, G, N, seed=9)
    i = {k: (v.contiguous() if v is not None else None) for k, v in i.items()}
    d = {k: cuda(v) for k, v in i.items()}
    f0, f1 = (torch.empty(len(lens), H, N, P, device="cuda") for _ in range(2))
    want = kda.ssm_fwd(cu_seqlens=cu_of(lens), S0=cuda(S0), S_final=f0, **d)
    at = ref.offsets(lens)[bad]
    for k in ("x", "B", "C", "dt", "z"):
        d[k] = d[k].clone()
        d[k][at:at + lens[bad]] = float("nan")
    d["x"][at] = float("inf")
    got = kda.ssm_fwd(cu_seqlens=cu_of(lens), S0=cuda(S0), S_final=f1, **d)
    for b, (t, n) in enumerate(zip(ref.offsets(lens), lens)):
        if b != bad:
            assert torch.equal(got[t:t + n], want[t:t + n]) and torch.equal(f0[b], f1[b])


def test_ssm_fwd_malformed_offsets_are_recorded():
    d = {k: cuda(v) for k, v in ref.ssm_inputs(200, 2, 64, 1, 64, 1).items()}
    for bad in ([0, 250, 200], [-3, 100, 200], [0, 150, 100], [0, 2 ** 30, 200]):
        final = torch.zeros(2, 2, 64, 64, device="cuda")
        kda.ssm_fwd(cu_seqlens=torch.tensor(bad, dtype=torch.int32, device="cuda"), S_final=final, **d)
        assert kda.device_status() == kda.KDA_ERR_SHAPE, bad


@pytest.mark.parametrize("H,P,G,N,wide,drop,softplus", SCANS)
@pytest.mark.parametrize("lens", [[1] * 5, [1, 3, 17, 8], [9, 0, 4]])
@pytest.mark.parametrize("mode", ["plain", "used", "keep", "advance"])
def test_ssm_tokens(H, P, G, N, wide, drop, softplus, lens, mode):
    n = len(lens)
    i, S = scan_case(lens, H, P, G, N, seed=H, drop=drop, softplus=softplus)
    slots = torch.randperm(n + 2, generator=torch.Generator().manual_seed(n))[:n]
    pool = torch.randn(n + 2, H, N, P, generator=torch.Generator().manual_seed(7))
    pool[slots] = S
    used = [(b * 2 + 1) % (L + 1) for b, L in enumerate(lens)] if mode in ("used", "advance") else None
    want, last, size, size_s = ref.ssm(lens=lens, S=S, dt_softplus=softplus, used=used, **i)
    d = {k: cuda(v) for k, v in i.items()}
    if wide:
        d["x"], d["B"], d["C"] = (wide_cuda(i[k], wide) for k in "xBC")
    p = cuda(pool)
    got = kda.ssm_tokens(state_pool=p, slots=cuda(slots.int()), dt_softplus=softplus,
                         cu_seqlens=None if lens == [1] * 5 else cu_of(lens),
                         used=None if used is None else torch.tensor(used, dtype=torch.int32, device="cuda"),
                         commit=mode != "keep", o=False if mode == "advance" else None, **d)
    if mode == "advance":
        assert got is None
    else:
        within(got, want, SUM32 * size)
    rest = [s for s in range(n + 2) if s not in slots.tolist()]
    assert torch.equal(p[rest].cpu(), pool[rest])
    if mode == "keep":
        assert torch.equal(p.cpu(), pool)
    else:
        check_states(p[cuda(slots)], last, size_s)
    assert kda.device_status() == 0


def test_prompt_then_tokens_equals_one_prompt():
    H, P, G, N, T = 4, 64, 2, 128, 200
    i, S0 = scan_case([T], H, P, G, N, seed=11)
    want, last, size, size_s = ref.ssm(lens=[T], S=S0, **i)
    d = {k: cuda(v) for k, v in i.items()}
    pool = torch.empty(1, H, N, P, device="cuda")
    rows = ("x", "dt", "B", "C", "z")
    kda.ssm_fwd(S0=cuda(S0), S_final=pool, **{k: v[:150] if k in rows else v for k, v in d.items()})
    got = [kda.ssm_tokens(state_pool=pool, **{k: v[t:t + 1] if k in rows else v for k, v in d.items()})
           for t in range(150, T)]
    within(torch.cat(got), want[150:], SUM32 * size[150:])
    check_states(pool, last, size_s)


# ---- draft verification ------------------------------------------------------------------------

RUNS = [[1], [5], [1, 4, 2, 6, 1], [3] * 40, [40, 2]]


@pytest.mark.parametrize("V", [1, 2, 37, 1000, 1024, 4099, 33000])
@pytest.mark.parametrize("lens", RUNS)
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("with_draft", [True, False])
def test_verify(V, lens, half, with_draft):
    p, q, tokens, u = ref.draft_inputs(lens, V, seed=V + len(lens), half=half)
    if not with_draft:
        q = None
        p[:, 0] = p[:, 1:].sum(1) if V > 1 else 1  # likely drafts
        tokens[::2] = 0
    want, count = ref.verify(p, tokens, u, lens, q)
    out, n = kda.verify_draft(cuda(p), cuda(tokens), cuda(u), cu_of(lens), draft=cuda(q))
    assert out.tolist() == want and n.tolist() == count
    assert kda.device_status() == 0


def test_verify_many_draws_follow_the_target():
    """Every u once over a grid: exactly the expected share of each token."""
    V, m = 8, 4096
    p = torch.tensor([0.5, 0.0, 0.25, 0.0, 0.125, 0.0625, 0.0625, 0.0]).repeat(m, 1)
    u = torch.arange(m).float() / m
    tokens = torch.zeros(m, dtype=torch.int32)
    out, n = kda.verify_draft(cuda(p), cuda(tokens), cuda(u), cu_of([1] * m))
    assert (n == 1).all()
    assert torch.bincount(out.cpu(), minlength=V).tolist() == (p[0] * m).long().tolist()


def test_verify_equal_distributions_and_ends_of_u():
    """p equal to q accepts whatever u is below 1; an all-zero difference falls back to p; u of 0
    takes the first token with weight and the largest u the last."""
    V, lens = 2050, [3, 3]
    p = torch.zeros(6, V)
    p[:, 100], p[:, 2049] = 0.5, 0.5
    q = p[[0, 1, 3, 4]].clone()
    tokens = torch.full((6,), 100, dtype=torch.int32)
    last = 1.0 - 2.0 ** -24
    u = torch.tensor([0.9, last, 0.0, 0.5, 0.5, last])
    out, n = kda.verify_draft(cuda(p), cuda(tokens), cuda(u), cu_of(lens), draft=cuda(q))
    assert out.tolist() == [100, 100, 100, 100, 100, 2049] and n.tolist() == [3, 3]
    tokens[1] = 7  # neither model gives it any weight: refused, and nothing is left of the row
    out, n = kda.verify_draft(cuda(p), cuda(tokens), cuda(u), cu_of(lens), draft=cuda(q))
    assert out.tolist() == [100, -1, -1, 100, 100, 2049] and n.tolist() == [1, 3]


def test_verify_malformed_inputs_are_recorded():
    V, lens = 300, [3, 2, 2]
    p, q, tokens, u = ref.draft_inputs(lens, V, seed=1)
    tokens[1] = V + 5
    out, n = kda.verify_draft(cuda(p), cuda(tokens), cuda(u), cu_of(lens), draft=cuda(q))
    assert kda.device_status() == kda.KDA_ERR_SHAPE
    assert n[0] == 1 and 0 <= int(out[0]) < V and out[1:3].tolist() == [-1, -1]
    tokens[1] = 0
    for bad in ([0, 3, 3, 7], [0, 9, 5, 7], [-1, 3, 5, 7]):
        _, n = kda.verify_draft(cuda(p), cuda(tokens), cuda(u),
                                torch.tensor(bad, dtype=torch.int32, device="cuda"), draft=cuda(q))
        assert kda.device_status() == kda.KDA_ERR_SHAPE and 0 in n.tolist()
    # rows without weight
    for value in (0.0, float("nan"), float("inf")):
        bad = p.clone()
        bad[3:5] = value
        out, n = kda.verify_draft(cuda(bad), cuda(tokens), cuda(u * 0 + 0.999), cu_of([3, 2, 2]))
        assert kda.device_status() & kda.KDA_ERR_RANGE
        assert -1 in out[3:5].tolist()


# ---- streams, graphs ---------------------------------------------------------------------------

def test_calls_on_another_stream():
    lens = [40, 3]
    i, S0 = scan_case(lens, 2, 64, 1, 64, seed=2)
    d = {k: cuda(v) for k, v in i.items()}
    w = torch.randn(64, 4).bfloat16().cuda()
    x = torch.randn(43, 64).bfloat16().cuda()
    p, q, tokens, u = (cuda(v) for v in ref.draft_inputs([3, 2], 500, seed=2))
    want = (kda.conv_fwd(x, w, cu_seqlens=cu_of(lens)), kda.ssm_fwd(cu_seqlens=cu_of(lens), **d),
            *kda.verify_draft(p, tokens, u, cu_of([3, 2]), draft=q))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = (kda.conv_fwd(x, w, cu_seqlens=cu_of(lens), stream=s),
           kda.ssm_fwd(cu_seqlens=cu_of(lens), stream=s, **d),
           *kda.verify_draft(p, tokens, u, cu_of([3, 2]), draft=q, stream=s))
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_speculative_step_in_a_graph():
    """Verify and commit captured once and replayed: the same as the calls one by one."""
    lens, H, P, G, N, V = [3, 1, 4], 2, 64, 1, 64, 600
    i, S0 = scan_case(lens, H, P, G, N, seed=4)
    d = {k: cuda(v) for k, v in i.items()}
    w = torch.randn(H * P, 4).bfloat16().cuda()
    x = torch.randn(sum(lens), H * P).bfloat16().cuda()
    p, q, tokens, u = (cuda(v) for v in ref.draft_inputs(lens, V, seed=3))
    cu = cu_of(lens)

    def step(conv, states):
        a = kda.conv_tokens(x, w, None, conv, cu_seqlens=cu, commit=False)
        o = kda.ssm_tokens(state_pool=states, cu_seqlens=cu, commit=False, **d)
        out, n = kda.verify_draft(p, tokens, u, cu, draft=q)
        kda.conv_tokens(x, w, None, conv, cu_seqlens=cu, used=n, o=False)
        kda.ssm_tokens(state_pool=states, cu_seqlens=cu, used=n, o=False, **d)
        return a, o, out, n

    pools = [(torch.randn(3, 3, H * P).bfloat16().cuda(), cuda(S0)) for _ in range(1)]
    pools.append(tuple(t.clone() for t in pools[0]))
    want = [step(*pools[0]) for _ in range(3)][-1]
    start = tuple(t.clone() for t in pools[1])
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        got = step(*pools[1])
    for t, v in zip(pools[1], start):
        t.copy_(v)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((*got, *pools[1]), (*want, *pools[0])):
        assert torch.equal(a, b)
    assert kda.device_status() == 0


def test_ssm_offsets_out_of_order_make_no_more_segments_than_there_is_room_for():
    """The same tokens over and over: every pair of offsets that rises is in range by itself."""
    d = {k: cuda(v) for k, v in ref.ssm_inputs(4096, 2, 64, 1, 64, 1).items()}
    assert kda.ssm_workspace_bytes(9, 4096, 2, 64, 1, 64) > 0  # sequences are cut
    cu = torch.tensor([0, 4096] * 5, dtype=torch.int32, device="cuda")
    final = torch.zeros(9, 2, 64, 64, device="cuda")
    kda.ssm_fwd(cu_seqlens=cu, S_final=final, **d)
    assert kda.device_status() == kda.KDA_ERR_SHAPE


@pytest.mark.parametrize("lens", [[2000, 0, 1, 700, 3000, 128], [1] * 130 + [4000], [5000] + [3] * 150])
def test_ssm_fwd_cut_sequences_among_short_ones(lens):
    """Segments of long sequences between empty and short ones; the states of all of them."""
    H, P, N = 2, 64, 64
    i, S0 = scan_case(lens, H, P, 1, N, seed=len(lens))
    i["A"], i["dt_bias"] = i["A"] * 0 - 0.3, i["dt_bias"] * 0 - 3.0
    assert kda.ssm_workspace_bytes(len(lens), sum(lens), H, P, 1, N) > 0
    want, last, size, size_s = ref.ssm(lens=lens, S=S0, **i)
    d = {k: cuda(v) for k, v in i.items()}
    final = torch.empty(len(lens), H, N, P, device="cuda")
    got = kda.ssm_fwd(cu_seqlens=cu_of(lens), S0=cuda(S0), S_final=final, **d)
    within(got, want, HALF_STEP * size)
    check_states(final, last, size_s)
    # without the room for segments each sequence is one chain: the same up to rounding
    got = kda.ssm_fwd(cu_seqlens=cu_of(lens), S0=cuda(S0), S_final=final,
                      workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), **d)
    within(got, want, HALF_STEP * size)
    check_states(final, last, size_s)
    assert kda.device_status() == 0


@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.bfloat16).min, -90.0])
def test_ssm_steps_of_nothing_leave_the_state_as_it_is(low):
    """A step of -inf, of the type's lowest value or far below 0 is 0 after softplus, in both forms."""
    lens, H, P, N = [200, 3], 2, 64, 64
    i, S0 = scan_case(lens, H, P, 1, N, seed=21)
    i["dt"] = i["dt"].clone()
    i["dt"][5:150] = low
    i["dt"][202] = low
    want, last, size, size_s = ref.ssm(lens=lens, S=S0, **i)
    d = {k: cuda(v) for k, v in i.items()}
    final = torch.empty(2, H, N, P, device="cuda")
    got = kda.ssm_fwd(cu_seqlens=cu_of(lens), S0=cuda(S0), S_final=final, **d)
    within(got, want, HALF_STEP * size)
    check_states(final, last, size_s)
    pool = cuda(S0)
    got = kda.ssm_tokens(state_pool=pool, cu_seqlens=cu_of(lens), **d)
    within(got, want, SUM32 * size)
    check_states(pool, last, size_s)


@pytest.mark.parametrize("value", [1e4, 40.0, 21.0, 19.0, 1.0, 0.0, -1.0, -20.0])
def test_ssm_softplus_over_its_range(value):
    """One token from nothing: the state is dt B x^T, so its step shows."""
    H, P, N = 1, 64, 64
    i, _ = scan_case([1], H, P, 1, N, seed=22, drop=("dt_bias", "z"))
    i["dt"] = torch.full((1, 1), value, dtype=torch.bfloat16)
    i["A"] = torch.tensor([-1e-6])
    S = torch.zeros(1, H, N, P)
    _, last, _, size_s = ref.ssm(lens=[1], S=S, **i)
    d = {k: cuda(v) for k, v in i.items()}
    for form in (0, 1):
        pool = cuda(S)
        if form:
            kda.ssm_tokens(state_pool=pool, **d)
        else:
            kda.ssm_fwd(S_final=pool, **d)
        check_states(pool, last, size_s)


def test_ssm_nan_step_is_not_lost():
    i, S0 = scan_case([4], 1, 64, 1, 64, seed=23)
    i["dt"] = i["dt"].clone()
    i["dt"][2] = float("nan")
    d = {k: cuda(v) for k, v in i.items()}
    pool = cuda(S0)
    o = kda.ssm_tokens(state_pool=pool, cu_seqlens=cu_of([4]), **d)
    assert torch.isnan(pool).all() and torch.isnan(o[2:]).all() and not torch.isnan(o[:2]).any()
    final = torch.empty(1, 1, 64, 64, device="cuda")
    kda.ssm_fwd(S0=cuda(S0), S_final=final, **d)
    assert torch.isnan(final).all()


# ---- offsets beyond 32 bits ----------------------------------------------------------------------

def test_rows_and_slots_beyond_two_to_the_31():
    """Rows of a buffer of 2.6e9 elements, and the last slots of pools as large: the same as small ones."""
    total, ld, D, H, P, N = 40000, 65536, 64, 1, 64, 64
    buf = torch.empty(total, ld, dtype=torch.bfloat16, device="cuda")
    small = torch.randn(total, D, device="cuda").bfloat16()
    x = buf[:, 1024:1024 + D]
    x.copy_(small)
    w = torch.randn(D, 4, device="cuda").bfloat16()
    assert torch.equal(kda.conv_fwd(x, w), kda.conv_fwd(small, w))
    rest = ref.ssm_inputs(total, H, P, 1, N, 5)
    d = {k: cuda(v) for k, v in rest.items()}
    want = kda.ssm_fwd(**dict(d, x=small.view(total, H, P)))
    assert torch.equal(kda.ssm_fwd(**dict(d, x=x.unflatten(1, (H, P)))), want)
    out = buf[:, 4096:4096 + D].unflatten(1, (H, P))
    kda.ssm_fwd(o=out, **dict(d, x=small.view(total, H, P)))
    assert torch.equal(out, want)
    del buf, x, out
    n, slots = 3, 600000
    pool = torch.empty(slots, H, N, P, device="cuda")
    conv = torch.empty(slots * 20, 3, D, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([slots - 1, 5, slots - 7], dtype=torch.int32, device="cuda")
    few = torch.randn(n, H, N, P, device="cuda")
    held = torch.randn(n, 3, D, device="cuda").bfloat16()
    pool[at.long()], conv[at.long() * 20] = few, held
    t = {k: v[:n] if k in ("x", "dt", "B", "C", "z") else v for k, v in d.items()}
    assert torch.equal(kda.ssm_tokens(state_pool=pool, slots=at, **t), kda.ssm_tokens(state_pool=few, **t))
    assert torch.equal(pool[at.long()], few)
    assert torch.equal(kda.conv_tokens(small[:n], w, None, conv, slots=at * 20),
                       kda.conv_tokens(small[:n], w, None, held))
    assert torch.equal(conv[at.long() * 20], held)


def test_verify_rows_beyond_two_to_the_31():
    n, V = 20000, 131072
    p = torch.zeros(n, V, device="cuda")
    want = torch.randint(0, V, (n,), device="cuda")
    p[torch.arange(n, device="cuda"), want] = 1.0
    out, count = kda.verify_draft(p, torch.zeros(n, dtype=torch.int32, device="cuda"),
                                  torch.rand(n, device="cuda"),
                                  torch.arange(n + 1, dtype=torch.int32, device="cuda"))
    assert torch.equal(out.long(), want) and (count == 1).all()
