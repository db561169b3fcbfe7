"""Edges of the short convolution, the selective scan and draft verification on the GPU: inputs
whose answers are easily lost, against their plain forms in 64 bits (tests/serving_ref.py)."""
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


def cu_of(lens):
    return torch.tensor(ref.offsets(lens), dtype=torch.int32, device="cuda")


def within(got, want, size, relative=HALF_STEP):
    """|got - want| within one rounding of the result and the sums' error."""
    err = (got.double().cpu() - want).abs()
    nan, worst = bool(torch.isnan(err).any()), float((err - relative * want.abs() - size).max())
    assert not nan and worst <= 0, worst


def drawn(row, u):
    """The token that u draws from a row of weights."""
    cdf = row.double().cumsum(0)
    return int((cdf <= float(u) * cdf[-1]).sum())


# ---- draft verification ------------------------------------------------------------------------

@pytest.mark.parametrize("V", [16, 300, 302, 1000, 1500, 32000])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("where", ["V", "V + 5", "-1", "-7", "far"])
def test_verify_certain_drafts_outside_the_vocabulary(V, half, where):
    """Such a token is refused and recorded, and the next one comes from the target's row as it is:
    the rows behind it, peaked where a longer row would go on, have no part in it."""
    bad = {"V": V, "V + 5": V + 5, "-1": -1, "-7": -7, "far": 2 ** 31 - 1}[where]
    n, total = 8, 24
    g = torch.Generator().manual_seed(V)
    p = torch.softmax(torch.randn(total, V, generator=g), 1)
    p[1::3] = 0.001 / V
    p[1::3, :min(V, 16)] = 1.0 / min(V, 16)  # the rows behind the judged ones
    p = p.bfloat16() if half else p
    tokens = torch.randint(0, V, (total,), generator=g, dtype=torch.int32)
    tokens[1::3] = bad  # the first draft of every run
    u = torch.rand(total, generator=g)
    out, count = kda.verify_draft(cuda(p), cuda(tokens), cuda(u), cu_of([3] * n))
    assert kda.device_status() == kda.KDA_ERR_SHAPE
    assert count.tolist() == [1] * n
    assert out.view(n, 3).tolist() == [[drawn(p[3 * b], u[3 * b + 2]), -1, -1] for b in range(n)]


@pytest.mark.parametrize("x", [0, 700, 1023, 1024, 2049])
def test_verify_certain_draft_that_outweighs_the_rest(x):
    """The refused token has all but 2^-20 of the row: what is left is drawn from by itself."""
    V, n = 2050, 64
    rest = torch.rand(V, generator=torch.Generator().manual_seed(x)) * 2 ** -31
    rest[x] = 0
    row = rest.clone()
    row[x] = 0.75
    p = row.repeat(2 * n, 1)
    tokens = torch.full((2 * n,), x, dtype=torch.int32)
    u = torch.full((2 * n,), 0.875)
    u[1::2] = torch.arange(n) / n
    out, count = kda.verify_draft(cuda(p), cuda(tokens), cuda(u), cu_of([2] * n))
    assert (count == 1).all() and (out[1::2] == -1).all()
    assert out[::2].tolist() == [drawn(rest, u[2 * b + 1]) for b in range(n)]
    assert kda.device_status() == 0


@pytest.mark.parametrize("V", [4096, 4099])
@pytest.mark.parametrize("with_draft", [False, True])
def test_verify_sums_of_large_and_small_weights(V, with_draft):
    """The sums' 43 bits: every lane of the first segment adds 31 weights of 0.94 2^-24 to one of 1,
    and tokens of 2^-38 are drawn from behind it.  In pairs of fp32 alone the sum of what the
    roundings lost is rounded itself, which is 2^-40 of each lane's sum and 3 such tokens."""
    small, fine = float(torch.tensor(0.94275 * 2 ** -24)), 2.0 ** -38
    p = torch.zeros(V, dtype=torch.float64)
    p[:1024] = small
    # the first element of each lane, vectors of four or single ones
    p[:128:4] = 1.0
    if V % 4:
        p[:128:4], p[:32] = small, 1.0
    front = 32 * (1 + 31 * small)                   # (48 bits: exact in 64)
    p[1024:2048] = fine
    left = front + fine
    for i in range(3):                              # the same again, in three weights, and half a token
        part = torch.tensor(left)
        part = part if float(part) <= left else torch.nextafter(part, torch.tensor(0.0))
        p[2048 + 40 * i] = float(part)
        left -= float(part)
    assert left == 0 and (p == p.float().double()).all()
    p = p.float()
    tokens = torch.full((2,), V - 50, dtype=torch.int32)
    if with_draft:  # the drafted token has no weight in p; 2^-60 less for all others
        q = torch.full((1, V), 2.0 ** -60)
        out, n = kda.verify_draft(cuda(p.repeat(2, 1)), cuda(tokens), torch.full((2,), 0.5).cuda(), cu_of([2]),
                                  draft=cuda(q))
    else:
        out, n = kda.verify_draft(cuda(p[None]), cuda(tokens[:1]), torch.full((1,), 0.5).cuda(), cu_of([1]))
    # half of all is the front and 512.5 of the 1024 tokens behind it
    assert n.tolist() == [1] and int(out[0]) == 1024 + 512
    assert kda.device_status() == 0


# ---- selective scan ----------------------------------------------------------------------------

def scan_inputs(lens, H, P, N, seed, **other):
    i = ref.ssm_inputs(sum(lens), H, P, 1, N, seed)
    i.update(other)
    return i, torch.randn(len(lens), H, N, P, generator=torch.Generator().manual_seed(seed + 1))


@pytest.mark.parametrize("step", [1e3, 1e5, 3e38])
@pytest.mark.parametrize("resets", [[3], [0, 31, 32, 64, 200, 255], list(range(0, 300, 4))])
@pytest.mark.parametrize("P", [64, 128])
def test_ssm_slow_tokens_behind_one_that_forgets_everything(step, resets, P):
    """Steps of 0.01 behind one whose decay is 0: what came before it has no part in the decays
    between the tokens behind it, in the prompt's form as in the token's."""
    lens, H, N = [300, 40], 2, 64
    i, S0 = scan_inputs(lens, H, P, N, seed=31, dt_bias=None, z=None)
    i["dt"] = torch.full((340, H), 0.01, dtype=torch.bfloat16)
    i["A"] = torch.tensor([-16.0, -1.0])
    at = torch.tensor(resets)
    i["dt"][at] = step
    for k in "xB":  # (its own part would hide everything else)
        i[k] = i[k].clone()
        i[k][at] = 0
    want, last, size, size_s = ref.ssm(lens=lens, S=S0, dt_softplus=False, **i)
    d = {k: cuda(v) for k, v in i.items()}
    final = torch.empty(2, H, N, P, device="cuda")
    got = kda.ssm_fwd(cu_seqlens=cu_of(lens), S0=cuda(S0), S_final=final, dt_softplus=False, **d)
    # the weights' rounding to bf16, and exponents from the difference of two sums of at most 14
    # additions, of at most 8 x 160 in a block of 32 tokens: 14 half steps of 2^-14, times log 2
    within(got, want, (HALF_STEP + 2.0 ** -10) * size)
    within(final, last, SUM32 * size_s, relative=0.0)
    pool = cuda(S0)
    got = kda.ssm_tokens(state_pool=pool, cu_seqlens=cu_of(lens), dt_softplus=False, **d)
    within(got, want, SUM32 * size)
    within(pool, last, SUM32 * size_s, relative=0.0)
    assert kda.device_status() == 0


@pytest.mark.parametrize("low", [torch.finfo(torch.bfloat16).min, -1e38])
@pytest.mark.parametrize("P", [64, 128])
def test_ssm_gate_of_the_lowest_value_closes(low, P):
    """silu of the type's lowest value is 0, whatever it is multiplied with."""
    lens, H, N = [150, 7], 2, 64
    i, S0 = scan_inputs(lens, H, P, N, seed=32)
    i["D"] = i["D"] * 100
    i["z"] = i["z"].clone()
    i["z"][5:140:3] = low
    i["z"][152] = low
    want, _, size, _ = ref.ssm(lens=lens, S=S0, **i)
    assert (want[152] == 0).all()
    d = {k: cuda(v) for k, v in i.items()}
    within(kda.ssm_fwd(cu_seqlens=cu_of(lens), S0=cuda(S0), **d), want, HALF_STEP * size)
    within(kda.ssm_tokens(state_pool=cuda(S0), cu_seqlens=cu_of(lens), **d), want, SUM32 * size)


def test_ssm_workspace_that_is_smaller_than_its_elements_is_refused():
    """One byte seen as many is no room for the segments."""
    d = {k: cuda(v) for k, v in ref.ssm_inputs(4096, 2, 64, 1, 64, 1).items()}
    need = kda.ssm_workspace_bytes(1, 4096, 2, 64, 1, 64)
    assert need > 0
    with pytest.raises(ValueError):
        kda.ssm_fwd(workspace=torch.empty(1, dtype=torch.uint8, device="cuda").expand(need), **d)
    with pytest.raises(ValueError):
        kda.ssm_fwd(workspace=torch.empty(need, dtype=torch.uint8), **d)


def test_ssm_many_prompts_of_one_token_cost_no_more_where_they_may_be_cut():
    """The work of each prompt does not grow with the number of prompts beside it."""
    n, H, P, N = 16384, 4, 64, 64
    d = {k: cuda(v) for k, v in ref.ssm_inputs(n, H, P, 1, N, 1).items()}
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    size = kda.ssm_workspace_bytes(n, n, H, P, 1, N)
    assert size > 0
    took, got = [], []
    for room in (size, 16):
        ws = torch.empty(room, dtype=torch.uint8, device="cuda")
        times = []
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            o = kda.ssm_fwd(cu_seqlens=cu, workspace=ws, **d)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        took.append(min(times))
        got.append(o)
    assert torch.equal(*got)
    assert took[0] < 2 * took[1], took


def test_ssm_cut_sequences_in_a_graph():
    """Both passes, the second launched beside the first's end, captured once and replayed on new inputs."""
    lens, H, P, N = [3000, 0, 40, 1500], 4, 64, 128
    size = kda.ssm_workspace_bytes(len(lens), sum(lens), H, P, 1, N)
    assert size > 0
    cu, ws = cu_of(lens), torch.empty(size, dtype=torch.uint8, device="cuda")
    cases = [scan_inputs(lens, H, P, N, seed) for seed in (41, 42, 43)]
    want = []
    for i, S0 in cases:
        final = torch.empty(len(lens), H, N, P, device="cuda")
        o = kda.ssm_fwd(cu_seqlens=cu, S0=cuda(S0), S_final=final, workspace=ws, **{k: cuda(v) for k, v in i.items()})
        want.append((o, final))
    d = {k: cuda(v) for k, v in cases[0][0].items()}
    S0, final = cuda(cases[0][1]), torch.empty_like(want[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = kda.ssm_fwd(cu_seqlens=cu, S0=S0, S_final=final, workspace=ws, **d)
    for (i, S), (want_o, want_s) in zip(cases, want):
        for k, v in i.items():
            d[k].copy_(v)
        S0.copy_(S)
        for _ in range(3):  # one replay behind another
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want_o) and torch.equal(final, want_s)
    assert kda.device_status() == 0
