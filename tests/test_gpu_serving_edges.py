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
    worst = (err - relative * want.abs() - size).max()
    assert not torch.isnan(err).any() and float(worst) <= 0, float(worst)


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
