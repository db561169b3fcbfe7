"""What the state space layer's operators and draft verification refuse before anything is launched
(no GPU needed), and the plain forms that their GPU tests compare with."""
import ctypes

import pytest
import torch

import linear_attention_serving_chunk_gb300 as kda
import serving_ref as ref

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call below is rejected first
NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5
off = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    kda.build()
    return kda.lib()


def call(fn, base, kw):
    a = dict(base)
    assert set(kw) <= set(a)
    a.update(kw)
    return fn(*a.values())


CONV = dict(x=FAKE, ldx=64, weight=FAKE, bias=None, cu=None, n=2, total=8, D=64, W=4, flags=1)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), SHAPE), (dict(total=-1), SHAPE), (dict(n=3), SHAPE), (dict(n=0), SHAPE), (dict(D=0), SHAPE),
    (dict(total=1 << 31), SHAPE), (dict(ldx=63), SHAPE), (dict(ldo=60), SHAPE), (dict(W=1), UNSUPPORTED),
    (dict(W=5), UNSUPPORTED), (dict(flags=2), UNSUPPORTED), (dict(x=None), NULL), (dict(weight=None), NULL),
    (dict(o=None), NULL), (dict(x=off(0x10001)), ALIGN), (dict(cu=off(0x10002)), ALIGN),
    (dict(conv0=FAKE, final=FAKE), SHAPE), (dict(n=0, total=0), 0), (dict(total=0, final=None), 0)])
def test_conv_fwd_refuses(L, kw, status):
    base = dict(CONV, conv0=None, final=None, o=off(0x20000), ldo=64, stream=None)
    assert call(L.kda_conv_fwd, base, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), SHAPE), (dict(n_slots=1), SHAPE), (dict(n_slots=-1, slots=FAKE), SHAPE), (dict(pool=None), NULL),
    (dict(o=None, commit=0), NULL), (dict(W=0), UNSUPPORTED), (dict(slots=off(0x10002)), ALIGN),
    (dict(used=off(0x10001)), ALIGN), (dict(pool=off(0x10001)), ALIGN), (dict(total=0), 0)])
def test_conv_tokens_refuses(L, kw, status):
    base = dict(CONV, pool=FAKE, n_slots=2, slots=None, used=None, commit=1, o=off(0x20000), ldo=64, stream=None)
    assert call(L.kda_conv_tokens, base, kw) == status


SSM = dict(x=FAKE, ldx=256, dt=FAKE, lddt=4, A=FAKE, B=FAKE, ldb=128, C=FAKE, ldc=128, D=None, z=None, ldz=0,
           bias=None, flags=1, cu=None, n=2, total=8, H=4, P=64, G=2, N=64)
SSM_WRONG = [
    (dict(n=-1), SHAPE), (dict(n=3), SHAPE), (dict(H=0), SHAPE), (dict(G=0), SHAPE), (dict(G=3), SHAPE),
    (dict(H=65536), SHAPE), (dict(P=96), UNSUPPORTED), (dict(N=32), UNSUPPORTED), (dict(flags=4), UNSUPPORTED),
    (dict(ldx=255), SHAPE), (dict(lddt=3), SHAPE), (dict(ldb=120), SHAPE), (dict(ldc=120), SHAPE),
    (dict(ldo=248), SHAPE), (dict(z=FAKE, ldz=248), SHAPE), (dict(x=None), NULL), (dict(dt=None), NULL),
    (dict(A=None), NULL), (dict(B=None), NULL), (dict(C=None), NULL), (dict(x=off(0x10008)), ALIGN),
    (dict(B=off(0x10002)), ALIGN), (dict(ldx=260), ALIGN), (dict(ldb=132), ALIGN), (dict(ldo=260), ALIGN),
    (dict(z=FAKE, ldz=257), ALIGN), (dict(A=off(0x10002)), ALIGN), (dict(dt=off(0x10001)), ALIGN)]


@pytest.mark.parametrize("kw,status", SSM_WRONG + [
    (dict(o=None), NULL), (dict(S0=FAKE, final=FAKE), SHAPE), (dict(ws=off(0x10008)), ALIGN),
    (dict(n=0, total=0), 0), (dict(total=0, final=None), 0)])
def test_ssm_fwd_refuses(L, kw, status):
    base = dict(SSM, S0=None, o=off(0x20000), ldo=256, final=None, ws=None, ws_bytes=0, stream=None)
    assert call(L.kda_ssm_fwd, base, kw) == status


@pytest.mark.parametrize("kw,status", SSM_WRONG + [
    (dict(n_slots=1), SHAPE), (dict(pool=None), NULL), (dict(o=None, commit=0), NULL),
    (dict(slots=off(0x10002)), ALIGN), (dict(used=off(0x10001)), ALIGN), (dict(pool=off(0x10004)), ALIGN),
    (dict(total=0), 0)])
def test_ssm_tokens_refuses(L, kw, status):
    base = dict(SSM, pool=FAKE, n_slots=2, slots=None, used=None, commit=1, o=off(0x20000), ldo=256, stream=None)
    assert call(L.kda_ssm_tokens, base, kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), SHAPE), (dict(V=0), SHAPE), (dict(total=1), SHAPE), (dict(size=3), UNSUPPORTED),
    (dict(V=(1 << 22) + 1), UNSUPPORTED), (dict(target=None), NULL), (dict(tokens=None), NULL), (dict(u=None), NULL),
    (dict(cu=None), NULL), (dict(out=None), NULL), (dict(n_out=None), NULL), (dict(target=off(0x10002)), ALIGN),
    (dict(draft=off(0x10001)), ALIGN), (dict(u=off(0x10002)), ALIGN), (dict(n=0, total=0), 0)])
def test_verify_draft_refuses(L, kw, status):
    base = dict(target=FAKE, draft=None, size=4, V=100, tokens=FAKE, u=FAKE, cu=FAKE, n=2, total=6, out=FAKE,
                n_out=FAKE, stream=None)
    assert call(L.kda_verify_draft, base, kw) == status


def test_binding_refuses_cpu_tensors_and_wrong_types():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(8, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kda.conv_fwd(x, w)
    with pytest.raises(TypeError):
        kda.verify_draft(torch.zeros(4, 8, dtype=torch.float64), None, None, None)


def test_plain_scan_against_one_token_and_a_decay_that_keeps_all():
    """One token from a zero state is (C.B) dt x + D x; with A = 0 the state is a sum."""
    i = ref.ssm_inputs(6, 2, 64, 1, 64, 0)
    i["A"] = torch.zeros(2)
    i["z"] = None
    o, S, _, _ = ref.ssm(lens=[6], S=torch.zeros(1, 2, 64, 64), **i)
    step = torch.nn.functional.softplus(i["dt"].double() + i["dt_bias"].double())
    first = (i["B"][0, 0].double() @ i["C"][0, 0].double()) * step[0, :, None] * i["x"][0].double()
    assert torch.allclose(o[0], first + i["D"].double()[:, None] * i["x"][0].double(), rtol=1e-12)
    total = torch.einsum("tn,th,thp->hnp", i["B"][:, 0].double(), step, i["x"].double())
    assert torch.allclose(S[0], total, rtol=1e-12)


def test_plain_convolution_against_a_padded_one():
    x, w = torch.randn(9, 5).bfloat16(), torch.randn(5, 4).bfloat16()
    o, last = ref.conv(x, w, None, [9], torch.zeros(1, 3, 5), False)
    want = torch.nn.functional.conv1d(torch.nn.functional.pad(x.double().t(), (3, 0))[None],
                                      w.double()[:, None], groups=5)[0].t()
    assert torch.allclose(o, want, rtol=1e-12) and torch.equal(last[0], x[6:].double())


def test_plain_verification_accepts_at_the_rate_of_the_overlap():
    """With drafts from q, the first draft is accepted in a share sum(min(p, q)) of all draws."""
    V, n = 5, 4000
    g = torch.Generator().manual_seed(0)
    p, q = torch.tensor([.1, .2, .3, .4, 0.]), torch.tensor([.4, .3, .2, .05, .05])
    tokens = torch.multinomial(q, 2 * n, True, generator=g).int()
    out, count = ref.verify(p.repeat(2 * n, 1), tokens, torch.rand(2 * n, generator=g), [2] * n, q.repeat(n, 1))
    accepted = sum(c == 2 for c in count) / n
    assert abs(accepted - float(torch.minimum(p, q).sum())) < 0.04
    first = torch.tensor([t for t in out[::2]])
    share = torch.bincount(first, minlength=V) / n
    assert (share - p).abs().max() < 0.04  # the emitted token follows p
