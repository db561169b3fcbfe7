"""Outputs in the place of an input: refused before anything is launched where blocks that run side
by side would read what others write (no GPU needed), right where one block alone reads it."""
import ctypes

import pytest
import torch

import linear_attention_serving_chunk_gb300 as kda
import serving_ref as ref

SHAPE = 2
at = ctypes.c_void_p  # never dereferenced: every call on them is rejected first


@pytest.fixture(scope="module")
def L():
    kda.build()
    return kda.lib()


def conv(fn, *rest):
    return fn(at(0x10000), 64, at(0x20000), None, None, 2, 8, 64, 4, 1, *rest)


def scan(fn, *rest):
    x, dt, A, B, C = (at(0x10000 * i) for i in range(1, 6))
    return fn(x, 256, dt, 4, A, B, 128, C, 128, None, None, 0, None, 1, None, 2, 8, 4, 64, 2, 64, *rest)


def test_prompts_refuse_an_output_in_the_place_of_an_input(L):
    assert conv(L.kda_conv_fwd, None, None, at(0x10000), 64, None) == SHAPE
    for i in (1, 2, 4, 5):  # x, dt, B, C
        assert scan(L.kda_ssm_fwd, None, at(0x10000 * i), 256, None, None, 0, None) == SHAPE


def test_tokens_refuse_an_output_in_the_place_of_what_others_read(L):
    assert conv(L.kda_conv_tokens, at(0x30000), 2, None, None, 1, at(0x10000), 64, None) == SHAPE
    for i in (2, 4, 5):  # dt, B, C
        assert scan(L.kda_ssm_tokens, at(0x60000), 2, None, None, 1, at(0x10000 * i), 256, None) == SHAPE


def test_verification_refuses_its_tokens_as_output(L):
    a, b = at(0x10000), at(0x20000)
    assert L.kda_verify_draft(a, None, 4, 100, b, a, a, 2, 6, b, a, None) == SHAPE


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[1] * 7, [1, 6, 17, 3]])
def test_in_place_where_it_is_allowed(lens):
    """conv_tokens without commit and ssm_tokens over x, both scans over z: as into a new tensor."""
    n, total, H, P, N = len(lens), sum(lens), 2, 64, 64
    d = {k: v if v is None else v.cuda() for k, v in ref.ssm_inputs(total, H, P, 1, N, 3).items()}
    cu = torch.tensor(ref.offsets(lens), dtype=torch.int32, device="cuda")
    x, w = torch.randn(total, 72).bfloat16().cuda(), torch.randn(72, 4).bfloat16().cuda()
    pool, S = torch.randn(n, 3, 72).bfloat16().cuda(), torch.randn(n, H, N, P).cuda()
    want = kda.conv_tokens(x, w, None, pool, cu_seqlens=cu, commit=False)
    assert torch.equal(kda.conv_tokens(x, w, None, pool, cu_seqlens=cu, commit=False, o=x), want)
    for name, call in (("x", kda.ssm_tokens), ("z", kda.ssm_tokens), ("z", kda.ssm_fwd)):
        kw = dict(state_pool=S, commit=False) if call is kda.ssm_tokens else dict(S0=S)
        want = call(cu_seqlens=cu, **kw, **d)
        e = dict(d)
        e[name] = d[name].clone()
        assert torch.equal(call(cu_seqlens=cu, o=e[name], **kw, **e), want)


@pytest.mark.gpu
def test_binding_refuses_overlap():
    x, w = torch.zeros(8, 64, dtype=torch.bfloat16).cuda(), torch.zeros(64, 4, dtype=torch.bfloat16).cuda()
    with pytest.raises(kda.KDAError):
        kda.conv_fwd(x, w, o=x)
    p, tokens = torch.ones(2, 8).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    with pytest.raises(kda.KDAError):
        kda.verify_draft(p, tokens, torch.zeros(2).cuda(), torch.tensor([0, 2], dtype=torch.int32).cuda(),
                         out_tokens=tokens)
