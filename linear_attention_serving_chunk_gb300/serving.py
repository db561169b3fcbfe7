"""The state space layer served beside KDA, and the drafts that it verifies: short causal
convolution, selective state space scan and draft verification (``include/kda.h`` has every
argument's layout).  As in the rest of the binding, everything here checks and marshals.

A step of speculative decoding on one layer::

    c = conv_tokens(xBC, w, b, conv_pool, slots, cu, commit=False)
    o = ssm_tokens(x, dt, A, B, C, state_pool, slots, cu, commit=False)   # x, B, C: slices of c
    tokens, n_out = verify_draft(target_probs, drafted, u, cu, draft=draft_probs)
    conv_tokens(xBC, w, b, conv_pool, slots, cu, used=n_out, o=False)
    ssm_tokens(x, dt, A, B, C, state_pool, slots, cu, used=n_out, o=False)
"""
from __future__ import annotations

import torch

from . import KDA_OK, KDAError, _check, lib

CONV_SILU = 1         # KDA_CONV_SILU
SSM_DT_SOFTPLUS = 1   # KDA_SSM_DT_SOFTPLUS

# The calls below take a few microseconds on the host beside kernels that take as long, so the
# checks go through one expression for each tensor; _check and _refuse say what is wrong where
# it does not hold.
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_Tensor = torch.Tensor
_raw_stream = torch._C._cuda_getCurrentRawStream


def _refuse(t, name, dev):
    raise ValueError(f"{name} is on {t.device}, the call on cuda:{dev}")


def _device(t, name):
    """The device of the call: the one its first tensor is on, which must be the current one."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on cuda:{dev}, which is not the current device")
    return dev


def _dense(t, name, dtype, shape, dev):
    """Address of a contiguous tensor of the given type and shape on the device, 0 for None."""
    if t is None:
        return 0
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.is_contiguous() and
            t.shape == shape and t.get_device() == dev):
        _check(t, name, dtype, shape)
        _refuse(t, name, dev)
    return t.data_ptr()


def _rows(t, name, shape, dev):
    """(address, row stride) of a bf16 tensor [tokens, ...] whose rows are dense: slices of wider
    rows are taken as they are."""
    if t is None:
        return 0, 0
    if not (isinstance(t, _Tensor) and t.dtype is _BF16 and t.shape == shape and
            t.get_device() == dev):
        if isinstance(t, _Tensor) and t.is_cuda and t.dtype is _BF16 and t.shape == shape:
            _refuse(t, name, dev)
        if isinstance(t, _Tensor) and not t.is_contiguous():
            t = t.contiguous()  # (only to name what else is wrong)
        _check(t, name, _BF16, shape)
    if t.is_contiguous():
        dense = shape[1] if len(shape) == 2 else shape[1] * shape[2]
        return t.data_ptr(), dense
    s = t.stride()
    if len(shape) == 2:
        ok = s[1] == 1 or shape[1] == 1
        dense = shape[1]
    else:
        ok = (s[2] == 1 or shape[2] == 1) and (s[1] == shape[2] or shape[1] == 1)
        dense = shape[1] * shape[2]
    if not ok:
        raise ValueError(f"{name} must have dense rows, got strides {tuple(s)}")
    # the stride of a single row means nothing
    return t.data_ptr(), s[0] if shape[0] > 1 else dense


def _empty(shape, dtype, dev, stream):
    """A new tensor that belongs to the stream of the call, so that the allocator cannot hand it
    to the call while earlier work of another stream still uses it, nor away from it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _on(stream, dev):
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _runs(cu_seqlens, n, dev):
    """(address of cu_seqlens, number of runs)"""
    if cu_seqlens is None:
        return 0, n
    at = _dense(cu_seqlens, "cu_seqlens", _I32, (cu_seqlens.numel(),), dev)
    return at, cu_seqlens.numel() - 1


def _result(o, shape, dev, stream):
    """(output tensor or None, its address, its row stride)"""
    if o is False:
        return None, 0, 0
    if o is None:
        o = _empty(shape, _BF16, dev, stream)
        return o, o.data_ptr(), shape[1] if len(shape) == 2 else shape[1] * shape[2]
    return o, *_rows(o, "o", shape, dev)


def _conv_inputs(x, weight, bias):
    dev = _device(x, "x")
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be [tokens, D] and weight [D, W]")
    total, D = x.shape
    W = weight.shape[1]
    return (dev, total, D, W, *_rows(x, "x", (total, D), dev),
            _dense(weight, "weight", _BF16, (D, W), dev), _dense(bias, "bias", _BF16, (D,), dev))


def conv_fwd(x, weight, bias=None, cu_seqlens=None, n_seq=1, conv0=None, conv_final=None,
             silu=True, o=None, stream=None):
    """Short causal depthwise convolution over packed prompts (kda_conv_fwd).  x [total, D] bf16
    (rows may be slices of wider ones); weight [D, W] bf16, W in 2..4; bias [D] bf16; cu_seqlens
    int32 [n_seq + 1] or None (n_seq equal sequences); conv0, conv_final [n_seq, W - 1, D] bf16,
    the inputs in front of and at the end of each sequence.  Returns o [total, D] bf16."""
    dev, total, D, W, xp, ldx, wp, bp = _conv_inputs(x, weight, bias)
    cu, n_seq = _runs(cu_seqlens, n_seq, dev)
    held = (n_seq, W - 1, D)
    o, op, ldo = _result(o, (total, D), dev, stream)
    st = lib().kda_conv_fwd(xp, ldx, wp, bp, cu, n_seq, total, D, W, CONV_SILU if silu else 0,
                            _dense(conv0, "conv0", _BF16, held, dev),
                            _dense(conv_final, "conv_final", _BF16, held, dev), op, ldo,
                            _on(stream, dev))
    if st != KDA_OK:
        raise KDAError("kda_conv_fwd", st)
    return o


def conv_tokens(x, weight, bias, conv_pool, slots=None, cu_seqlens=None, used=None, commit=True,
                silu=True, o=None, stream=None):
    """The convolution for single tokens (cu_seqlens None: one token for each row of x) or short
    runs on conv_pool [n_slots, W - 1, D] bf16 (kda_conv_tokens).  slots int32 [n] or None; used
    int32 [n] or None: how many tokens of each run count; commit: whether the pool is advanced.
    o=False: only advance the pool.  Returns o [total, D] bf16, or None."""
    dev, total, D, W, xp, ldx, wp, bp = _conv_inputs(x, weight, bias)
    cu, n = _runs(cu_seqlens, total, dev)
    n_slots = conv_pool.shape[0]
    o, op, ldo = _result(o, (total, D), dev, stream)
    st = lib().kda_conv_tokens(xp, ldx, wp, bp, cu, n, total, D, W, CONV_SILU if silu else 0,
                               _dense(conv_pool, "conv_pool", _BF16, (n_slots, W - 1, D), dev),
                               n_slots, _dense(slots, "slots", _I32, (n,), dev),
                               _dense(used, "used", _I32, (n,), dev), 1 if commit else 0, op, ldo,
                               _on(stream, dev))
    if st != KDA_OK:
        raise KDAError("kda_conv_tokens", st)
    return o


def _ssm_inputs(x, dt, A, B, C, D, z, dt_bias, dt_softplus):
    """(device, sizes, the C arguments from x to flags)"""
    dev = _device(x, "x")
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be [tokens, H, P] and B, C [tokens, G, N]")
    total, H, P = x.shape
    _, G, N = B.shape
    heads, cols, groups = (H,), (total, H, P), (total, G, N)
    if A is None:
        raise TypeError("A must be a torch.Tensor")
    return dev, (total, H, P, G, N), (
        *_rows(x, "x", cols, dev), *_rows(dt, "dt", (total, H), dev),
        _dense(A, "A", _F32, heads, dev), *_rows(B, "B", groups, dev), *_rows(C, "C", groups, dev),
        _dense(D, "D", _F32, heads, dev), *_rows(z, "z", cols, dev),
        _dense(dt_bias, "dt_bias", _F32, heads, dev), SSM_DT_SOFTPLUS if dt_softplus else 0)


def ssm_workspace_bytes(n_seq, total_tokens, H, P, G, N):
    return int(lib().kda_ssm_fwd_workspace_bytes(n_seq, total_tokens, H, P, G, N))


def ssm_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, cu_seqlens=None,
            n_seq=1, S0=None, S_final=None, o=None, workspace=None, stream=None):
    """Selective state space scan over packed prompts (kda_ssm_fwd).  x, z [total, H, P], dt
    [total, H], B, C [total, G, N] bf16 (rows may be slices of wider ones); A, D, dt_bias [H]
    fp32; S0, S_final [n_seq, H, N, P] fp32.  workspace: ssm_workspace_bytes(...) bytes, allocated
    where it is None.  Returns o [total, H, P] bf16."""
    dev, (total, H, P, G, N), args = _ssm_inputs(x, dt, A, B, C, D, z, dt_bias, dt_softplus)
    cu, n_seq = _runs(cu_seqlens, n_seq, dev)
    states = (n_seq, H, N, P)
    o, op, ldo = _result(o, (total, H, P), dev, stream)
    L = lib()
    if workspace is None:
        size = L.kda_ssm_fwd_workspace_bytes(n_seq, total, H, P, G, N)
        workspace = _empty(size, torch.uint8, dev, stream) if size else None
    else:
        if not workspace.is_cuda or workspace.get_device() != dev:
            _refuse(workspace, "workspace", dev)
        if not workspace.is_contiguous():  # (its elements say how large it is)
            raise ValueError("workspace must be contiguous")
        size = workspace.numel() * workspace.element_size()
    st = L.kda_ssm_fwd(*args, cu, n_seq, total, H, P, G, N, _dense(S0, "S0", _F32, states, dev),
                       op, ldo, _dense(S_final, "S_final", _F32, states, dev),
                       0 if workspace is None else workspace.data_ptr(), size, _on(stream, dev))
    if st != KDA_OK:
        raise KDAError("kda_ssm_fwd", st)
    return o


def ssm_tokens(x, dt, A, B, C, state_pool, slots=None, cu_seqlens=None, used=None, commit=True,
               D=None, z=None, dt_bias=None, dt_softplus=True, o=None, stream=None):
    """The scan's recurrence for single tokens (cu_seqlens None: one token for each row of x) or
    short runs on state_pool [n_slots, H, N, P] fp32 (kda_ssm_tokens).  slots, used, commit and
    o=False as for conv_tokens.  Returns o [total, H, P] bf16, or None."""
    dev, (total, H, P, G, N), args = _ssm_inputs(x, dt, A, B, C, D, z, dt_bias, dt_softplus)
    cu, n = _runs(cu_seqlens, total, dev)
    n_slots = state_pool.shape[0]
    o, op, ldo = _result(o, (total, H, P), dev, stream)
    st = lib().kda_ssm_tokens(*args, cu, n, total, H, P, G, N,
                              _dense(state_pool, "state_pool", _F32, (n_slots, H, N, P), dev),
                              n_slots, _dense(slots, "slots", _I32, (n,), dev),
                              _dense(used, "used", _I32, (n,), dev), 1 if commit else 0, op, ldo,
                              _on(stream, dev))
    if st != KDA_OK:
        raise KDAError("kda_ssm_tokens", st)
    return o


def verify_draft(target, tokens, u, cu_seqlens, draft=None, out_tokens=None, n_out=None,
                 stream=None):
    """Verification of drafted runs (kda_verify_draft).  target [total, V] and draft [total - n, V]
    (or None: certain drafts) probabilities, both fp32 or both bf16; tokens int32 [total] and u
    fp32 [total] by run, cu_seqlens int32 [n + 1].  Returns (out_tokens int32 [total], n_out int32
    [n]): the accepted tokens and the drawn one, then -1; and how many there are."""
    if not isinstance(target, _Tensor) or target.dtype not in (_F32, _BF16):
        raise TypeError("target must be a float32 or bfloat16 tensor")
    if target.dim() != 2:
        raise ValueError("target must be [total, V]")
    dev = _device(target, "target")
    total, V = target.shape
    kind, runs = target.dtype, (total,)
    cu, n = _runs(cu_seqlens, -1, dev)
    if out_tokens is None:
        out_tokens = _empty(runs, _I32, dev, stream)
    if n_out is None:
        n_out = _empty((n,), _I32, dev, stream)
    st = lib().kda_verify_draft(_dense(target, "target", kind, (total, V), dev),
                                _dense(draft, "draft", kind, (total - n, V), dev),
                                2 if kind is _BF16 else 4, V,
                                _dense(tokens, "tokens", _I32, runs, dev),
                                _dense(u, "u", _F32, runs, dev), cu, n, total,
                                _dense(out_tokens, "out_tokens", _I32, runs, dev),
                                _dense(n_out, "n_out", _I32, (n,), dev), _on(stream, dev))
    if st != KDA_OK:
        raise KDAError("kda_verify_draft", st)
    return out_tokens, n_out
