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

from . import KDA_OK, KDAError, _check, _ptr, _stream, lib

CONV_SILU = 1         # KDA_CONV_SILU
SSM_DT_SOFTPLUS = 1   # KDA_SSM_DT_SOFTPLUS


def _rows(t, name, shape):
    """Row stride of a bf16 CUDA tensor [tokens, ...] whose rows are dense (slices of wider rows
    are taken as they are)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    strides = t.stride()
    dense = 1
    for n, s in zip(shape[:0:-1], strides[:0:-1]):
        if n > 1 and s != dense:
            raise ValueError(f"{name} must have dense rows, got strides {strides}")
        dense *= n
    # the stride of a single row means nothing
    return strides[0] if shape[0] > 1 else dense


def _batch(cu_seqlens, n, total):
    """Number of runs, from cu_seqlens where given."""
    if cu_seqlens is None:
        return n
    _check(cu_seqlens, "cu_seqlens", torch.int32)
    return cu_seqlens.numel() - 1


def _empty(shape, dtype, device, stream):
    """A new tensor that belongs to the stream of the call, so that the allocator cannot hand it
    to the call while earlier work of another stream still uses it, nor away from it."""
    if isinstance(stream, torch.cuda.Stream):
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


def _result(o, like, shape, stream):
    """(output tensor or None, its row stride)"""
    if o is False:
        return None, 0
    if o is None:
        o = _empty(shape, torch.bfloat16, like.device, stream)
    return o, _rows(o, "o", shape)


def _on_device(ref, *tensors):
    """The tensors of one call live on one device, the current one."""
    if ref.device.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {ref.device}, not on the current device")
    for t in tensors:
        if t is not None and t is not False and t.device != ref.device:
            raise ValueError(f"tensors are on {ref.device} and {t.device}")


def _pool(slots, used, n, n_slots):
    if slots is not None:
        _check(slots, "slots", torch.int32, (n,))
    elif n_slots < n:
        raise ValueError("the pool has fewer slots than runs")
    if used is not None:
        _check(used, "used", torch.int32, (n,))


def _conv_check(x, weight, bias):
    if x.dim() != 2 or weight.dim() != 2:
        raise ValueError("x must be [tokens, D] and weight [D, W]")
    total, D = x.shape
    ldx = _rows(x, "x", (total, D))
    _check(weight, "weight", torch.bfloat16, (D, weight.shape[1]))
    if bias is not None:
        _check(bias, "bias", torch.bfloat16, (D,))
    return total, D, weight.shape[1], ldx


def conv_fwd(x, weight, bias=None, cu_seqlens=None, n_seq=1, conv0=None, conv_final=None,
             silu=True, o=None, stream=None):
    """Short causal depthwise convolution over packed prompts (kda_conv_fwd).  x [total, D] bf16
    (rows may be slices of wider ones); weight [D, W] bf16, W in 2..4; bias [D] bf16; cu_seqlens
    int32 [n_seq + 1] or None (n_seq equal sequences); conv0, conv_final [n_seq, W - 1, D] bf16,
    the inputs in front of and at the end of each sequence.  Returns o [total, D] bf16."""
    total, D, W, ldx = _conv_check(x, weight, bias)
    n_seq = _batch(cu_seqlens, n_seq, total)
    for t, nm in ((conv0, "conv0"), (conv_final, "conv_final")):
        if t is not None:
            _check(t, nm, torch.bfloat16, (n_seq, W - 1, D))
    o, ldo = _result(o, x, (total, D), stream)
    _on_device(x, weight, bias, cu_seqlens, conv0, conv_final, o)
    st = lib().kda_conv_fwd(_ptr(x), ldx, _ptr(weight), _ptr(bias), _ptr(cu_seqlens), n_seq, total,
                            D, W, CONV_SILU if silu else 0, _ptr(conv0), _ptr(conv_final), _ptr(o),
                            ldo, _stream(stream))
    if st != KDA_OK:
        raise KDAError("kda_conv_fwd", st)
    return o


def conv_tokens(x, weight, bias, conv_pool, slots=None, cu_seqlens=None, used=None, commit=True,
                silu=True, o=None, stream=None):
    """The convolution for single tokens (cu_seqlens None: one token for each row of x) or short
    runs on conv_pool [n_slots, W - 1, D] bf16 (kda_conv_tokens).  slots int32 [n] or None; used
    int32 [n] or None: how many tokens of each run count; commit: whether the pool is advanced.
    o=False: only advance the pool.  Returns o [total, D] bf16, or None."""
    total, D, W, ldx = _conv_check(x, weight, bias)
    n = _batch(cu_seqlens, total, total)
    _check(conv_pool, "conv_pool", torch.bfloat16, (conv_pool.shape[0], W - 1, D))
    _pool(slots, used, n, conv_pool.shape[0])
    o, ldo = _result(o, x, (total, D), stream)
    _on_device(x, weight, bias, cu_seqlens, conv_pool, slots, used, o)
    st = lib().kda_conv_tokens(_ptr(x), ldx, _ptr(weight), _ptr(bias), _ptr(cu_seqlens), n, total,
                               D, W, CONV_SILU if silu else 0, _ptr(conv_pool),
                               conv_pool.shape[0], _ptr(slots), _ptr(used), 1 if commit else 0,
                               _ptr(o), ldo, _stream(stream))
    if st != KDA_OK:
        raise KDAError("kda_conv_tokens", st)
    return o


def _ssm_check(x, dt, A, B, C, D, z, dt_bias):
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be [tokens, H, P] and B, C [tokens, G, N]")
    total, H, P = x.shape
    G, N = B.shape[1:]
    ld = [_rows(x, "x", (total, H, P)), _rows(dt, "dt", (total, H)), _rows(B, "B", (total, G, N)),
          _rows(C, "C", (total, G, N)), 0 if z is None else _rows(z, "z", (total, H, P))]
    for t, nm in ((A, "A"), (D, "D"), (dt_bias, "dt_bias")):
        if t is not None or nm == "A":
            _check(t, nm, torch.float32, (H,))
    return total, H, P, G, N, ld


def ssm_workspace_bytes(n_seq, total_tokens, H, P, G, N):
    return int(lib().kda_ssm_fwd_workspace_bytes(n_seq, total_tokens, H, P, G, N))


def ssm_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, cu_seqlens=None,
            n_seq=1, S0=None, S_final=None, o=None, workspace=None, stream=None):
    """Selective state space scan over packed prompts (kda_ssm_fwd).  x, z [total, H, P], dt
    [total, H], B, C [total, G, N] bf16 (rows may be slices of wider ones); A, D, dt_bias [H]
    fp32; S0, S_final [n_seq, H, N, P] fp32.  workspace: ssm_workspace_bytes(...) bytes, allocated
    where it is None.  Returns o [total, H, P] bf16."""
    total, H, P, G, N, ld = _ssm_check(x, dt, A, B, C, D, z, dt_bias)
    n_seq = _batch(cu_seqlens, n_seq, total)
    for t, nm in ((S0, "S0"), (S_final, "S_final")):
        if t is not None:
            _check(t, nm, torch.float32, (n_seq, H, N, P))
    o, ldo = _result(o, x, (total, H, P), stream)
    _on_device(x, dt, A, B, C, D, z, dt_bias, cu_seqlens, S0, S_final, o, workspace)
    if workspace is None:
        need = ssm_workspace_bytes(n_seq, total, H, P, G, N)
        if need:
            workspace = _empty(need, torch.uint8, x.device, stream)
    size = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().kda_ssm_fwd(_ptr(x), ld[0], _ptr(dt), ld[1], _ptr(A), _ptr(B), ld[2], _ptr(C),
                           ld[3], _ptr(D), _ptr(z), ld[4], _ptr(dt_bias),
                           SSM_DT_SOFTPLUS if dt_softplus else 0, _ptr(cu_seqlens), n_seq, total,
                           H, P, G, N, _ptr(S0), _ptr(o), ldo, _ptr(S_final), _ptr(workspace),
                           size, _stream(stream))
    if st != KDA_OK:
        raise KDAError("kda_ssm_fwd", st)
    return o


def ssm_tokens(x, dt, A, B, C, state_pool, slots=None, cu_seqlens=None, used=None, commit=True,
               D=None, z=None, dt_bias=None, dt_softplus=True, o=None, stream=None):
    """The scan's recurrence for single tokens (cu_seqlens None: one token for each row of x) or
    short runs on state_pool [n_slots, H, N, P] fp32 (kda_ssm_tokens).  slots, used, commit and
    o=False as for conv_tokens.  Returns o [total, H, P] bf16, or None."""
    total, H, P, G, N, ld = _ssm_check(x, dt, A, B, C, D, z, dt_bias)
    n = _batch(cu_seqlens, total, total)
    _check(state_pool, "state_pool", torch.float32, (state_pool.shape[0], H, N, P))
    _pool(slots, used, n, state_pool.shape[0])
    o, ldo = _result(o, x, (total, H, P), stream)
    _on_device(x, dt, A, B, C, D, z, dt_bias, cu_seqlens, state_pool, slots, used, o)
    st = lib().kda_ssm_tokens(_ptr(x), ld[0], _ptr(dt), ld[1], _ptr(A), _ptr(B), ld[2], _ptr(C),
                              ld[3], _ptr(D), _ptr(z), ld[4], _ptr(dt_bias),
                              SSM_DT_SOFTPLUS if dt_softplus else 0, _ptr(cu_seqlens), n, total, H,
                              P, G, N, _ptr(state_pool), state_pool.shape[0], _ptr(slots),
                              _ptr(used), 1 if commit else 0, _ptr(o), ldo, _stream(stream))
    if st != KDA_OK:
        raise KDAError("kda_ssm_tokens", st)
    return o


def verify_draft(target, tokens, u, cu_seqlens, draft=None, out_tokens=None, n_out=None,
                 stream=None):
    """Verification of drafted runs (kda_verify_draft).  target [total, V] and draft [total - n, V]
    (or None: certain drafts) probabilities, both fp32 or both bf16; tokens int32 [total] and u
    fp32 [total] by run, cu_seqlens int32 [n + 1].  Returns (out_tokens int32 [total], n_out int32
    [n]): the accepted tokens and the drawn one, then -1; and how many there are."""
    if not isinstance(target, torch.Tensor) or target.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("target must be a float32 or bfloat16 tensor")
    if target.dim() != 2:
        raise ValueError("target must be [total, V]")
    total, V = target.shape
    _check(target, "target", target.dtype)
    _check(cu_seqlens, "cu_seqlens", torch.int32)
    n = cu_seqlens.numel() - 1
    _check(tokens, "tokens", torch.int32, (total,))
    _check(u, "u", torch.float32, (total,))
    if draft is not None:
        _check(draft, "draft", target.dtype, (total - n, V))
    if out_tokens is None:
        out_tokens = _empty(total, torch.int32, target.device, stream)
    _check(out_tokens, "out_tokens", torch.int32, (total,))
    if n_out is None:
        n_out = _empty(n, torch.int32, target.device, stream)
    _check(n_out, "n_out", torch.int32, (n,))
    _on_device(target, tokens, u, cu_seqlens, draft, out_tokens, n_out)
    st = lib().kda_verify_draft(_ptr(target), _ptr(draft), target.element_size(), V, _ptr(tokens),
                                _ptr(u), _ptr(cu_seqlens), n, total, _ptr(out_tokens), _ptr(n_out),
                                _stream(stream))
    if st != KDA_OK:
        raise KDAError("kda_verify_draft", st)
    return out_tokens, n_out
