"""The paged cache of the attention layers that stand between the recurrent ones: writing keys and
values into it, attention over it, and its pages (``include/kda.h`` has every argument's layout).
As in the rest of the binding, everything here checks and marshals.

A step of a batch of runs (prompt chunks, single tokens, drafted runs)::

    pages_grow(table, lens, want, page, n_pages)                # want: lens + the runs' tokens
    for each layer:
        kv_append(k, v, cache[layer], table, lens, slots, cu)
        o = attn_paged(q, cache[layer], table, lens, slots, cu)
    lens[slots.long()] += tokens that stand                     # verify_draft's n_out, say
"""
from __future__ import annotations

import functools

import torch

from . import KDA_OK, KDAError, lib
from .serving import (_BF16, _I32, _dense, _device, _empty, _on, _refuse, _result, _rows, _runs,
                      _Tensor)


def _cache(cache, layers, dev):
    """(address, layers, n_pages, H, page, D) of a cache of one layer or of several."""
    if not isinstance(cache, _Tensor):
        raise TypeError("cache must be a torch.Tensor")
    shape = cache.shape
    if not (len(shape) == 5 or layers and len(shape) == 6) or shape[-4] != 2:
        raise ValueError(f"cache must be {'[layers, ' if layers else '['}n_pages, 2, H, page, D], "
                         f"got {tuple(shape)}")
    at = _dense(cache, "cache", _BF16, shape, dev)
    return (at, shape[0] if len(shape) == 6 else 1, shape[-5], *shape[-3:])


def _table(table, lens, dev):
    """(address of the table, max_pages, address of lens, n_slots)"""
    if not isinstance(table, _Tensor) or table.dim() != 2:
        raise TypeError("table must be an int32 tensor [n_slots, max_pages]")
    n_slots, most = table.shape
    if lens is None:
        raise TypeError("lens must be a torch.Tensor")
    return (_dense(table, "table", _I32, (n_slots, most), dev), most,
            _dense(lens, "lens", _I32, (n_slots,), dev), n_slots)


def _int32(v, name):
    """v, which the C call takes as an int: others would be cut to 32 bits without a word."""
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name} must be a 32-bit integer, got {v}")
    return v


def _scratch(workspace, size, dev, stream):
    """(the workspace, its address, its bytes)"""
    if workspace is None:
        workspace = _empty(size, torch.uint8, dev, stream) if size else None
        return workspace, 0 if workspace is None else workspace.data_ptr(), size
    if not isinstance(workspace, _Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if not workspace.is_cuda or workspace.get_device() != dev:
        _refuse(workspace, "workspace", dev)
    if not workspace.is_contiguous():  # (its elements say how large it is)
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def kv_append(k, v, cache, table, lens, slots=None, cu_seqlens=None, stream=None):
    """Writes the keys and values of a batch of runs behind the lens[slot] tokens of their slots
    (kda_kv_append).  k, v [total, H, D] bf16 (rows may be slices of wider ones); cache [n_pages,
    2, H, page, D] bf16; table int32 [n_slots, max_pages]; lens int32 [n_slots]; slots int32 [n]
    or None (run b is slot b); cu_seqlens int32 [n + 1] or None (one token for each row)."""
    dev = _device(k, "k")
    if k.dim() != 3:
        raise ValueError("k must be [tokens, H, D]")
    total, H, D = k.shape
    cu, n = _runs(cu_seqlens, total, dev)
    if v is None:
        raise TypeError("v must be a torch.Tensor")
    at, _, n_pages, H_c, page, D_c = _cache(cache, False, dev)
    if (H_c, D_c) != (H, D):
        raise ValueError(f"cache has {H_c} heads of {D_c}, k {H} of {D}")
    tp, most, lp, n_slots = _table(table, lens, dev)
    st = lib().kda_kv_append(*_rows(k, "k", (total, H, D), dev), *_rows(v, "v", (total, H, D), dev),
                             cu, n, total, H, D, at, n_pages, page, tp, most, lp, n_slots,
                             _dense(slots, "slots", _I32, (n,), dev), _on(stream, dev))
    if st != KDA_OK:
        raise KDAError("kda_kv_append", st)


@functools.lru_cache(maxsize=256)  # (a function of the sizes alone, and 0.7 us of a call)
def attn_workspace_bytes(n, total_tokens, Hq, H, D):
    return int(lib().kda_attn_paged_workspace_bytes(n, total_tokens, Hq, H, D))


@functools.lru_cache(maxsize=256)
def _pages_workspace_bytes(n):
    return int(lib().kda_pages_workspace_bytes(n))


def attn_paged(q, cache, table, lens, slots=None, cu_seqlens=None, scale=None, window=0, o=None,
               workspace=None, stream=None):
    """Causal attention of a batch of runs over the pages of their sequences (kda_attn_paged).  q
    [total, Hq, D] bf16 (rows may be slices of wider ones); cache, table, lens, slots and
    cu_seqlens as for kv_append, which has put the runs' own keys and values there; scale: D ** -0.5
    where it is None; window: the positions a token sees, 0 for all.  workspace:
    attn_workspace_bytes(...) bytes, allocated where it is None.  Returns o [total, Hq, D] bf16."""
    dev = _device(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [tokens, Hq, D]")
    total, Hq, D = q.shape
    cu, n = _runs(cu_seqlens, total, dev)
    at, _, n_pages, H, page, D_c = _cache(cache, False, dev)
    if D_c != D:
        raise ValueError(f"cache has heads of {D_c}, q of {D}")
    tp, most, lp, n_slots = _table(table, lens, dev)
    o, op, ldo = _result(o, (total, Hq, D), dev, stream)
    workspace, wp, size = _scratch(
        workspace, attn_workspace_bytes(n, total, Hq, H, D), dev, stream)
    st = lib().kda_attn_paged(*_rows(q, "q", (total, Hq, D), dev), cu, n, total, Hq, H, D, at, n_pages,
                          page, tp, most, lp, n_slots, _dense(slots, "slots", _I32, (n,), dev),
                          D ** -0.5 if scale is None else scale, _int32(window, "window"), op, ldo, wp, size,
                          _on(stream, dev))
    if st != KDA_OK:
        raise KDAError("kda_attn_paged", st)
    return o


def _count(t, name, dev, stream):
    if t is None:
        t = _empty((1,), _I32, dev, stream)
    return t, _dense(t, name, _I32, (1,), dev)


def pages_grow(table, lens, want, page, n_pages, left=None, stream=None):
    """Gives rows of the table the lowest unused pages of a pool of n_pages for want[s] instead of
    lens[s] tokens (kda_pages_grow), in place.  want int32 [n_slots].  Returns left int32 [1]: the
    pages still unused, negative where as many are missing."""
    dev = _device(table, "table")
    tp, most, lp, n_slots = _table(table, lens, dev)
    if want is None:
        raise TypeError("want must be a torch.Tensor")
    left, cp = _count(left, "left", dev, stream)
    st = lib().kda_pages_grow(tp, most, lp, _dense(want, "want", _I32, (n_slots,), dev), n_slots,
                              _int32(n_pages, "n_pages"), _int32(page, "page"), cp, _on(stream, dev))
    if st != KDA_OK:
        raise KDAError("kda_pages_grow", st)
    return left


def pages_fork(cache, table, lens, src, dst, left=None, workspace=None, stream=None):
    """Lets slots dst continue what slots src hold (kda_pages_fork), in place on table, lens and
    cache ([layers, n_pages, 2, H, page, D] or one layer's).  src, dst int32 [n].  Returns left
    int32 [1], as pages_grow."""
    dev = _device(cache, "cache")
    at, layers, n_pages, H, page, D = _cache(cache, True, dev)
    tp, most, lp, n_slots = _table(table, lens, dev)
    if not isinstance(src, _Tensor) or dst is None:
        raise TypeError("src and dst must be int32 tensors")
    n = src.numel()
    left, cp = _count(left, "left", dev, stream)
    workspace, wp, size = _scratch(workspace, _pages_workspace_bytes(n), dev, stream)
    st = lib().kda_pages_fork(at, layers, n_pages, H, page, D, tp, most, lp, n_slots,
                          _dense(src, "src", _I32, (n,), dev), _dense(dst, "dst", _I32, (n,), dev),
                          n, cp, wp, size, _on(stream, dev))
    if st != KDA_OK:
        raise KDAError("kda_pages_fork", st)
    return left


def pages_compact(cache, table, lens, table_out=None, used=None, workspace=None, stream=None):
    """Moves the pages in use to the front of the pool (kda_pages_compact), in place on cache
    ([layers, n_pages, 2, H, page, D] or one layer's).  Returns (the table with the new numbers: a
    new one, or table_out, which may be table; used int32 [1]: how many pages are in use)."""
    dev = _device(cache, "cache")
    at, layers, n_pages, H, page, D = _cache(cache, True, dev)
    tp, most, lp, n_slots = _table(table, lens, dev)
    if table_out is None:
        table_out = _empty((n_slots, most), _I32, dev, stream)
    used, cp = _count(used, "used", dev, stream)
    workspace, wp, size = _scratch(workspace, _pages_workspace_bytes(n_pages), dev, stream)
    st = lib().kda_pages_compact(at, layers, n_pages, H, page, D, tp, most, lp, n_slots,
                             _dense(table_out, "table_out", _I32, (n_slots, most), dev), cp, wp,
                             size, _on(stream, dev))
    if st != KDA_OK:
        raise KDAError("kda_pages_compact", st)
    return table_out, used
