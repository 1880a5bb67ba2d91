"""Eviction from the paged 4-bit key/value cache (C ABI: ``include/hadarot_evict.h``).

    cache_weights(q, pool, spec, table, lens, lse, weights, ...)  -> hr_cache_weights
    cache_evict(pool, spec, table, lens, weights, budget, ...)    -> hr_cache_evict

A decoding step with eviction appends and attends as always (cache.py), adds the
step's attention weights, and from time to time cuts the rows that have grown
past their budget:

    o, lse = cache_attention(q, pool[i], spec, table, lens, lse=True)
    cache_weights(q, pool[i], spec, table, lens, lse, weights[i])
    ...
    step = cache_evict(pool, spec, table, lens, weights, budget=4096, sinks=4, recent=64)
"""
from __future__ import annotations

import ctypes

import torch

from . import cache as K
from .cache import CacheSpec, hr_cache_seqs, hr_cache_spec

# every exported symbol declared in include/hadarot_evict.h
EXPORTS = ("hr_cache_weights", "hr_cache_weights_work", "hr_cache_evict", "hr_cache_evict_work")

_ready = None


def _evict_lib() -> ctypes.CDLL:
    """The library with the eviction's entry points declared."""
    global _ready
    if _ready is None:
        l = K._cache_lib()
        vp, i64, i32, ci, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_float
        sp, sq, out = ctypes.POINTER(hr_cache_spec), ctypes.POINTER(hr_cache_seqs), ctypes.POINTER(i64)
        l.hr_cache_weights.argtypes = [vp, i64, i64, ci, i64, i32, vp, i64, sp, sq, vp, f32, ci, i64, ci, f32, vp, i64, i64, vp,
                                       i64, vp]
        l.hr_cache_weights_work.argtypes = [ci, i64, i32, sp, i64, i64, out]
        l.hr_cache_evict.argtypes = [vp, i64, i64, sp, vp, vp, i64, i64, vp, i64, i64, i64, i64, vp, vp, vp, vp, vp, i64, vp]
        l.hr_cache_evict_work.argtypes = [i64, i64, out]
        for n in EXPORTS:
            getattr(l, n).restype = ci
        _ready = l
    return _ready


def _weights(t: torch.Tensor, shape: tuple, device) -> int:
    """Checks the float32 weights [*shape, width]; the width."""
    if t.dtype is not torch.float32 or t.dim() != len(shape) + 1 or t.shape[:-1] != shape or not t.is_contiguous() or t.device != device:
        raise ValueError("weights must be a contiguous float32 tensor %s on %s, got %s %s on %s"
                         % ([*shape, "width"], device, t.dtype, list(t.shape), t.device))
    return t.shape[-1]


def cache_weights(q: torch.Tensor, pool: torch.Tensor, spec: CacheSpec, table: torch.Tensor, lens: torch.Tensor,
                  lse: torch.Tensor, weights: torch.Tensor, cu_q: torch.Tensor | None = None, max_q: int = 0,
                  scale: float | None = None, causal: bool = True, window: int = 0, rotate: bool = True, decay: float = 1.0,
                  work: torch.Tensor | None = None) -> torch.Tensor:
    """Adds to ``weights`` (float32 [rows, kv_heads, width], width at least
    max_pages * page_size) the attention weight that each position gets from the
    new tokens q [tokens, q_heads, head_dim], whose log-sum-exp cache_attention
    gave with the same arguments; earlier positions' weights are multiplied by
    ``decay`` first, new positions start at 0.  A token whose lse is -inf adds
    nothing, whatever its query is.  Returns ``weights``.  ``work``:
    scratch of hr_cache_weights_work bytes (allocated if not given)."""
    r, dev, l = K._resolved(spec), pool.device, _evict_lib()
    _, n = K._pages(pool, r, False)
    seqs = K._seqs(table, lens, cu_q, dev)
    qt, qh = K._vectors(q, "q", None, None, spec.head_dim, dev)
    tokens, heads = q.shape[0], q.shape[1]
    dt = K._dt(q)
    if lse.dtype is not torch.float32 or lse.shape != (tokens, heads) or not lse.is_contiguous() or lse.device != dev:
        raise ValueError("lse must be a contiguous float32 tensor [tokens, q_heads] = %s on %s" % ([tokens, heads], dev))
    width = _weights(weights, (seqs.rows, spec.kv_heads), dev)
    if scale is not None and scale != 0 and ctypes.c_float(scale).value == 0:
        raise ValueError("scale = %r is 0 in float32" % scale)   # (which would mean the default)
    wp = wb = 0
    if work is not None:
        wp, wb = K._bytes(work, dev)
    else:
        key = ("weights", dt, tokens, heads, seqs.rows, max_q, dev.index)
        need = r.work.get(key)
        if need is None:
            bytes_ = ctypes.c_int64()
            K._call(dev, l.hr_cache_weights_work, dt, tokens, heads, r.ref, seqs.rows, max_q, ctypes.byref(bytes_))
            need = bytes_.value
            if len(r.work) > 4096:
                r.work.clear()
            r.work[key] = need
        if need:
            work = torch.empty(need, dtype=torch.uint8, device=dev)
            wp, wb = work.data_ptr(), need
    K._call(dev, l.hr_cache_weights, q.data_ptr(), qt, qh, dt, tokens, heads, pool.data_ptr(), n, r.ref, ctypes.byref(seqs),
            lse.data_ptr(), 0.0 if scale is None else scale, 1 if causal else 0, window, 1 if rotate else 0, decay,
            weights.data_ptr(), width, max_q, wp, wb, K._stream(dev))
    return weights


def cache_evict(pool: torch.Tensor, spec: CacheSpec, table: torch.Tensor, lens: torch.Tensor, weights: torch.Tensor,
                budget: int, sinks: int = 0, recent: int = 0, out: dict | None = None, work: torch.Tensor | None = None) -> dict:
    """Cuts every row of more than ``budget`` positions to that many: the first
    ``sinks``, the last ``recent``, and the heaviest of the others by ``weights``
    (float32 [rows, kv_heads, width], with a leading dimension of layers where the
    pool has one), for each layer and kv head, moved together in their order in
    ``pool`` and ``weights``.  Returns dict(table, lens, refs, status): holders of
    each page, and int32 [4] = pages in use, lacking, rows evicted, pages free.
    ``out``: those four tensors, if the caller has them; ``work``: scratch of
    hr_cache_evict_work bytes."""
    r, dev, l = K._resolved(spec), pool.device, _evict_lib()
    layers, n = K._pages(pool, r, True)
    tp, rows, width = K._table(table, dev)
    lp = K._ints(lens, "lens", (rows,), dev)
    wide = _weights(weights, (layers, rows, spec.kv_heads) if pool.dim() == 3 else (rows, spec.kv_heads), dev)
    if out is None:
        out = {"table": torch.empty((rows, width), dtype=torch.int32, device=dev)}
        out["lens"], out["refs"], out["status"] = torch.empty(rows + n + 4, dtype=torch.int32, device=dev).split((rows, n, 4))
    if work is None:
        work = K._scratch(l.hr_cache_evict_work, dev, n, rows)
    wp, wb = K._bytes(work, dev)
    K._call(dev, l.hr_cache_evict, pool.data_ptr(), layers, n, r.ref, tp, lp, rows, width, weights.data_ptr(), wide, budget, sinks,
            recent, K._ints(out["table"], "out['table']", (rows, width), dev), K._ints(out["lens"], "out['lens']", (rows,), dev),
            K._ints(out["refs"], "out['refs']", (n,), dev), K._ints(out["status"], "out['status']", (4,), dev), wp, wb,
            K._stream(dev))
    return out
