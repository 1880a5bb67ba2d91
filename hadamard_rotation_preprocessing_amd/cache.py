"""The paged 4-bit key/value cache (C ABI: ``include/hadarot_cache.h``).

Like the package's other entry points these marshal torch tensors and allocate
outputs and scratch with torch; every step runs in the HIP kernels, on the
current stream of the tensors' device.

    CacheSpec(kv_heads, head_dim, page_size, qspec)    what a cache holds
    cache_pool(spec, n_pages, layers=None)             zeroed pages
    cache_sections(pool, spec)                         views of codes, scales and zero points
    cache_append(pool, spec, k, v, table, lens, ...)   -> hr_cache_append
    cache_attention(q, pool, spec, table, lens, ...)   -> hr_cache_attention
    cache_update(pool, spec, table, lens, parents, grow) -> hr_cache_update
    cache_compact(pool, spec, table, lens, into=None)  -> hr_cache_compact
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, field
from functools import lru_cache

import torch

from . import _lib as L
from ._lib import check, lib

# every exported symbol declared in include/hadarot_cache.h
EXPORTS = ("hr_cache_page_layout", "hr_cache_append", "hr_cache_attention", "hr_cache_attention_work",
           "hr_cache_update", "hr_cache_update_work", "hr_cache_compact", "hr_cache_compact_work")


class hr_cache_spec(ctypes.Structure):
    _fields_ = [("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("q", L.hr_qspec)]


class hr_cache_page(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("page_bytes", "head_bytes", "k_codes", "v_codes", "k_scales", "v_scales",
                                              "k_zeros", "v_zeros")]


class hr_cache_seqs(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("cu_q", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("max_pages", ctypes.c_int64)]


_ready = None


def _cache_lib() -> ctypes.CDLL:
    """The library with the cache's entry points declared."""
    global _ready
    if _ready is None:
        l = lib()
        vp, i64, i32, ci, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_float
        sp, sq, out = ctypes.POINTER(hr_cache_spec), ctypes.POINTER(hr_cache_seqs), ctypes.POINTER(i64)
        l.hr_cache_page_layout.argtypes = [sp, ctypes.POINTER(hr_cache_page)]
        l.hr_cache_append.argtypes = [vp, i64, sp, sq, vp, i64, i64, vp, i64, i64, ci, i64, ci, vp]
        l.hr_cache_attention.argtypes = [vp, i64, i64, ci, i64, i32, vp, i64, sp, sq, f32, ci, i64, ci, vp, i64, i64, vp,
                                         i64, vp, i64, vp]
        l.hr_cache_attention_work.argtypes = [ci, i64, i32, sp, i64, i64, out]
        l.hr_cache_update.argtypes = [vp, i64, i64, sp, vp, vp, i64, i64, vp, vp, i64, vp, vp, vp, vp, vp, i64, vp]
        l.hr_cache_update_work.argtypes = [i64, i64, out]
        l.hr_cache_compact.argtypes = [vp, i64, i64, sp, vp, vp, i64, i64, vp, i64, vp, vp, vp, vp, i64, vp]
        l.hr_cache_compact_work.argtypes = [i64, out]
        for n in EXPORTS:
            getattr(l, n).restype = ci
        _ready = l
    return _ready


def _default_qspec():
    from . import QSpec
    return QSpec("int", 4, 128, False, "bf16")


@dataclass(frozen=True)
class CacheSpec:
    """What a cache holds: kv heads, head dimension (64, 128 or 256), positions
    of a page (16 to 256, a power of two) and the quantizer of K and V (INT,
    group_size from 32 to head_dim)."""
    kv_heads: int
    head_dim: int
    page_size: int = 64
    qspec: "QSpec" = field(default_factory=_default_qspec)  # noqa: F821

    def c(self) -> hr_cache_spec:
        return hr_cache_spec(self.kv_heads, self.head_dim, self.page_size, self.qspec.c())

    def layout(self) -> dict:
        """Byte sizes and offsets of the page record (hr_cache_page)."""
        return dict(_layout(self))

    @property
    def page_bytes(self) -> int:
        return _layout(self)["page_bytes"]


@lru_cache(maxsize=None)
def _layout(spec: CacheSpec) -> dict:
    p = hr_cache_page()
    check(_cache_lib().hr_cache_page_layout(ctypes.byref(spec.c()), ctypes.byref(p)))
    return {n: getattr(p, n) for n, _ in hr_cache_page._fields_}


def cache_pool(spec: CacheSpec, n_pages: int, layers: int | None = None, device="cuda") -> torch.Tensor:
    """Zeroed pages: uint8 [n_pages, page_bytes], or [layers, n_pages, page_bytes]."""
    shape = (n_pages, spec.page_bytes) if layers is None else (layers, n_pages, spec.page_bytes)
    return torch.zeros(shape, dtype=torch.uint8, device=device)


def cache_sections(pool: torch.Tensor, spec: CacheSpec) -> dict:
    """Views of every page's sections, uint8 [..., n_pages, kv_heads, bytes]:
    k_codes, v_codes, k_scales, v_scales and, asymmetric, k_zeros and v_zeros.
    One head of one page is what rotate_quantize_act writes for page_size rows
    of head_dim, so dequant_check reads it (after .contiguous())."""
    lay, q = _layout(spec), spec.qspec
    groups = spec.page_size * spec.head_dim // q.group_size
    size = {"codes": spec.page_size * spec.head_dim // 2, "scales": groups * (4 if q.scale_dtype == "f32" else 2),
            "zeros": 0 if q.sym else groups // 2}
    heads = pool.unflatten(-1, (spec.kv_heads, lay["head_bytes"]))
    return {"%s_%s" % (x, n): heads[..., lay["%s_%s" % (x, n)]: lay["%s_%s" % (x, n)] + b]
            for n, b in size.items() if b for x in "kv"}


def _dt(t):
    from . import _dt as dt
    return dt(t)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(t):
    return torch.cuda.current_stream(t.device).cuda_stream


def _ints(t: torch.Tensor, name: str, dim: int, device) -> torch.Tensor:
    if t.dtype != torch.int32 or t.dim() != dim or not t.is_contiguous() or t.device != device:
        raise ValueError("%s must be a contiguous int32 tensor of %d dimension(s) on %s" % (name, dim, device))
    return t


def _pool(pool: torch.Tensor, spec: CacheSpec, layers: bool):
    """(layers, n_pages) of a pool."""
    if pool.dtype != torch.uint8 or not pool.is_contiguous() or pool.dim() not in ((2, 3) if layers else (2,)):
        raise ValueError("pool must be a contiguous uint8 tensor [%sn_pages, page_bytes]" % ("layers, " if layers else ""))
    if pool.shape[-1] != spec.page_bytes:
        raise ValueError("pool pages have %d bytes: the spec's have %d" % (pool.shape[-1], spec.page_bytes))
    return (pool.shape[0] if pool.dim() == 3 else 1), pool.shape[-2]


def _seqs(table, lens, cu_q, device):
    _ints(table, "table", 2, device)
    if _ints(lens, "lens", 1, device).shape[0] != table.shape[0]:
        raise ValueError("lens must have one entry for each row of the table")
    if cu_q is not None and _ints(cu_q, "cu_q", 1, device).shape[0] != table.shape[0] + 1:
        raise ValueError("cu_q must have one entry more than the table has rows")
    return hr_cache_seqs(_ptr(table), _ptr(lens), _ptr(cu_q), table.shape[0], table.shape[1])


def _vectors(x: torch.Tensor, name: str, heads: int | None, spec: CacheSpec, device):
    """Checks a [tokens, heads, head_dim] tensor whose last dimension is
    contiguous; returns its (token, head) strides."""
    if x.dim() != 3 or x.shape[2] != spec.head_dim or (heads is not None and x.shape[1] != heads):
        raise ValueError("%s must be [tokens, %s, %d]" % (name, heads if heads is not None else "heads", spec.head_dim))
    if x.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    if x.numel() and x.stride(2) != 1:
        raise ValueError("%s: the last dimension must be contiguous" % name)
    return x.stride(0), x.stride(1)


def cache_append(pool: torch.Tensor, spec: CacheSpec, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor,
                 lens: torch.Tensor, cu_q: torch.Tensor | None = None, rotate: bool = True) -> None:
    """Rotates (keys, if ``rotate``) and quantizes the new tokens' k and v
    [tokens, kv_heads, head_dim] into their pages of ``pool`` [n_pages,
    page_bytes].  ``lens`` counts the new tokens already; ``cu_q`` [rows + 1]
    bounds each row's tokens (default: the same number for each)."""
    _, n = _pool(pool, spec, False)
    seqs = _seqs(table, lens, cu_q, pool.device)
    ks = _vectors(k, "k", spec.kv_heads, spec, pool.device)
    vs = _vectors(v, "v", spec.kv_heads, spec, pool.device)
    if k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must have the same shape and dtype")
    check(_cache_lib().hr_cache_append(_ptr(pool), n, ctypes.byref(spec.c()), ctypes.byref(seqs), _ptr(k), *ks, _ptr(v), *vs,
                                       _dt(k), k.shape[0], int(rotate), _stream(pool)))


def cache_attention(q: torch.Tensor, pool: torch.Tensor, spec: CacheSpec, table: torch.Tensor, lens: torch.Tensor,
                    cu_q: torch.Tensor | None = None, max_q: int = 0, scale: float | None = None, causal: bool = True,
                    window: int = 0, rotate: bool = True, out: torch.Tensor | None = None, lse=None,
                    work: torch.Tensor | None = None):
    """Attention of q [tokens, q_heads, head_dim] over the cache; returns out
    (like q), or (out, lse) with ``lse`` True or a float32 [tokens, q_heads]
    tensor.  ``max_q``: an upper bound of a row's new tokens, if known (it
    only chooses the kernel); ``work``: scratch of cache_attention_work bytes
    (allocated if not given)."""
    _, n = _pool(pool, spec, False)
    dev = pool.device
    seqs = _seqs(table, lens, cu_q, dev)
    qs = _vectors(q, "q", None, spec, dev)
    tokens, heads = q.shape[0], q.shape[1]
    if out is None:
        out = torch.empty((tokens, heads, spec.head_dim), dtype=q.dtype, device=dev)
    os_ = _vectors(out, "out", heads, spec, dev)
    if out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must have q's shape and dtype")
    want = lse is not None and lse is not False
    if lse is True:
        lse = torch.empty((tokens, heads), dtype=torch.float32, device=dev)
    elif want and (lse.dtype != torch.float32 or lse.shape != (tokens, heads) or not lse.is_contiguous() or lse.device != dev):
        raise ValueError("lse must be a contiguous float32 tensor [tokens, q_heads]")
    dt, l = _dt(q), _cache_lib()
    cs = spec.c()
    with torch.cuda.device(dev):
        if work is None:
            need = ctypes.c_int64()
            check(l.hr_cache_attention_work(dt, tokens, heads, ctypes.byref(cs), table.shape[0], max_q, ctypes.byref(need)))
            work = torch.empty(need.value, dtype=torch.uint8, device=dev) if need.value else None
        check(l.hr_cache_attention(_ptr(q), *qs, dt, tokens, heads, _ptr(pool), n, ctypes.byref(cs), ctypes.byref(seqs),
                                   0.0 if scale is None else scale, int(causal), window, int(rotate), _ptr(out), *os_,
                                   _ptr(lse) if want else None, max_q, _ptr(work), 0 if work is None else work.numel(),
                                   _stream(pool)))
    return (out, lse) if want else out


def cache_attention_work(dtype: torch.dtype, tokens: int, q_heads: int, spec: CacheSpec, rows: int, max_q: int = 0) -> int:
    """Bytes of scratch of a cache_attention call on the current device."""
    dt = {torch.float32: L.HR_F32, torch.bfloat16: L.HR_BF16}[dtype]
    need = ctypes.c_int64()
    check(_cache_lib().hr_cache_attention_work(dt, tokens, q_heads, ctypes.byref(spec.c()), rows, max_q, ctypes.byref(need)))
    return need.value


def _scratch(fn, device, *sizes):
    need = ctypes.c_int64()
    check(fn(*sizes, ctypes.byref(need)))
    return torch.empty(need.value, dtype=torch.uint8, device=device)


def cache_update(pool: torch.Tensor, spec: CacheSpec, table: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor,
                 grow: torch.Tensor, out: dict | None = None, work: torch.Tensor | None = None) -> dict:
    """One scheduling step: row i of the new table continues row parents[i]
    (-1: a new sequence) grown by grow[i] positions.  Shares full pages, copies
    partly filled ones that two rows would write, hands out free pages in
    ascending order; rows that are nobody's parent give theirs up.  Returns
    dict(table, lens, refs, status): holders of each page, and int32 [4] =
    pages in use, lacking, copied, free."""
    layers, n = _pool(pool, spec, True)
    dev = pool.device
    _seqs(table, lens, None, dev)
    rows = _ints(parents, "parents", 1, dev).shape[0]
    if _ints(grow, "grow", 1, dev).shape[0] != rows:
        raise ValueError("parents and grow must have the same length")
    i32 = dict(dtype=torch.int32, device=dev)
    if out is None:
        out = {"table": torch.empty((rows, table.shape[1]), **i32), "lens": torch.empty(rows, **i32),
               "refs": torch.empty(n, **i32), "status": torch.empty(4, **i32)}
    for name, shape in (("table", (rows, table.shape[1])), ("lens", (rows,)), ("refs", (n,)), ("status", (4,))):
        if _ints(out[name], name, len(shape), dev).shape != shape:
            raise ValueError("out[%r] must be %s" % (name, shape))
    l = _cache_lib()
    if work is None:
        work = _scratch(l.hr_cache_update_work, dev, n, rows)
    check(l.hr_cache_update(_ptr(pool), layers, n, ctypes.byref(spec.c()), _ptr(table), _ptr(lens), table.shape[0],
                            table.shape[1], _ptr(parents), _ptr(grow), rows, _ptr(out["table"]), _ptr(out["lens"]),
                            _ptr(out["refs"]), _ptr(out["status"]), _ptr(work), work.numel(), _stream(pool)))
    return out


def cache_compact(pool: torch.Tensor, spec: CacheSpec, table: torch.Tensor, lens: torch.Tensor,
                  into: torch.Tensor | None = None, out: dict | None = None, work: torch.Tensor | None = None) -> dict:
    """Moves the live pages to the front of the pool, or copies them into the
    pool ``into``.  Returns dict(table, refs, status): the table in the new
    places, holders of each place, and int32 [4] = live pages, pages without a
    place, moved, free."""
    layers, n = _pool(pool, spec, True)
    dev = pool.device
    _seqs(table, lens, None, dev)
    places = n
    if into is not None:
        ll, places = _pool(into, spec, True)
        if ll != layers or into.device != dev:
            raise ValueError("into must have the pool's layers and device")
    i32 = dict(dtype=torch.int32, device=dev)
    if out is None:
        out = {"table": torch.empty(tuple(table.shape), **i32), "refs": torch.empty(places, **i32),
               "status": torch.empty(4, **i32)}
    for name, shape in (("table", tuple(table.shape)), ("refs", (places,)), ("status", (4,))):
        if tuple(_ints(out[name], name, len(shape), dev).shape) != shape:
            raise ValueError("out[%r] must be %s" % (name, shape))
    l = _cache_lib()
    if work is None:
        work = _scratch(l.hr_cache_compact_work, dev, n)
    check(l.hr_cache_compact(_ptr(pool), layers, n, ctypes.byref(spec.c()), _ptr(table), _ptr(lens), table.shape[0],
                             table.shape[1], _ptr(into), places if into is not None else 0, _ptr(out["table"]),
                             _ptr(out["refs"]), _ptr(out["status"]), _ptr(work), work.numel(), _stream(pool)))
    return out
