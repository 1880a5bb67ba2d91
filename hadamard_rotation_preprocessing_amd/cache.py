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
        return dict(_resolved(self).layout)

    @property
    def page_bytes(self) -> int:
        return _resolved(self).page_bytes


class _Resolved:
    """What the calls need of a spec: the C struct, the page's layout, and the
    scratch sizes asked for so far (attention's, by the sizes and device)."""

    def __init__(self, spec: CacheSpec):
        self.spec = spec.c()
        self.ref = ctypes.byref(self.spec)
        p = hr_cache_page()
        check(_cache_lib().hr_cache_page_layout(self.ref, ctypes.byref(p)))
        self.layout = {n: getattr(p, n) for n, _ in hr_cache_page._fields_}
        self.page_bytes = p.page_bytes
        self.work = {}


_resolved = lru_cache(maxsize=256)(_Resolved)


def cache_pool(spec: CacheSpec, n_pages: int, layers: int | None = None, device="cuda") -> torch.Tensor:
    """Zeroed pages: uint8 [n_pages, page_bytes], or [layers, n_pages, page_bytes]."""
    shape = (n_pages, spec.page_bytes) if layers is None else (layers, n_pages, spec.page_bytes)
    return torch.zeros(shape, dtype=torch.uint8, device=device)


def cache_sections(pool: torch.Tensor, spec: CacheSpec) -> dict:
    """Views of every page's sections, uint8 [..., n_pages, kv_heads, bytes]:
    k_codes, v_codes, k_scales, v_scales and, asymmetric, k_zeros and v_zeros.
    One head of one page is what rotate_quantize_act writes for page_size rows
    of head_dim, so dequant_check reads it (after .contiguous())."""
    lay, q = _resolved(spec).layout, spec.qspec
    groups = spec.page_size * spec.head_dim // q.group_size
    size = {"codes": spec.page_size * spec.head_dim // 2, "scales": groups * (4 if q.scale_dtype == "f32" else 2),
            "zeros": 0 if q.sym else groups // 2}
    heads = pool.unflatten(-1, (spec.kv_heads, lay["head_bytes"]))
    return {"%s_%s" % (x, n): heads[..., lay["%s_%s" % (x, n)]: lay["%s_%s" % (x, n)] + b]
            for n, b in size.items() if b for x in "kv"}


_DTYPES = {torch.float32: L.HR_F32, torch.bfloat16: L.HR_BF16}


def _dt(t):
    if t.dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16, got %s" % t.dtype)
    return _DTYPES[t.dtype]


def _ptr(t):
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> int:
    """The device's current HIP stream (without the Stream object where torch
    has a call for that: these calls are a few microseconds long)."""
    return _raw_stream(device.index) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream


_current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)   # (the latter also initializes: 0.4 us)


def _call(device, fn, *args) -> None:
    """Makes a C call with the tensors' device current: kernels, their sizes and
    the default stream are those of the current device."""
    if _current() == device.index:
        st = fn(*args)
    else:
        with torch.cuda.device(device):
            st = fn(*args)
    if st:
        check(st)


def _ints(t: torch.Tensor, name: str, shape: tuple, device) -> int:
    """Checks a contiguous int32 tensor; its address."""
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError("%s must be a contiguous int32 tensor %s on %s, got %s %s on %s"
                         % (name, list(shape), device, t.dtype, list(t.shape), t.device))
    return t.data_ptr()


def _bytes(work: torch.Tensor, device):
    """(address, bytes) of a caller's scratch."""
    if work.device != device or not work.is_contiguous():
        raise ValueError("work must be a contiguous tensor on %s, got one on %s%s"
                         % (device, work.device, "" if work.is_contiguous() else " with strides %s" % list(work.stride())))
    return work.data_ptr(), work.numel() * work.element_size()


def _table(t: torch.Tensor, device):
    """(address, rows, max_pages) of a page table."""
    if t.dim() != 2:
        raise ValueError("table must be [rows, max_pages], got %s" % list(t.shape))
    return (_ints(t, "table", t.shape, device), *t.shape)


def _pages(pool: torch.Tensor, r: _Resolved, layers: bool):
    """(layers, n_pages) of a pool."""
    if pool.dtype is not torch.uint8 or not pool.is_contiguous() or not (pool.dim() == 2 or (layers and pool.dim() == 3)):
        raise ValueError("pool must be a contiguous uint8 tensor [%sn_pages, page_bytes]" % ("layers, " if layers else ""))
    shape = pool.shape
    if shape[-1] != r.page_bytes:
        raise ValueError("pool pages have %d bytes: the spec's have %d" % (shape[-1], r.page_bytes))
    return (shape[0] if len(shape) == 3 else 1), shape[-2]


def _seqs(table, lens, cu_q, device):
    tp, rows, width = _table(table, device)
    return hr_cache_seqs(tp, _ints(lens, "lens", (rows,), device),
                         None if cu_q is None else _ints(cu_q, "cu_q", (rows + 1,), device), rows, width)


def _vectors(x: torch.Tensor, name: str, tokens, heads, d: int, device):
    """Checks a [tokens, heads, head_dim] tensor (None: any number) whose last
    dimension is contiguous; returns its (token, head) strides."""
    shape = x.shape
    if len(shape) != 3 or shape[2] != d or (heads is not None and shape[1] != heads) or (tokens is not None and shape[0] != tokens):
        raise ValueError("%s must be [%s, %s, %d], got %s" % (name, "tokens" if tokens is None else tokens,
                                                             "heads" if heads is None else heads, d, list(shape)))
    if x.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    st, sh, se = x.stride()
    if se != 1 and x.numel():
        raise ValueError("%s: the last dimension must be contiguous" % name)
    return st, sh


def cache_append(pool: torch.Tensor, spec: CacheSpec, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor,
                 lens: torch.Tensor, cu_q: torch.Tensor | None = None, rotate: bool = True) -> None:
    """Rotates (keys, if ``rotate``) and quantizes the new tokens' k and v
    [tokens, kv_heads, head_dim] into their pages of ``pool`` [n_pages,
    page_bytes].  ``lens`` counts the new tokens already; ``cu_q`` [rows + 1]
    bounds each row's tokens (default: the same number for each)."""
    r, dev = _resolved(spec), pool.device
    _, n = _pages(pool, r, False)
    seqs = _seqs(table, lens, cu_q, dev)
    kt, kh = _vectors(k, "k", None, spec.kv_heads, spec.head_dim, dev)
    tokens = k.shape[0]
    vt, vh = _vectors(v, "v", tokens, spec.kv_heads, spec.head_dim, dev)
    if k.dtype != v.dtype:
        raise ValueError("k and v must have the same dtype")
    _call(dev, _cache_lib().hr_cache_append, pool.data_ptr(), n, r.ref, ctypes.byref(seqs), k.data_ptr(), kt, kh, v.data_ptr(),
          vt, vh, _dt(k), tokens, 1 if rotate else 0, _stream(dev))


def cache_attention(q: torch.Tensor, pool: torch.Tensor, spec: CacheSpec, table: torch.Tensor, lens: torch.Tensor,
                    cu_q: torch.Tensor | None = None, max_q: int = 0, scale: float | None = None, causal: bool = True,
                    window: int = 0, rotate: bool = True, out: torch.Tensor | None = None, lse=None,
                    work: torch.Tensor | None = None):
    """Attention of q [tokens, q_heads, head_dim] over the cache; returns out
    (like q), or (out, lse) with ``lse`` True or a float32 [tokens, q_heads]
    tensor.  ``max_q``: an upper bound of a row's new tokens, if known (it
    only chooses the kernel); ``scale``: None or 0 means 1 / sqrt(head_dim);
    ``work``: scratch of cache_attention_work bytes (allocated if not given)."""
    r, dev, l = _resolved(spec), pool.device, _cache_lib()
    _, n = _pages(pool, r, False)
    seqs = _seqs(table, lens, cu_q, dev)
    qt, qh = _vectors(q, "q", None, None, spec.head_dim, dev)
    tokens, heads = q.shape[0], q.shape[1]
    dt = _dt(q)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    elif out.dtype != q.dtype:
        raise ValueError("out must have q's dtype")
    ot, oh = _vectors(out, "out", tokens, heads, spec.head_dim, dev)
    lp, with_lse = None, lse is not None and lse is not False
    if lse is True:
        lse = torch.empty((tokens, heads), dtype=torch.float32, device=dev)
    if with_lse:
        if lse.dtype is not torch.float32 or lse.shape != (tokens, heads) or not lse.is_contiguous() or lse.device != dev:
            raise ValueError("lse must be a contiguous float32 tensor [tokens, q_heads]")
        lp = lse.data_ptr()
    if scale is not None and scale != 0 and ctypes.c_float(scale).value == 0:
        raise ValueError("scale = %r is 0 in float32" % scale)   # (which would mean the default)
    wp = wb = 0
    if work is not None:
        wp, wb = _bytes(work, dev)
    else:
        key = (dt, tokens, heads, seqs.rows, max_q, dev.index)
        need = r.work.get(key)
        if need is None:
            bytes_ = ctypes.c_int64()
            _call(dev, l.hr_cache_attention_work, dt, tokens, heads, r.ref, seqs.rows, max_q, ctypes.byref(bytes_))
            need = bytes_.value
            if len(r.work) > 4096:
                r.work.clear()
            r.work[key] = need
        if need:
            work = torch.empty(need, dtype=torch.uint8, device=dev)
            wp, wb = work.data_ptr(), need
    _call(dev, l.hr_cache_attention, q.data_ptr(), qt, qh, dt, tokens, heads, pool.data_ptr(), n, r.ref, ctypes.byref(seqs),
          0.0 if scale is None else scale, 1 if causal else 0, window, 1 if rotate else 0, out.data_ptr(), ot, oh, lp, max_q,
          wp, wb, _stream(dev))
    return (out, lse) if with_lse else out


def cache_attention_work(dtype: torch.dtype, tokens: int, q_heads: int, spec: CacheSpec, rows: int, max_q: int = 0) -> int:
    """Bytes of scratch of a cache_attention call on the current device."""
    need = ctypes.c_int64()
    check(_cache_lib().hr_cache_attention_work(_DTYPES[dtype], tokens, q_heads, _resolved(spec).ref, rows, max_q,
                                               ctypes.byref(need)))
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
    pages in use, lacking, copied, free.  ``out``: those four tensors, if the
    caller has them; ``work``: scratch of hr_cache_update_work bytes."""
    r, dev, l = _resolved(spec), pool.device, _cache_lib()
    layers, n = _pages(pool, r, True)
    tp, rows, width = _table(table, dev)
    lp = _ints(lens, "lens", (rows,), dev)
    new = parents.numel()
    pp = _ints(parents, "parents", (new,), dev)
    gp = _ints(grow, "grow", (new,), dev)
    if out is None:
        out = {"table": torch.empty((new, width), dtype=torch.int32, device=dev)}
        out["lens"], out["refs"], out["status"] = torch.empty(new + n + 4, dtype=torch.int32, device=dev).split((new, n, 4))
    if work is None:
        work = _scratch(l.hr_cache_update_work, dev, n, new)
    wp, wb = _bytes(work, dev)
    _call(dev, l.hr_cache_update, pool.data_ptr(), layers, n, r.ref, tp, lp, rows, width, pp, gp, new,
          _ints(out["table"], "out['table']", (new, width), dev), _ints(out["lens"], "out['lens']", (new,), dev),
          _ints(out["refs"], "out['refs']", (n,), dev), _ints(out["status"], "out['status']", (4,), dev), wp, wb, _stream(dev))
    return out


def cache_compact(pool: torch.Tensor, spec: CacheSpec, table: torch.Tensor, lens: torch.Tensor,
                  into: torch.Tensor | None = None, out: dict | None = None, work: torch.Tensor | None = None) -> dict:
    """Moves the live pages to the front of the pool, or copies them into the
    pool ``into``.  Returns dict(table, refs, status): the table in the new
    places, holders of each place, and int32 [4] = live pages, pages without a
    place, moved, free.  ``out``: those three tensors, if the caller has them;
    ``work``: scratch of hr_cache_compact_work bytes."""
    r, dev, l = _resolved(spec), pool.device, _cache_lib()
    layers, n = _pages(pool, r, True)
    tp, rows, width = _table(table, dev)
    lp = _ints(lens, "lens", (rows,), dev)
    places = n
    if into is not None:
        ll, places = _pages(into, r, True)
        if ll != layers or into.device != dev:
            raise ValueError("into must have the pool's layers and device")
    if out is None:
        out = {"table": torch.empty((rows, width), dtype=torch.int32, device=dev)}
        out["refs"], out["status"] = torch.empty(places + 4, dtype=torch.int32, device=dev).split((places, 4))
    if work is None:
        work = _scratch(l.hr_cache_compact_work, dev, n)
    wp, wb = _bytes(work, dev)
    _call(dev, l.hr_cache_compact, pool.data_ptr(), layers, n, r.ref, tp, lp, rows, width, _ptr(into),
          0 if into is None else places, _ints(out["table"], "out['table']", (rows, width), dev),
          _ints(out["refs"], "out['refs']", (places,), dev), _ints(out["status"], "out['status']", (4,), dev), wp, wb, _stream(dev))
    return out
