"""Latent attention over a paged 4-bit cache (C ABI: ``include/hadarot_latent.h``).

A position holds one latent, that all heads' keys and values are linear maps of,
in 4 bits, and one rotary key that all heads share:

    LatentSpec(latent_dim, rope_dim, page_size, qspec)     what a cache holds
    latent_append(pool, spec, c, rope, table, lens, ...)   -> hr_latent_append
    latent_read(pool, spec, table, lens, cu_k, n, ...)     -> hr_latent_read
    latent_attention(q, q_rope, pool, spec, ...)           -> hr_latent_attention
    latent_prompt_attention(q, k, rope, v, cu_q, cu_k)     -> hr_latent_prompt_attention

cache_pool, cache_update and cache_compact (cache.py) take a LatentSpec too.  With
the maps wk [heads, nope, latent] and wv [heads, nope, latent] of a layer, single
tokens attend in the latent's space,

    q_c = torch.bmm(q[..., :nope].transpose(0, 1), wk).transpose(0, 1)
    o = latent_attention(q_c, q[..., nope:], pool, spec, table, lens, scale)
    o = torch.bmm(o.transpose(0, 1), wv.transpose(1, 2)).transpose(0, 1)

and prompts over expanded keys and values, the cached ones included:

    c, rope = latent_read(pool, spec, table, lens, cu_k, positions)
    kv = (c @ w).view(positions, heads, 2 * nope)
    o = latent_prompt_attention(q, kv[..., :nope], rope, kv[..., nope:], cu_q, cu_k)
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass, field

import torch

from . import _lib as L
from . import cache as K
from ._lib import check
from .cache import hr_cache_seqs

# every exported symbol declared in include/hadarot_latent.h
EXPORTS = ("hr_latent_page_layout", "hr_latent_append", "hr_latent_read", "hr_latent_attention", "hr_latent_attention_work",
           "hr_latent_prompt_attention", "hr_latent_update", "hr_latent_compact")


class hr_latent_spec(ctypes.Structure):
    _fields_ = [("latent_dim", ctypes.c_int32), ("rope_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("q", L.hr_qspec)]


class hr_latent_page(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("page_bytes", "codes", "scales", "zeros", "rope")]


_ready = None


def _latent_lib() -> ctypes.CDLL:
    """The library with the latent cache's entry points declared."""
    global _ready
    if _ready is None:
        l = K._cache_lib()
        vp, i64, i32, ci, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_float
        sp, sq, out = ctypes.POINTER(hr_latent_spec), ctypes.POINTER(hr_cache_seqs), ctypes.POINTER(i64)
        l.hr_latent_page_layout.argtypes = [sp, ctypes.POINTER(hr_latent_page)]
        l.hr_latent_append.argtypes = [vp, i64, sp, sq, vp, i64, vp, i64, ci, i64, ci, vp]
        l.hr_latent_read.argtypes = [vp, i64, sp, sq, vp, i64, vp, i64, ci, i64, ci, vp]
        l.hr_latent_attention.argtypes = [vp, i64, i64, vp, i64, i64, ci, i64, i32, vp, i64, sp, sq, f32, ci, ci, vp, i64, i64,
                                          vp, i64, vp, i64, vp]
        l.hr_latent_attention_work.argtypes = [ci, i64, i32, sp, i64, i64, out]
        l.hr_latent_prompt_attention.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, i64, vp, i64, ci, i64, i64, i32, i32, vp, vp,
                                                 i64, f32, ci, vp, i64, i64, vp, vp]
        l.hr_latent_update.argtypes = [vp, i64, i64, sp, vp, vp, i64, i64, vp, vp, i64, vp, vp, vp, vp, vp, i64, vp]
        l.hr_latent_compact.argtypes = [vp, i64, i64, sp, vp, vp, i64, i64, vp, i64, vp, vp, vp, vp, i64, vp]
        for n in EXPORTS:
            getattr(l, n).restype = ci
        _ready = l
    return _ready


@dataclass(frozen=True)
class LatentSpec:
    """What a cache of latents holds: the latent's dimension (256 or 512), that of
    the rotary keys (64), positions of a page (16 to 256, a power of two) and the
    quantizer of the latents (INT, group_size from 128 to latent_dim)."""
    latent_dim: int = 512
    rope_dim: int = 64
    page_size: int = 64
    qspec: "QSpec" = field(default_factory=K._default_qspec)  # noqa: F821

    def c(self) -> hr_latent_spec:
        return hr_latent_spec(self.latent_dim, self.rope_dim, self.page_size, self.qspec.c())

    def layout(self) -> dict:
        """Byte size and offsets of the page record (hr_latent_page)."""
        return dict(K._resolved(self).layout)

    @property
    def page_bytes(self) -> int:
        return K._resolved(self).page_bytes

    def _make(self) -> "_Resolved":
        return _Resolved(self)


class _Resolved:
    """What the calls need of a spec: the C struct, the page's layout, and the
    scratch sizes asked for so far (by the sizes and device)."""
    update, compact = "hr_latent_update", "hr_latent_compact"   # the calls that move such pages

    def __init__(self, spec: LatentSpec):
        self.spec = spec.c()
        self.ref = ctypes.byref(self.spec)
        l, p = _latent_lib(), hr_latent_page()
        check(l.hr_latent_page_layout(self.ref, ctypes.byref(p)))
        self.layout = {n: getattr(p, n) for n, _ in hr_latent_page._fields_}
        self.page_bytes = p.page_bytes
        self.work = {}


def _flat(x: torch.Tensor, name: str, tokens, d: int, device) -> int:
    """Checks a [tokens, d] tensor (None: any number) whose rows are contiguous; its stride."""
    if x.dim() != 2 or x.shape[1] != d or (tokens is not None and x.shape[0] != tokens):
        raise ValueError("%s must be [%s, %d], got %s" % (name, "tokens" if tokens is None else tokens, d, list(x.shape)))
    if x.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    if x.stride(1) != 1 and x.numel():
        raise ValueError("%s: the last dimension must be contiguous" % name)
    return x.stride(0)


def _lse(lse, tokens: int, heads: int, device):
    """The log-sum-exp's tensor (or None) of an argument that may be True."""
    if lse is None or lse is False:
        return None
    if lse is True:
        return torch.empty((tokens, heads), dtype=torch.float32, device=device)
    if lse.dtype is not torch.float32 or lse.shape != (tokens, heads) or not lse.is_contiguous() or lse.device != device:
        raise ValueError("lse must be a contiguous float32 tensor [tokens, heads]")
    return lse


def latent_append(pool: torch.Tensor, spec: LatentSpec, c: torch.Tensor, rope: torch.Tensor, table: torch.Tensor,
                  lens: torch.Tensor, cu_q: torch.Tensor | None = None, rotate: bool = True) -> None:
    """Rotates (if ``rotate``) and quantizes the new tokens' latents c [tokens,
    latent_dim], and rounds their rotary keys [tokens, rope_dim] to bfloat16, into
    their pages of ``pool`` [n_pages, page_bytes]; ``lens`` and ``cu_q`` as in
    cache_append."""
    r, dev = K._resolved(spec), pool.device
    _, n = K._pages(pool, r, False)
    seqs = K._seqs(table, lens, cu_q, dev)
    ct = _flat(c, "c", None, spec.latent_dim, dev)
    tokens = c.shape[0]
    rt = _flat(rope, "rope", tokens, spec.rope_dim, dev)
    if c.dtype != rope.dtype:
        raise ValueError("c and rope must have the same dtype")
    K._call(dev, _latent_lib().hr_latent_append, pool.data_ptr(), n, r.ref, ctypes.byref(seqs), c.data_ptr(), ct, rope.data_ptr(),
            rt, K._dt(c), tokens, 1 if rotate else 0, K._stream(dev))


def latent_read(pool: torch.Tensor, spec: LatentSpec, table: torch.Tensor, lens: torch.Tensor, cu_k: torch.Tensor | None,
                positions: int, dtype: torch.dtype = torch.bfloat16, rotate: bool = True, out=None):
    """The latents [positions, latent_dim], rotated back (if ``rotate``), and the
    rotary keys [positions, rope_dim] of the sequences' positions from the first:
    rows cu_k[b] ... cu_k[b + 1] - 1 are sequence b's (cu_k None: as many for each).
    ``out``: (c, rope), if the caller has them."""
    r, dev = K._resolved(spec), pool.device
    _, n = K._pages(pool, r, False)
    seqs = K._seqs(table, lens, cu_k, dev)
    if out is None:
        out = (torch.empty((positions, spec.latent_dim), dtype=dtype, device=dev),
               torch.empty((positions, spec.rope_dim), dtype=dtype, device=dev))
    c, rope = out
    if c.dtype != rope.dtype:
        raise ValueError("c and rope must have the same dtype")
    ct = _flat(c, "c", positions, spec.latent_dim, dev)
    rt = _flat(rope, "rope", positions, spec.rope_dim, dev)
    K._call(dev, _latent_lib().hr_latent_read, pool.data_ptr(), n, r.ref, ctypes.byref(seqs), c.data_ptr(), ct, rope.data_ptr(), rt,
            K._dt(c), positions, 1 if rotate else 0, K._stream(dev))
    return out


def latent_attention(q: torch.Tensor, q_rope: torch.Tensor, pool: torch.Tensor, spec: LatentSpec, table: torch.Tensor,
                     lens: torch.Tensor, scale: float, cu_q: torch.Tensor | None = None, max_q: int = 0, causal: bool = True,
                     rotate: bool = True, out: torch.Tensor | None = None, lse=None, work: torch.Tensor | None = None):
    """Attention of q [tokens, heads, latent_dim] and q_rope [tokens, heads,
    rope_dim] over the cached latents, which are keys and values of all heads;
    returns out (like q), or (out, lse) with ``lse`` True or a float32 [tokens,
    heads] tensor.  ``scale``: of the scores; ``rotate`` False: q and out are in the
    rotated latents' space; ``max_q``: an upper bound of a row's new tokens, if known
    (it only chooses the kernel); ``work``: scratch of hr_latent_attention_work
    bytes (allocated if not given)."""
    r, dev, l = K._resolved(spec), pool.device, _latent_lib()
    _, n = K._pages(pool, r, False)
    seqs = K._seqs(table, lens, cu_q, dev)
    qt, qh = K._vectors(q, "q", None, None, spec.latent_dim, dev)
    tokens, heads = q.shape[0], q.shape[1]
    rt, rh = K._vectors(q_rope, "q_rope", tokens, heads, spec.rope_dim, dev)
    dt = K._dt(q)
    if q_rope.dtype != q.dtype:
        raise ValueError("q and q_rope must have the same dtype")
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    elif out.dtype != q.dtype:
        raise ValueError("out must have q's dtype")
    ot, oh = K._vectors(out, "out", tokens, heads, spec.latent_dim, dev)
    lse = _lse(lse, tokens, heads, dev)
    wp = wb = 0
    if work is not None:
        wp, wb = K._bytes(work, dev)
    else:
        key = (dt, tokens, heads, seqs.rows, max_q, dev.index)
        need = r.work.get(key)
        if need is None:
            bytes_ = ctypes.c_int64()
            K._call(dev, l.hr_latent_attention_work, dt, tokens, heads, r.ref, seqs.rows, max_q, ctypes.byref(bytes_))
            need = bytes_.value
            if len(r.work) > 4096:
                r.work.clear()
            r.work[key] = need
        if need:
            work = torch.empty(need, dtype=torch.uint8, device=dev)
            wp, wb = work.data_ptr(), need
    K._call(dev, l.hr_latent_attention, q.data_ptr(), qt, qh, q_rope.data_ptr(), rt, rh, dt, tokens, heads, pool.data_ptr(), n, r.ref,
            ctypes.byref(seqs), scale, 1 if causal else 0, 1 if rotate else 0, out.data_ptr(), ot, oh, K._ptr(lse), max_q, wp, wb,
            K._stream(dev))
    return out if lse is None else (out, lse)


def latent_prompt_attention(q: torch.Tensor, k: torch.Tensor, rope: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                            cu_k: torch.Tensor, scale: float | None = None, causal: bool = True, out: torch.Tensor | None = None,
                            lse=None):
    """Attention of prompts q [tokens, heads, nope + rope_dim] over keys k
    [positions, heads, nope], rotary keys [positions, rope_dim] and values v
    [positions, heads, nope] made from latents; returns out [tokens, heads, nope],
    or (out, lse).  ``cu_q`` and ``cu_k`` (int32 [rows + 1]) bound the sequences'
    tokens and positions; ``scale``: None or 0 means 1 / sqrt(nope + rope_dim)."""
    dev, l = q.device, _latent_lib()
    if k.dim() != 3 or rope.dim() != 2 or cu_q.dim() != 1:
        raise ValueError("k must be [positions, heads, nope], rope [positions, rope_dim] and cu_q [rows + 1]")
    positions, heads, nope = k.shape
    kt, kh = K._vectors(k, "k", None, None, nope, dev)
    vt, vh = K._vectors(v, "v", positions, heads, nope, dev)
    rt = _flat(rope, "rope", positions, 64, dev)
    qt, qh = K._vectors(q, "q", None, heads, nope + 64, dev)
    tokens, rows = q.shape[0], cu_q.shape[0] - 1
    if not q.dtype == k.dtype == v.dtype == rope.dtype:
        raise ValueError("q, k, rope and v must have the same dtype")
    if out is None:
        out = torch.empty((tokens, heads, nope), dtype=q.dtype, device=dev)
    elif out.dtype != q.dtype:
        raise ValueError("out must have q's dtype")
    ot, oh = K._vectors(out, "out", tokens, heads, nope, dev)
    lse = _lse(lse, tokens, heads, dev)
    if scale is not None and scale != 0 and ctypes.c_float(scale).value == 0:
        raise ValueError("scale = %r is 0 in float32" % scale)   # (which would mean the default)
    K._call(dev, l.hr_latent_prompt_attention, q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, rope.data_ptr(), rt,
            K._dt(q), tokens, positions, heads, nope, K._ints(cu_q, "cu_q", (rows + 1,), dev), K._ints(cu_k, "cu_k", (rows + 1,), dev),
            rows, 0.0 if scale is None else scale, 1 if causal else 0, out.data_ptr(), ot, oh, K._ptr(lse), K._stream(dev))
    return out if lse is None else (out, lse)
