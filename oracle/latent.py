"""Definitions of latent attention over a paged 4-bit cache in float64 (TEST
INFRASTRUCTURE ONLY).

Plain numpy over explicit loops: the page record, attention over cached latents
and over expanded keys and values, written from the descriptions in
``include/hadarot_latent.h`` and sharing no code with the library.  Parity status:
the record's sections are pinned to ``oracle.quant`` (packing and RTN) by the
tests; softmax attention is the textbook formula.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

from .cache import bytes_to_f64, f32_to_bytes
from .hadamard import sylvester
from .quant import unpack_nibbles


@dataclass(frozen=True)
class LatentDef:
    d: int
    page: int
    group: int
    sym: bool
    sdt: str              # "bf16" or "f32"
    rope: int = 64

    @property
    def ng(self):
        return self.d // self.group

    def offsets(self):
        """(offset, bytes) of each section, and the page's bytes."""
        def up(v, a):
            return -(-v // a) * a
        at, out = 0, {}
        sizes = {"codes": self.page * self.d // 2, "scales": self.page * self.ng * (4 if self.sdt == "f32" else 2),
                 "zeros": 0 if self.sym else self.page * self.ng // 2, "rope": self.page * self.rope * 2}
        for name, size in sizes.items():
            if size:
                out[name] = (at, size)
                at += up(size, 16)
        return out, up(at, 128)

    @property
    def page_bytes(self):
        return self.offsets()[1]


def section(page_row, c: LatentDef, name: str):
    """Bytes of one section of one page ([page_bytes] uint8): a view."""
    a, n = c.offsets()[0][name]
    return page_row[a: a + n]


def latents(page_row, c: LatentDef):
    """(latents [page, d], scales by element [page, d], rotary keys [page, rope])."""
    q = unpack_nibbles(section(page_row, c, "codes"), c.page * c.d, c.sym).reshape(c.page, c.ng, c.group)
    s = bytes_to_f64(section(page_row, c, "scales"), c.sdt).reshape(c.page, c.ng, 1)
    z = np.zeros((c.page, c.ng, 1))
    if not c.sym:
        z = unpack_nibbles(section(page_row, c, "zeros"), c.page * c.ng).reshape(c.page, c.ng, 1)
    with np.errstate(invalid="ignore"):
        v = (q - z) * s
    full = (c.page, c.d)
    return v.reshape(full), np.broadcast_to(s, (c.page, c.ng, c.group)).reshape(full), bytes_to_f64(section(page_row, c, "rope"), "bf16").reshape(c.page, c.rope)


def random_pool(c: LatentDef, n_pages: int, seed: int, spread: float = 0.4):
    """Pages of random codes, scales, zero points and rotary keys."""
    rng = np.random.default_rng(seed)
    pool = rng.integers(0, 256, (n_pages, c.page_bytes), dtype=np.uint8)
    for p in range(n_pages):
        s = (0.2 * np.exp(spread * rng.standard_normal(c.page * c.ng))).astype(np.float32)
        r = rng.standard_normal(c.page * c.rope).astype(np.float32)
        if c.sdt == "bf16":
            s = (s.view(np.uint32) & 0xFFFF0000).view(np.float32)
        section(pool[p], c, "scales")[:] = f32_to_bytes(s, c.sdt)
        section(pool[p], c, "rope")[:] = f32_to_bytes((r.view(np.uint32) & 0xFFFF0000).view(np.float32), "bf16")
    return pool


def poison(pool, c: LatentDef, page: int, slot: int):
    """Makes a position's scales and rotary key NaN (bytes nobody may look at)."""
    for name in ("scales", "rope"):
        section(pool[page], c, name).reshape(c.page, -1)[slot] = 0xFF


def gather(pool, c: LatentDef, row, n):
    """(latents, scales, rotary keys, whether there) of n positions of a sequence."""
    x, s, r, there = np.zeros((n, c.d)), np.zeros((n, c.d)), np.zeros((n, c.rope)), np.zeros(n, dtype=bool)
    for j in range(-(-n // c.page)):
        p = row[j]
        if 0 <= p < len(pool):
            a, b = j * c.page, min(n, (j + 1) * c.page)
            v = latents(pool[p], c)
            x[a:b], s[a:b], r[a:b], there[a:b] = v[0][: b - a], v[1][: b - a], v[2][: b - a], True
    return x, s, r, there


def softmax_rows(w):
    top = w.max()
    e = np.exp(w - top)
    return e / e.sum(), top + np.log(e.sum())


def attention(q, q_rope, pool, c: LatentDef, table, lens, cu, scale, causal=True, rotate=True):
    """(out, lse, need): the formula in float64, and what a bound on the error needs:
    need["score"] = largest scale sum |q'_i c_i| over the keys seen, need["rope"]
    the same of rotary keys, need["norm"] = largest scale ||q|| ||c||, by (token,
    head); need["value"] = norm of sum p |c|, need["unit"] = norm of the largest
    p 15 s, by (token, head)."""
    q, q_rope = np.asarray(q, dtype=np.float64), np.asarray(q_rope, dtype=np.float64)
    tokens, heads, d = q.shape
    had = sylvester(d) / np.sqrt(d)
    if rotate:
        q = q @ had
    out, lse = np.zeros(q.shape), np.full((tokens, heads), -np.inf)
    need = {k: np.zeros((tokens, heads)) for k in ("score", "rope", "norm", "value", "unit", "size")}
    for b in range(len(lens)):
        n = min(max(int(lens[b]), 0), table.shape[1] * c.page)
        x, s, r, there = gather(pool, c, table[b], n)
        for t in range(cu[b], cu[b + 1]):
            pos, j = n - cu[b + 1] + t, np.arange(n)
            sees = there & ((j <= pos) if causal else True)
            if not sees.any():
                continue
            for h in range(heads):
                k, kr = x[sees], r[sees]
                w = scale * (k @ q[t, h] + kr @ q_rope[t, h])
                p, lse[t, h] = softmax_rows(w)
                o = p @ k
                need["score"][t, h] = scale * (np.abs(k) @ np.abs(q[t, h])).max()
                need["rope"][t, h] = scale * (np.abs(kr) @ np.abs(q_rope[t, h])).max()
                need["norm"][t, h] = scale * np.linalg.norm(q[t, h]) * np.linalg.norm(k, axis=1).max()
                need["value"][t, h] = np.linalg.norm(p @ np.abs(k))
                need["unit"][t, h] = np.linalg.norm((p[:, None] * 15 * s[sees]).max(0))
                need["size"][t, h] = np.linalg.norm(o)
                out[t, h] = o @ had if rotate else o
    return out, lse, need


def prompt(q, k, rope, v, cu_q, cu_k, scale=None, causal=True):
    """(out, lse, score, value): the formula in float64, the largest scale sum
    |q_i k_i| of a row's keys, and sum p |v| by element."""
    q, k, rope, v = (np.asarray(t, dtype=np.float64) for t in (q, k, rope, v))
    tokens, heads, wide = q.shape
    n = k.shape[-1]
    scale = scale or 1.0 / np.sqrt(wide)
    out, lse = np.zeros((tokens, heads, n)), np.full((tokens, heads), -np.inf)
    score, value = np.zeros((tokens, heads)), np.zeros((tokens, heads, n))
    for b in range(len(cu_q) - 1):
        for t in range(cu_q[b], cu_q[b + 1]):
            end = cu_k[b + 1] if not causal else cu_k[b + 1] - cu_q[b + 1] + t + 1
            if end <= cu_k[b]:
                continue
            at = slice(cu_k[b], end)
            for h in range(heads):
                key = np.concatenate((k[at, h], rope[at]), 1)
                p, lse[t, h] = softmax_rows(scale * (key @ q[t, h]))
                with np.errstate(invalid="ignore"):
                    out[t, h] = p @ v[at, h]
                score[t, h] = scale * (np.abs(key) @ np.abs(q[t, h])).max()
                value[t, h] = p @ np.abs(v[at, h])
    return out, lse, score, value
