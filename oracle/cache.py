"""Definitions of the paged 4-bit key/value cache in float64 (TEST INFRASTRUCTURE ONLY).

Plain numpy over explicit loops: the page record, attention over it, and the
page-table operations, written from their descriptions in
``include/hadarot_cache.h`` and sharing no code with the library.  Parity
status: the record's sections are pinned to ``oracle.quant`` (packing and RTN)
by the tests; softmax attention is the textbook formula.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

from .hadamard import sylvester
from .quant import pack_nibbles, unpack_nibbles


@dataclass(frozen=True)
class CacheDef:
    heads: int
    d: int
    page: int
    group: int
    sym: bool
    sdt: str              # "bf16" or "f32"

    @property
    def ng(self):
        return self.d // self.group

    def offsets(self):
        """(offset, bytes) of each section of a head, and the head's bytes."""
        def up(v, a):
            return -(-v // a) * a
        at, out = 0, {}
        sizes = {"codes": self.page * self.d // 2, "scales": self.page * self.ng * (4 if self.sdt == "f32" else 2),
                 "zeros": 0 if self.sym else self.page * self.ng // 2}
        for name, size in sizes.items():
            for x in "kv":
                if size:
                    out["%s_%s" % (x, name)] = (at, size)
                    at += up(size, 16)
        return out, up(at, 128)

    @property
    def page_bytes(self):
        return self.offsets()[1] * self.heads


def f32_to_bytes(v, sdt):
    """Little-endian bytes of float32 or bfloat16 (v must be representable)."""
    u = np.asarray(v, dtype=np.float32).view(np.uint32)
    return u.astype("<u4").view(np.uint8) if sdt == "f32" else (u >> 16).astype("<u2").view(np.uint8)


def bytes_to_f64(b, sdt):
    b = np.ascontiguousarray(b)
    u = b.view("<u4") if sdt == "f32" else b.view("<u2").astype(np.uint32) << 16
    return u.astype(np.uint32).view(np.float32).astype(np.float64)


def section(page_row, c: CacheDef, head: int, name: str):
    """Bytes of one section in one page ([page_bytes] uint8): a view."""
    off, hb = c.offsets()
    a, n = off[name]
    return page_row[head * hb + a: head * hb + a + n]


def vectors(page_row, c: CacheDef, head: int, x: str):
    """(values, codes - zero, scales), each [page, d], of K or V ("k", "v") of
    one head of one page."""
    q = unpack_nibbles(section(page_row, c, head, x + "_codes"), c.page * c.d, c.sym).reshape(c.page, c.ng, c.group)
    s = bytes_to_f64(section(page_row, c, head, x + "_scales"), c.sdt).reshape(c.page, c.ng, 1)
    z = np.zeros((c.page, c.ng, 1))
    if not c.sym:
        z = unpack_nibbles(section(page_row, c, head, x + "_zeros"), c.page * c.ng).reshape(c.page, c.ng, 1)
    q = q - z
    with np.errstate(invalid="ignore"):
        v = q * s
    full = (c.page, c.d)
    return v.reshape(full), q.reshape(full), np.broadcast_to(s, (c.page, c.ng, c.group)).reshape(full)


def random_pool(c: CacheDef, n_pages: int, seed: int, v_spread: float = 0.5):
    """Pages of random codes, scales and zero points (float32 scales use all
    their bits)."""
    rng = np.random.default_rng(seed)
    pool = rng.integers(0, 256, (n_pages, c.page_bytes), dtype=np.uint8)
    for p in range(n_pages):
        for h in range(c.heads):
            for x in "kv":
                s = 0.2 * np.exp((0.2 if x == "k" else v_spread) * rng.standard_normal(c.page * c.ng))
                s = s.astype(np.float32)
                if c.sdt == "bf16":
                    s = (s.view(np.uint32) & 0xFFFF0000).view(np.float32)
                section(pool[p], c, h, x + "_scales")[:] = f32_to_bytes(s, c.sdt)
    return pool


def poison(pool, c: CacheDef, page: int, slot: int):
    """Makes a position's scales NaN in every head (bytes nobody may look at)."""
    for h in range(c.heads):
        for x in "kv":
            b = section(pool[page], c, h, x + "_scales")
            w = b.reshape(c.page, -1)
            w[slot] = 0xFF


def attention(q, pool, c: CacheDef, table, lens, cu, scale=None, causal=True, window=0, rotate=True):
    """(out, lse, err): the formula in float64, and for each output what a
    bound on its error needs: err[...] = (largest sum |q_i| 15 s_i over the
    keys seen, times the scale; sum p 15 s_v by element)."""
    q = np.asarray(q, dtype=np.float64)
    tokens, hq, d = q.shape
    rep = hq // c.heads
    scale = 1.0 / np.sqrt(d) if not scale else scale
    if rotate:
        q = q @ (sylvester(d) / np.sqrt(d))
    out = np.zeros(q.shape)
    lse = np.full((tokens, hq), -np.inf)
    mag, vabs = np.zeros((tokens, hq)), np.zeros(q.shape)
    for b in range(len(lens)):
        n, length = cu[b + 1] - cu[b], int(lens[b])
        if n == 0 or length == 0:
            continue
        pages = [int(p) for p in table[b][: -(-length // c.page)]]
        there = np.repeat([0 <= p < len(pool) for p in pages], c.page)[:length]
        pos = length - n + np.arange(n)
        j = np.arange(length)
        seen = np.broadcast_to(there, (n, length)).copy()
        if causal:
            seen &= j[None] <= pos[:, None]
            if window:
                seen &= j[None] > pos[:, None] - window
        for h in range(c.heads):
            kv = {}
            for x in "kv":
                parts = [vectors(pool[p], c, h, x) if 0 <= p < len(pool) else (np.zeros((c.page, d)),) * 3 for p in pages]
                kv[x] = [np.concatenate([a[i] for a in parts])[:length] for i in (0, 2)]
            for r in range(h * rep, (h + 1) * rep):
                for i in range(n):
                    w = seen[i]
                    if not w.any():
                        continue
                    t = cu[b] + i
                    s = kv["k"][0][w] @ q[t, r] * scale
                    top = s.max()
                    e = np.exp(s - top)
                    total = e.sum()
                    out[t, r] = (e / total) @ kv["v"][0][w]
                    lse[t, r] = top + np.log(total)
                    mag[t, r] = (15 * kv["k"][1][w] @ np.abs(q[t, r])).max() * scale
                    vabs[t, r] = (e / total) @ (15 * kv["v"][1][w])
    return out, lse, (mag, vabs)


def update(c_page, max_pages, n_pages, table, lens, parents, grow):
    """(table, lens, refs, status, copies) with copies = [(source, target)]."""
    cap = max_pages * c_page
    rows = []
    for p, g in zip(parents, grow):
        has = 0 <= p < len(lens)
        before = min(max(int(lens[p]), 0), cap) if has else 0
        after = min(max(before + int(g), 0), cap)
        kept = min(-(-before // c_page), -(-after // c_page))
        pages = [int(x) if 0 <= x < n_pages else -1 for x in (table[p][:kept] if has else [])]
        rows.append(dict(before=before, after=after, pages=pages))
    holders = [0] * n_pages
    for r in rows:
        for p in r["pages"]:
            if p >= 0:
                holders[p] += 1
    free = [p for p in range(n_pages) if holders[p] == 0]
    grows_in = {}
    for i, r in enumerate(rows):
        last = r["before"] // c_page
        if r["after"] > r["before"] and r["before"] % c_page and r["pages"][last] >= 0:
            grows_in.setdefault(r["pages"][last], []).append(i)
    keeper = {p: min(w) for p, w in grows_in.items() if len(w) == holders[p]}
    copies, lacking = [], 0
    for i, r in enumerate(rows):
        last = r["before"] // c_page
        old = r["pages"][last] if last < len(r["pages"]) else -1
        if old in grows_in and i in grows_in[old] and keeper.get(old) != i:
            if free:
                r["pages"][last] = free.pop(0)
                copies.append((old, r["pages"][last]))
            else:
                r["pages"][last] = -1
                lacking += 1
        while len(r["pages"]) < -(-r["after"] // c_page):
            if free:
                r["pages"].append(free.pop(0))
            else:
                r["pages"].append(-1)
                lacking += 1
    refs = np.zeros(n_pages, dtype=np.int32)
    new = np.full((len(rows), max_pages), -1, dtype=np.int32)
    for i, r in enumerate(rows):
        new[i, : len(r["pages"])] = r["pages"]
        for p in r["pages"]:
            if p >= 0:
                refs[p] += 1
    used = int((refs > 0).sum())
    status = [used, lacking, len(copies), n_pages - used]
    return new, np.array([r["after"] for r in rows], dtype=np.int32), refs, status, copies


def compact(c_page, max_pages, n_pages, table, lens, into_pages=None):
    """(table, refs, status, moves) with moves = [(source, target)]."""
    held = [min(max(int(n), 0), max_pages * c_page) for n in lens]
    held = [-(-n // c_page) for n in held]
    live = sorted({int(p) for row, k in zip(table, held) for p in row[:k] if 0 <= p < n_pages})
    if into_pages is None:
        holes = iter([p for p in range(len(live)) if p not in set(live)])
        to = {p: p if p < len(live) else next(holes) for p in live}
        moves = [(p, t) for p, t in to.items() if p != t]
        places = n_pages
    else:
        to = {p: i for i, p in enumerate(live) if i < into_pages}
        moves = list(to.items())
        places = into_pages
    new = np.full((len(held), max_pages), -1, dtype=np.int32)
    refs = np.zeros(places, dtype=np.int32)
    for i, k in enumerate(held):
        for j in range(k):
            t = to.get(int(table[i][j]), -1)
            new[i, j] = t
            if t >= 0:
                refs[t] += 1
    status = [len(live), len(live) - len(to), len(moves), places - len(to)]
    return new, refs, status, moves


__all__ = ["CacheDef", "attention", "bytes_to_f64", "compact", "f32_to_bytes", "pack_nibbles", "poison", "random_pool",
           "section", "update", "vectors"]
