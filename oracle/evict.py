"""Definitions of the eviction from the paged 4-bit cache in float64 (TEST
INFRASTRUCTURE ONLY).

Plain numpy over explicit loops, written from the descriptions in
``include/hadarot_evict.h`` and sharing no code with the library: attention
weights added up by position, and the choice and moves of an eviction.
"""
from __future__ import annotations

import numpy as np

from .cache import CacheDef, section, vectors
from .hadamard import sylvester


def weights(q, pool, c: CacheDef, table, lens, cu, lse, old, scale=None, causal=True, window=0, rotate=True, decay=1.0):
    """(new weights [rows, heads, width], what a bound on their error needs):
    need[0] = sum of p, need[1] = sum of p scale |q'| . |k|, need[2] = sum of p
    scale ||q|| ||k||, need[3] = sum of p (|lse| + 1), by position."""
    q = np.asarray(q, dtype=np.float64)
    d, rep = c.d, q.shape[1] // c.heads
    scale = 1.0 / np.sqrt(d) if not scale else scale
    if rotate:
        q = q @ (sylvester(d) / np.sqrt(d))
    out, need = np.array(old, dtype=np.float64), np.zeros((4,) + old.shape)
    for b in range(len(lens)):
        n, t0, t1 = min(max(lens[b], 0), table.shape[1] * c.page), cu[b], cu[b + 1]
        if t1 == t0:
            continue
        first = n - (t1 - t0)
        out[b, :, :max(first, 0)] *= decay
        out[b, :, max(first, 0):n] = 0.0
        for h in range(c.heads):
            keys, seen = np.zeros((n, d)), np.zeros(n, dtype=bool)
            for j in range(-(-n // c.page)):
                p = table[b, j]
                if 0 <= p < len(pool):
                    k = min(c.page, n - j * c.page)
                    keys[j * c.page: j * c.page + k] = vectors(pool[p], c, h, "k")[0][:k]
                    seen[j * c.page: j * c.page + k] = True
            for t in range(t0, t1):
                pos, j = first + t - t0, np.arange(n)
                sees = seen & ((j <= pos) if causal else True)
                if window:
                    sees &= j > pos - window
                for i in range(h * rep, (h + 1) * rep):
                    if not sees.any() or lse[t, i] == -np.inf:
                        continue
                    k = keys[sees]
                    p = np.exp(scale * (k @ q[t, i]) - float(lse[t, i]))
                    out[b, h, :n][sees] += p
                    at = np.flatnonzero(sees)
                    need[0, b, h, at] += p
                    need[1, b, h, at] += p * scale * (np.abs(k) @ np.abs(q[t, i]))
                    need[2, b, h, at] += p * scale * np.linalg.norm(q[t, i]) * np.linalg.norm(k, axis=1)
                    need[3, b, h, at] += p * (abs(float(lse[t, i])) + 1)
    return out, need


def order(w):
    """Sort keys of weights: larger is heavier, NaN heaviest, -0 as 0."""
    return np.where(np.isnan(w), np.inf, w), np.isnan(w)


def keeps(w, n, budget, sinks, recent):
    """The positions of w[:n] that stay, in order."""
    middle = list(range(sinks, n - recent))
    v, nan = order(np.asarray(w, dtype=np.float64))
    middle.sort(key=lambda j: (not nan[j], -v[j], j))
    return sorted(list(range(sinks)) + middle[: budget - sinks - recent] + list(range(n - recent, n)))


def evict(pool, c: CacheDef, table, lens, w, budget, sinks=0, recent=0):
    """(table, lens, refs, status); pool [layers, n_pages, bytes] and w [layers,
    rows, heads, width] are changed in place."""
    layers, n_pages = pool.shape[:2]
    rows, mp = table.shape
    lens = [min(max(int(n), 0), mp * c.page) for n in lens]
    held = [[int(p) if 0 <= p < n_pages else -1 for p in table[i, : -(-lens[i] // c.page)]] for i in range(rows)]
    count = np.zeros(n_pages, dtype=np.int64)
    for r in held:
        for p in r:
            if p >= 0:
                count[p] += 1
    free = [p for p in range(n_pages) if count[p] == 0]
    stay, wanted, done = -(-budget // c.page), 0, 0
    new = [list(r) for r in held]
    after = list(lens)
    for i in range(rows):
        if lens[i] <= budget or -1 in held[i]:
            continue
        slots = [j for j in range(stay) if count[held[i][j]] > 1]
        at, wanted = wanted, wanted + len(slots)
        if slots and wanted > len(free):
            continue
        done += 1
        after[i] = budget
        new[i] = held[i][:stay]
        for k, j in enumerate(slots):
            new[i][j] = free[at + k]
    # the moves read the pool as it was
    old = pool.copy()
    for i in range(rows):
        if after[i] == lens[i]:
            continue
        for l in range(layers):
            for h in range(c.heads):
                src = keeps(w[l, i, h], lens[i], budget, sinks, recent)
                w[l, i, h, :budget] = w[l, i, h, src]
                for d, s in enumerate(src):
                    move(old[l, held[i][s // c.page]], pool[l, new[i][d // c.page]], c, h, s % c.page, d % c.page)
    out = np.full((rows, mp), -1, dtype=np.int32)
    refs = np.zeros(n_pages, dtype=np.int32)
    for i, r in enumerate(new):
        for j, p in enumerate(r):
            out[i, j] = p
            if p >= 0:
                refs[p] += 1
    used = int((refs > 0).sum())
    return out, np.array(after, dtype=np.int32), refs, np.array([used, max(wanted - len(free), 0), done, n_pages - used], dtype=np.int32)


def move(a, b, c: CacheDef, h, s, d):
    """Position s of head h of page a to position d of page b."""
    for x in "kv":
        for name, width in (("codes", c.d // 2), ("scales", c.ng * (4 if c.sdt == "f32" else 2))):
            f, t = section(a, c, h, "%s_%s" % (x, name)), section(b, c, h, "%s_%s" % (x, name))
            t[d * width: (d + 1) * width] = f[s * width: (s + 1) * width]
        if not c.sym:
            f, t = section(a, c, h, x + "_zeros"), section(b, c, h, x + "_zeros")
            for g in range(c.ng):
                i, o = s * c.ng + g, d * c.ng + g
                v = (f[i // 2] >> (4 * (i % 2))) & 15
                t[o // 2] = (t[o // 2] & (0xF0 if o % 2 == 0 else 0x0F)) | (v << (4 * (o % 2)))
