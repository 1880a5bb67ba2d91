"""The paged 4-bit key/value cache, measured: writing it, attention over it, and the moves of its pages.

Each case is one call of one operator of the cache on seeded inputs.  ``run`` makes it through the package where ``own``
is true, and in elementary torch operations in float32 where it is false; ``exact`` gives the definition in float64.

A page is one record of bytes: for each kv head the codes of K and V (two 4-bit codes a byte, element 2j in the low
nibble), their scales, and for asymmetric groups their zero points (two a byte), each section and each head padded as
in ``layout``.  What an operator writes into pages is returned as the pages' own bytes, which have to be equal bit for
bit: that holds every 4-bit code, every scale and every zero point at once.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one user's next token in a short chat: the smallest call, all latency
        _attend("decode_one", batch=1, new=1, ragged=False, length=331, hq=32, hkv=8, d=128),
        # the R3 cache of this repository's benchmark (16 sequences of 2048, 32 heads of 128, INT4 asymmetric per
        # head vector): one decoding step
        _attend("decode_r3", batch=16, new=1, ragged=False, length=2048, hq=32, hkv=32, d=128),
        # a server's decoding step: grouped heads, lengths from a few tokens to 32768
        _attend("decode_ragged", batch=24, new=1, ragged=True, length=32768, hq=32, hkv=8, d=128),
        # drafted tokens of many sequences at once (1 to 8 each), sliding window, symmetric groups of 32
        _attend("draft_window", batch=32, new=8, ragged=True, length=8000, hq=28, hkv=4, d=128, group=32, sym=True,
                sdt="f32", page=16, window=1024),
        # a chunk of a long prompt against what is already cached
        _attend("prefill_chunk", batch=2, new=2048, ragged=False, length=8192, hq=32, hkv=8, d=128),
        # float32 activations, small heads, prompts of odd lengths from the first token
        _attend("prefill_f32", batch=3, new=777, ragged=True, length=777, hq=12, hkv=4, d=64, group=32, dtype="f32"),
        # one new token in each of 64 sequences
        _append("append_step", batch=64, new=1, ragged=False, length=4096, hkv=8, d=128),
        # the prompt of the R3 benchmark: 16 x 2048 tokens of 32 heads
        _append("append_r3", batch=16, new=2048, ragged=False, length=2048, hkv=32, d=128),
        # 16 beams: some parents twice, some dropped, one token each
        _update("update_beams", rows=16, new_rows=16, pages=512, max_pages=24, grow=1, layers=2, hkv=8, d=128, page=64),
        # a server's scheduling step over 256 sequences: forks, ends, prompts that arrive
        _update("update_server", rows=256, new_rows=256, pages=12000, max_pages=128, grow=700, layers=2, hkv=2, d=128,
                page=64),
        # a fragmented pool moved together in place
        _compact("compact_inplace", rows=32, pages=2048, max_pages=64, layers=2, hkv=8, d=128, page=64, into=0),
        # the live pages of a large pool into a smaller one
        _compact("compact_into", rows=64, pages=6000, max_pages=64, layers=2, hkv=8, d=128, page=64, into=3000),
    ]


def _attend(name, batch, new, ragged, length, hq, hkv, d, group=0, sym=False, sdt="bf16", page=64, window=0,
            dtype="bf16"):
    return {"name": name, "op": "attention", "batch": batch, "new": new, "ragged": ragged, "length": length, "hq": hq,
            "hkv": hkv, "d": d, "group": group or d, "sym": sym, "sdt": sdt, "page": page, "window": window,
            "dtype": dtype}


def _append(name, batch, new, ragged, length, hkv, d, group=0, sym=False, sdt="bf16", page=64, dtype="bf16"):
    return {"name": name, "op": "append", "batch": batch, "new": new, "ragged": ragged, "length": length, "hkv": hkv,
            "d": d, "group": group or d, "sym": sym, "sdt": sdt, "page": page, "dtype": dtype}


def _update(name, rows, new_rows, pages, max_pages, grow, layers, hkv, d, page, group=0, sym=False, sdt="bf16"):
    return {"name": name, "op": "update", "rows": rows, "new_rows": new_rows, "pages": pages, "max_pages": max_pages,
            "grow": grow, "layers": layers, "hkv": hkv, "d": d, "page": page, "group": group or d, "sym": sym,
            "sdt": sdt}


def _compact(name, rows, pages, max_pages, layers, hkv, d, page, into, group=0, sym=False, sdt="bf16"):
    return {"name": name, "op": "compact", "rows": rows, "pages": pages, "max_pages": max_pages, "layers": layers,
            "hkv": hkv, "d": d, "page": page, "into": into, "group": group or d, "sym": sym, "sdt": sdt}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    d = rng.choice([64, 128, 128, 256])
    group = rng.choice([d, d, d, 64, 32])
    fmt = {"d": d, "group": min(group, d), "sym": rng.random() < 0.3, "sdt": rng.choice(["bf16", "bf16", "f32"]),
           "page": rng.choice([16, 32, 64, 128])}
    op = rng.choice(["decode", "decode", "chunk", "append", "update", "compact"])
    if op in ("decode", "chunk"):
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 7, 8])
        if op == "decode":  # at most 2^18 tokens x heads of cache for each of up to 8 new tokens
            length = _log(rng, 1, 32768)
            batch = _log(rng, 1, max(1, min(64, (1 << 20) // (length * hkv))))
            new = rng.choice([1, 1, 1, 2, 5, 8])
        else:               # rows x keys as in the largest listed chunk at most
            length = _log(rng, 64, 8192)
            new = _log(rng, 16, min(length, 2048))
            batch = _log(rng, 1, max(1, min(8, (1 << 30) // (length * new * hq * (d // 64)))))
        return {"op": "attention", "batch": batch, "new": new, "ragged": rng.random() < 0.5, "length": length, "hq": hq,
                "hkv": hkv, "window": rng.choice([0, 0, 0, _log(rng, 1, length)]),
                "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"]), **fmt}
    if op == "append":
        hkv = _log(rng, 1, 32)
        new = _log(rng, 1, 2048)
        batch = _log(rng, 1, max(1, min(64, (1 << 22) // (new * hkv * d // 16))))
        return {"op": "append", "batch": batch, "new": new, "ragged": rng.random() < 0.5, "length": new + _log(rng, 1, 500),
                "hkv": hkv, "dtype": rng.choice(["bf16", "bf16", "f32"]), **fmt}
    hkv = rng.choice([1, 2, 3, 8])
    rows, max_pages = _log(rng, 1, 256), _log(rng, 2, 128)
    layers = rng.choice([1, 2, 3])
    most = 800_000_000 // (layers * hkv * fmt["page"] * (fmt["d"] + 32))
    pages = _log(rng, 64, max(64, min(12000, most)))
    if op == "update":
        return {"op": "update", "rows": rows, "new_rows": _log(rng, 1, 256), "pages": pages, "max_pages": max_pages,
                "grow": _log(rng, 1, fmt["page"] * 10), "layers": layers, "hkv": hkv, **fmt}
    return {"op": "compact", "rows": rows, "pages": pages, "max_pages": max_pages, "layers": layers, "hkv": hkv,
            "into": rng.choice([0, 0, pages // 2 + 1]), **fmt}


# ---------------------------------------------------------------------------------------------------------------------
# the page record

def layout(c):
    """(offsets of a head's sections, bytes of a head, bytes of a page)."""
    up = lambda v, a: (v + a - 1) // a * a  # noqa: E731
    p, d, ng = c["page"], c["d"], c["d"] // c["group"]
    scales = up(p * ng * (4 if c["sdt"] == "f32" else 2), 16)
    zeros = 0 if c["sym"] else up(p * ng // 2, 16)
    at = {"kc": 0, "vc": p * d // 2, "ks": p * d}
    at["vs"] = at["ks"] + scales
    at["kz"] = at["vs"] + scales
    at["vz"] = at["kz"] + zeros
    head = up(at["vz"] + zeros, 128)
    return at, head, head * c["hkv"]


def _section(pool, c, name, width):
    """[..., heads, width] view of one section of every page."""
    at, head, _ = layout(c)
    return pool.unflatten(-1, (c["hkv"], head))[..., at[name]: at[name] + width]


def _sections(pool, c):
    """{name: view} of the sections that hold something."""
    p, d, ng = c["page"], c["d"], c["d"] // c["group"]
    es = 4 if c["sdt"] == "f32" else 2
    out = {k: _section(pool, c, k, p * d // 2).unflatten(-1, (p, d // 2)) for k in ("kc", "vc")}
    out.update({k: _section(pool, c, k, p * ng * es).unflatten(-1, (p, ng * es)) for k in ("ks", "vs")})
    if not c["sym"]:
        out.update({k: _section(pool, c, k, p * ng // 2) for k in ("kz", "vz")})
    return out


def _spec(c):
    import hadamard_rotation_preprocessing_amd as hr
    return hr.CacheSpec(c["hkv"], c["d"], c["page"], hr.QSpec("int", 4, c["group"], c["sym"], c["sdt"]))


# ---------------------------------------------------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _lengths(c, g=None):
    """(new tokens, total length) of each sequence: ragged ones are spread over the logarithm of the range, the same
    pairs for every seed, in an order that follows it."""
    b = c["batch"]
    if not c["ragged"]:
        return torch.full((b,), c["new"], dtype=torch.int32), torch.full((b,), max(c["length"], c["new"]), dtype=torch.int32)
    u = torch.from_numpy(np.random.default_rng(b).random((2, b)))
    new = torch.clamp((c["new"] + 1.0) ** u[0], 1, c["new"]).to(torch.int32)
    new[0] = c["new"]
    total = torch.clamp((c["length"] + 1.0) ** (0.3 + 0.7 * u[1]), 1, c["length"]).to(torch.int32)
    total[0] = c["length"]
    order = torch.arange(b) if g is None else torch.randperm(b, generator=g, device=DEV).cpu()
    return new[order], torch.maximum(total, new)[order]


def _tables(c, total, g, spare):
    """A pool's page table with pages in no order, entries past each length -1."""
    page, b = c["page"], total.numel()
    need = (total.to(torch.int64) + page - 1) // page
    n_pages = int(need.sum()) + spare
    ids = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    width = int(need.max())
    first = torch.cumsum(need, 0) - need
    at = first[:, None] + torch.arange(width)[None]
    held = torch.arange(width)[None] < need[:, None]
    table = torch.where(held.to(DEV), ids[at.clamp(max=n_pages - 1).to(DEV)], torch.tensor(-1, dtype=torch.int32, device=DEV))
    return table.contiguous(), n_pages


def _filled_pool(c, n_pages, g):
    """Pages of Gaussian keys and of values whose size differs from token to token, quantized as the cache holds them."""
    _, head, page_bytes = layout(c)
    pool = torch.zeros((n_pages, page_bytes), dtype=torch.uint8, device=DEV)
    some = max(1, (1 << 26) // (c["hkv"] * c["page"] * c["d"]))
    for a in range(0, n_pages, some):
        part = pool[a: a + some]
        shape = (part.shape[0], c["hkv"], c["page"], c["d"])
        s = _sections(part, c)
        for k in "kv":
            x = torch.randn(shape, generator=g, device=DEV)
            if k == "v":
                x *= torch.exp(0.5 * torch.randn(shape[:3] + (1,), generator=g, device=DEV))
            codes, scales, zeros = _quantize(x, c)
            s[k + "c"].copy_(codes)
            s[k + "s"].copy_(scales)
            if zeros is not None:
                z = zeros.flatten(-2)
                s[k + "z"].copy_(z[..., 0::2] | (z[..., 1::2] << 4))
    return pool


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"c": c}
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}.get(c.get("dtype", "bf16"))
    if c["op"] in ("attention", "append"):
        new, total = _lengths(c, g)
        st["table"], n_pages = _tables(c, total, g, spare=3)
        st["lens"] = total.to(DEV)
        cu = torch.cat([torch.zeros(1, dtype=torch.int32), torch.cumsum(new, 0).to(torch.int32)])
        st["cu"], st["tokens"], st["most"] = cu.to(DEV), int(cu[-1]), int(new.max())
        if c["op"] == "attention":
            st["pool"] = _filled_pool(c, n_pages, g)
            st["q"] = (1.5 * torch.randn((st["tokens"], c["hq"], c["d"]), generator=g, device=DEV)).to(dt)
        else:
            st["pool"] = torch.zeros((n_pages, layout(c)[2]), dtype=torch.uint8, device=DEV)
            st["k"] = torch.randn((st["tokens"], c["hkv"], c["d"]), generator=g, device=DEV).to(dt)
            v = torch.randn((st["tokens"], c["hkv"], c["d"]), generator=g, device=DEV)
            st["v"] = (v * torch.exp(0.5 * torch.randn(v.shape[:2] + (1,), generator=g, device=DEV))).to(dt)
        return st
    # rows that hold about half of the pool, some of them sharing their first pages
    rows, mp, n_pages, page = c["rows"], c["max_pages"], c["pages"], c["page"]
    u = torch.rand((4, max(rows, c.get("new_rows", 1))), generator=g, device=DEV, dtype=torch.float64).cpu()
    room = max(1, min(mp, n_pages // (2 * rows)))
    lens = torch.clamp((room * page) * (0.05 + 0.95 * u[0, :rows]), 1, room * page).to(torch.int64)
    if rows * 2 > n_pages:  # more rows than half of the pages: the last ones are empty
        lens[n_pages // 2:] = 0
    need = (lens + page - 1) // page
    ids = torch.randperm(n_pages, generator=g, device=DEV).cpu()
    at = (torch.cumsum(need, 0) - need)[:, None] + torch.arange(mp)[None]
    table = torch.where(torch.arange(mp)[None] < need[:, None], ids[at.clamp(max=n_pages - 1)], torch.tensor(-1))
    shared = (lens // page).clone()  # full pages of the row before that every fourth row starts with
    for i in range(1, rows, 4):
        k = int(min(shared[i - 1], shared[i], 8))
        table[i, :k] = table[i - 1, :k]
    st["table"] = table.to(torch.int32).to(DEV).contiguous()
    st["lens"] = lens.to(torch.int32).to(DEV)
    shape = (c["layers"], n_pages, layout(c)[2])
    st["pool"] = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
    if c["op"] == "update":
        n = c["new_rows"]
        parents = torch.floor(u[1, :n] * rows * 1.2).to(torch.int32)  # some drawn twice, some not at all
        parents[parents >= rows] = -1                                 # and one in six a new, empty row
        grow = torch.clamp(torch.floor(c["grow"] * u[2, :n] ** 2) + 1, 1, c["grow"]).to(torch.int32)
        grow[u[3, :n] < 0.1] *= -1                                    # one in ten cut back
        grow[u[3, :n] > 0.9] = 0
        st["parents"], st["grow"] = parents.to(DEV), grow.to(DEV)
    elif c["into"]:
        st["into"] = torch.zeros((c["layers"], c["into"], layout(c)[2]), dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------------------------------------------------------------
# one pass

def run(st):
    return (_run_own if own else _run_plain)[st["c"]["op"]](st)


def _own_attention(st):
    import hadamard_rotation_preprocessing_amd as hr
    c = st["c"]
    return hr.cache_attention(st["q"], st["pool"], _spec(c), st["table"], st["lens"], cu_q=st["cu"], max_q=st["most"],
                              window=c["window"], rotate=True)


def _own_append(st):
    import hadamard_rotation_preprocessing_amd as hr
    hr.cache_append(st["pool"], _spec(st["c"]), st["k"], st["v"], st["table"], st["lens"], cu_q=st["cu"], rotate=True)
    return st["pool"]


def _own_update(st):
    import hadamard_rotation_preprocessing_amd as hr
    o = hr.cache_update(st["pool"], _spec(st["c"]), st["table"], st["lens"], st["parents"], st["grow"])
    return {"pool": st["pool"], "table": o["table"], "lens": o["lens"], "refs": o["refs"], "status": o["status"]}


def _own_compact(st):
    import hadamard_rotation_preprocessing_amd as hr
    o = hr.cache_compact(st["pool"], _spec(st["c"]), st["table"], st["lens"], into=st.get("into"))
    return {"pool": st.get("into", st["pool"]), "table": o["table"], "refs": o["refs"], "status": o["status"]}


_run_own = {"attention": _own_attention, "append": _own_append, "update": _own_update, "compact": _own_compact}


def _hadamard(x):
    """x . H / sqrt(d) over the last dimension: the sums and differences of elements 1, 2, 4, ... apart."""
    d = x.shape[-1]
    h = 1
    while h < d:
        x = x.unflatten(-1, (d // (2 * h), 2, h))
        a, b = x[..., 0, :], x[..., 1, :]
        x = torch.stack((a + b, a - b), dim=-2).flatten(-3)
        h *= 2
    return x * (1.0 / math.sqrt(d))


def _quantize(x, c):
    """Codes (packed), scales (as bytes) and zero points of float32 x [..., d]; the stored scale gives the codes."""
    g = c["group"]
    y = x.unflatten(-1, (c["d"] // g, g))
    steps = torch.tensor(7.0 if c["sym"] else 15.0, device=DEV).expand(y.shape[:-1])  # a tensor: a true division
    if c["sym"]:
        s = y.abs().amax(-1) / steps
    else:
        lo, hi = y.amin(-1).clamp(max=0.0), y.amax(-1).clamp(min=0.0)
        s = (hi - lo) / steps
    s = torch.where(s == 0, torch.ones_like(s), s)
    stored = s if c["sdt"] == "f32" else s.to(torch.bfloat16)
    s = stored.float()[..., None]
    q = torch.round(y / s)
    zeros = None
    if c["sym"]:
        q = q.clamp(-8, 7).to(torch.int32) & 15
    else:
        z = torch.round(-lo[..., None] / s).clamp(0, 15)
        q = (q + z).clamp(0, 15).to(torch.int32)
        zeros = z[..., 0].to(torch.uint8)
    q = q.to(torch.uint8).flatten(-2)
    return q[..., 0::2] | (q[..., 1::2] << 4), stored.contiguous().view(torch.uint8), zeros


def _dequantize(s, k, c):
    """float32 [..., page, d] of the codes, scales and zero points in the sections `s` of K (k = "k") or V."""
    codes = s[k + "c"]
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).to(torch.float32)
    scales = s[k + "s"].contiguous().view(torch.float32 if c["sdt"] == "f32" else torch.bfloat16).to(torch.float32)
    q = q.unflatten(-1, (c["d"] // c["group"], c["group"]))
    if c["sym"]:
        q = torch.where(q >= 8, q - 16, q)
    else:
        z = s[k + "z"]
        z = torch.stack((z & 15, z >> 4), dim=-1).flatten(-2).to(torch.float32)
        q = q - z.unflatten(-1, (c["page"], -1))[..., None]
    return (q * scales[..., None]).flatten(-2)


def _plain_attention(st):
    c = st["c"]
    b, hkv, d, most = c["batch"], c["hkv"], c["d"], st["most"]
    rep = c["hq"] // hkv
    pages = st["pool"][st["table"].clamp(min=0).long()]                     # [b, pages of a row, bytes]
    s = _sections(pages, c)
    k, v = (_dequantize(s, x, c).transpose(1, 2).flatten(2, 3) for x in "kv")  # [b, hkv, keys, d]
    cu, lens = st["cu"].long(), st["lens"].long()
    n = cu[1:] - cu[:-1]
    i = torch.arange(most, device=DEV)
    at = (cu[:-1, None] + i).clamp(max=st["tokens"] - 1)
    q = _hadamard(st["q"].float())[at]                                      # [b, most, hq, d]
    q = q.unflatten(2, (hkv, rep)).permute(0, 2, 3, 1, 4).reshape(b, hkv, rep * most, d)
    w = torch.matmul(q, k.transpose(-1, -2)).unflatten(2, (rep, most)) * (1.0 / math.sqrt(d))
    pos = (lens - n)[:, None] + i                                           # each query's place in its sequence
    j = torch.arange(k.shape[2], device=DEV)
    seen = (j <= pos[..., None]) & (j < lens[:, None, None])
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    w = torch.where(seen[:, None, None], w, torch.tensor(-math.inf, device=DEV))
    top = w.amax(-1, keepdim=True)
    e = torch.exp(w - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.flatten(2, 3), v) / torch.where(total == 0, torch.ones_like(total), total).flatten(2, 3)
    o = o.unflatten(2, (rep, most)).permute(0, 3, 1, 2, 4).reshape(b, most, c["hq"], d)
    token = torch.arange(st["tokens"], device=DEV)
    row = torch.searchsorted(cu[1:], token, right=True)
    return o[row, token - cu[row]].to(st["q"].dtype)


def _plain_append(st):
    c, pool = st["c"], st["pool"]
    cu, lens = st["cu"].long(), st["lens"].long()
    token = torch.arange(st["tokens"], device=DEV)
    row = torch.searchsorted(cu[1:], token, right=True)
    pos = (lens - (cu[1:] - cu[:-1]))[row] + token - cu[row]
    page, off = st["table"][row, pos // c["page"]].long(), pos % c["page"]
    s = _sections(pool, c)
    for k in "kv":
        x = st[k].float()
        codes, scales, zeros = _quantize(_hadamard(x) if k == "k" else x, c)
        s[k + "c"][page, :, off] = codes
        s[k + "s"][page, :, off] = scales
        if zeros is not None:
            z = s[k + "z"]
            z = torch.stack((z & 15, z >> 4), dim=-1).flatten(-2).unflatten(-1, (c["page"], -1))
            z[page, :, off] = zeros
            z = z.flatten(-2)
            s[k + "z"].copy_(z[..., 0::2] | (z[..., 1::2] << 4))
    return pool


def _counts(index, n):
    """How often each of 0..n-1 is in `index` (n: nowhere)."""
    return torch.zeros(n + 1, dtype=torch.int32, device=DEV).index_add_(
        0, index.flatten(), torch.ones(index.numel(), dtype=torch.int32, device=DEV))[:n]


def _plain_update(st):
    c, pool = st["c"], st["pool"]
    page, mp, n = c["page"], c["max_pages"], c["pages"]
    parents, grow, old = st["parents"].long(), st["grow"].long(), st["table"].long()
    has = (parents >= 0) & (parents < old.shape[0])
    at = torch.where(has, parents, torch.zeros_like(parents))
    before = torch.where(has, st["lens"].long()[at], torch.zeros_like(at)).clamp(0, mp * page)
    after = (before + grow).clamp(0, mp * page)
    up = lambda x: (x + page - 1) // page  # noqa: E731
    kept, held = torch.minimum(up(before), up(after)), up(after)
    slot, i = torch.arange(mp, device=DEV)[None], torch.arange(parents.numel(), device=DEV)
    row = old[at]
    row = torch.where((slot < kept[:, None]) & (row >= 0) & (row < n), row, torch.full_like(row, -1))
    nowhere = torch.where(row < 0, torch.full_like(row, n), row)
    refs = _counts(nowhere, n)
    # rows that go on in a partly filled page: the lowest keeps it if nobody else holds it, the others copy it
    last = (before // page).clamp(max=mp - 1)
    mine = row.gather(1, last[:, None])[:, 0]
    writes = (after > before) & (before % page > 0) & (mine >= 0)
    target = torch.where(writes, mine, torch.full_like(mine, n))
    writers = _counts(target, n)
    lowest = torch.full((n + 1,), parents.numel(), device=DEV).scatter_reduce_(0, target, i, "amin")[:n]
    m = mine.clamp(min=0)
    copies = writes & ~((lowest[m] == i) & (refs[m] == writers[m]))
    # fresh pages, in ascending order, row by row: the copy first
    need = copies.long() + held - kept
    base = torch.cumsum(need, 0) - need
    free = torch.argsort((refs > 0).to(torch.uint8), stable=True)
    n_free = (refs == 0).sum()
    take = lambda k: torch.where(k < n_free, free[k.clamp(0, n - 1)], torch.full_like(k, -1))  # noqa: E731
    fresh = take(base[:, None] + copies.long()[:, None] + slot - kept[:, None])
    new = torch.where(slot < kept[:, None], row, torch.where(slot < held[:, None], fresh, torch.full_like(fresh, -1)))
    private = take(base)
    new = torch.where(copies[:, None] & (slot == last[:, None]), private[:, None].expand_as(new), new)
    done = copies & (private >= 0)
    pool[:, private[done]] = pool[:, mine[done]]
    refs = _counts(torch.where(new < 0, torch.full_like(new, n), new), n)
    used = (refs > 0).sum()
    status = torch.stack((used, (need.sum() - n_free).clamp(min=0), done.sum(), n - used)).to(torch.int32)
    return {"pool": pool, "table": new.to(torch.int32), "lens": after.to(torch.int32), "refs": refs, "status": status}


def _plain_compact(st):
    c, pool = st["c"], st["pool"]
    page, mp, n = c["page"], c["max_pages"], c["pages"]
    old, lens = st["table"].long(), st["lens"].long().clamp(0, mp * page)
    slot = torch.arange(mp, device=DEV)[None]
    held = (slot < ((lens + page - 1) // page)[:, None]) & (old >= 0) & (old < n)
    refs = _counts(torch.where(held, old, torch.full_like(old, n)), n)
    live = refs > 0
    total, ids = live.sum(), torch.arange(n, device=DEV)
    if "into" in st:
        rank = torch.cumsum(live, 0) - 1
        room = st["into"].shape[1]
        to = torch.where(live & (rank < room), rank, torch.full_like(rank, -1))
        moves = to >= 0
        st["into"][:, to[moves]] = pool[:, ids[moves]]
        out, lacking = st["into"], (total - room).clamp(min=0)
    else:
        movers, holes = ids[live & (ids >= total)], ids[~live & (ids < total)]
        to = torch.where(live, ids, torch.full_like(ids, -1)).index_put((movers,), holes)
        moves = live & (ids >= total)
        pool[:, holes] = pool[:, movers]
        room, out, lacking = n, pool, total * 0
    table = torch.where(held, to[old.clamp(0, n - 1)], torch.full_like(old, -1))
    refs = _counts(torch.where(table < 0, torch.full_like(table, room), table), room)
    status = torch.stack((total, lacking, moves.sum(), room - (refs > 0).sum())).to(torch.int32)
    return {"pool": out, "table": table.to(torch.int32), "refs": refs, "status": status}


_run_plain = {"attention": _plain_attention, "append": _plain_append, "update": _plain_update, "compact": _plain_compact}


# ---------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without

def _record(c):
    """Bytes of one token's K and V of one head in the cache."""
    ng = c["d"] // c["group"]
    return 2 * (c["d"] / 2 + ng * (4 if c["sdt"] == "f32" else 2) + (0 if c["sym"] else ng / 2))


def work(case):
    c = case
    e = 4 if c.get("dtype") == "f32" else 2
    if c["op"] in ("attention", "append"):
        new, total = (x.double() for x in _lengths(c))
        if c["op"] == "append":
            t = float(new.sum())
            return {"bytes": t * c["hkv"] * (2 * c["d"] * e + _record(c)), "flops": t * c["hkv"] * c["d"] * (math.log2(c["d"]) + 8)}
        first = total - new
        seen = total.clone()          # keys that some query of the sequence sees
        pairs = new * first + new * (new + 1) / 2
        if c["window"]:
            w = float(c["window"])
            seen = torch.minimum(total, w + new - 1)
            lo = torch.clamp(w - first, min=0).minimum(new)  # queries whose window reaches the first key
            pairs = lo * first + lo * (lo + 1) / 2 + (new - lo) * w
        return {"bytes": float(seen.sum()) * c["hkv"] * _record(c) + 2 * float(new.sum()) * c["hq"] * c["d"] * e,
                "flops": 4.0 * c["d"] * c["hq"] * float(pairs.sum())}
    st_bytes = layout(c)[2] * c["layers"]
    if c["op"] == "update":
        # about a quarter of the rows needs a private page
        meta = 4 * (c["rows"] + c["new_rows"]) * c["max_pages"] + 4 * c["pages"]
        return {"bytes": meta + 2 * st_bytes * 0.25 * c["new_rows"], "flops": 0}
    room = max(1, min(c["max_pages"], c["pages"] // (2 * c["rows"])))
    live = min(c["rows"], c["pages"] // 2) * max(1.0, room * 0.525) * 0.95
    moved = min(live, c["into"]) if c["into"] else live * (1 - live / c["pages"])
    return {"bytes": 8 * c["rows"] * c["max_pages"] + 4 * c["pages"] + 2 * st_bytes * moved, "flops": 0}


# ---------------------------------------------------------------------------------------------------------------------
# attention's definition in 64 bits, a sequence and a head at a time

def exact(case, seed):
    c = case
    if c["op"] != "attention":
        return None  # whole numbers only
    st = prepare(case, seed)
    d, grp, page, rep = c["d"], c["group"], c["page"], c["hq"] // c["hkv"]
    cu, lens, table = st["cu"].tolist(), st["lens"].tolist(), st["table"].cpu().numpy()
    if sum((b - a) * n for a, b, n in zip(cu, cu[1:], lens)) * c["hq"] * d > 4e13:
        return None
    a = np.arange(d)
    sign = np.array([[bin(i & j).count("1") & 1 for j in a] for i in a])
    had = torch.from_numpy((1.0 - 2.0 * sign) / math.sqrt(d)).to(DEV)
    q = torch.matmul(st["q"].double(), had)
    at, head, _ = layout(c)
    ng, es = d // grp, 4 if c["sdt"] == "f32" else 2
    out = torch.zeros((st["tokens"], c["hq"], d), dtype=torch.float64, device=DEV)

    def rows(raw, name, n):
        """n vectors of one head in 64 bits from the bytes [pages, head] of its pages."""
        o = at[name + "c"]
        b = raw[:, o: o + page * d // 2].reshape(-1, d // 2)[:n]
        x = torch.empty((n, d), dtype=torch.float64, device=DEV)
        x[:, 0::2], x[:, 1::2] = b.remainder(16).double(), b.div(16, rounding_mode="floor").double()
        o = at[name + "s"]
        s = raw[:, o: o + page * ng * es].contiguous().view(torch.float32 if es == 4 else torch.bfloat16)
        s = s.reshape(-1, ng)[:n].double().repeat_interleave(grp, 1)
        if c["sym"]:
            return (x - 16.0 * (x > 7)) * s
        o = at[name + "z"]
        b = raw[:, o: o + page * ng // 2].reshape(-1, 1)
        z = torch.cat((b.remainder(16), b.div(16, rounding_mode="floor")), 1).double().reshape(-1, ng)[:n]
        return (x - z.repeat_interleave(grp, 1)) * s

    for b, n in enumerate(lens):
        t0, t1 = cu[b], cu[b + 1]
        if t1 == t0 or n == 0:
            continue
        ids = torch.from_numpy(table[b, : -(-n // page)].astype(np.int64)).to(DEV)
        pos = torch.arange(n - (t1 - t0), n, device=DEV)[:, None]
        j = torch.arange(n, device=DEV)[None]
        hidden = j > pos
        if c["window"]:
            hidden = hidden | (j <= pos - c["window"])
        for h in range(c["hkv"]):
            raw = st["pool"][ids, h * head: (h + 1) * head]
            k, v = rows(raw, "k", n), rows(raw, "v", n)
            for r in range(h * rep, (h + 1) * rep):
                w = torch.matmul(q[t0:t1, r], k.t()) / math.sqrt(d)
                w = w.masked_fill(hidden, -math.inf).nan_to_num(nan=-math.inf)
                out[t0:t1, r] = torch.matmul(torch.softmax(w, -1).nan_to_num(nan=0.0), v)
    return out
