"""Latent attention over the paged 4-bit cache on the GPU against its definitions
in float64 (oracle/latent.py) at the sizes, masks and layouts where it can go wrong.

Tolerances.  Pages that are written follow the rules of tests/parity.py for
rotate_quantize_act.  Absorbed attention: with u the rounding of a float16 operand
(2^-11; pairs of float16 for float32 activations: 2^-22), a score errs by
    e = (u + (D + 8) 2^-24) scale sum |q'_i c_i|      (codes are exact)
        + (72 2^-24) scale sum |q_r r|                (exact products, float32 sums)
        + log2(D) 2^-24 scale ||q|| ||c||             (the query's rotation)
        + 2^-20                                       (the exponent)
a probability by a factor exp(2 e), and by u in its product or, where it is a
float16 subnormal of its unit (at least 2^8 for the largest), by 2^-33 of the
largest p s; the vector of sums errs in its norm by
    (exp(2 e) - 1 + 2 u + (keys / 32 + 64) 2^-24) || sum p |c| || + keys 2^-33 || max p 15 s ||
which the rotation back leaves (it is orthogonal, and adds log2(D) 2^-24 of the
norm), and an element by no more, and by its own rounding (2^-8, or 2^-23).
Expanded attention: products are exact, so e = (N + 72) 2^-24 scale sum |q_i k_i|
+ 2^-20, probabilities are rounded to bfloat16 (2^-8), and an element errs by
    (exp(2 e) - 1 + 2^-8 + (keys / 32 + 64) 2^-24) sum p |v| + 2^-8 of itself.
The root mean square over a case is also held to what rounding the result once
leaves (at most 2^-9), times 1.3, and for expanded attention, whose probabilities
are rounded as well, twice that in the sum of squares, for rows of many keys.
"""
import math
import sys

import numpy as np
import pytest
import torch

import hadamard_rotation_preprocessing_amd as hr
import oracle
from oracle import latent as O
from parity import Report, check_int

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the gpu-marked tests need an MI355X")
    hr.lib()


def spec_of(c):
    return hr.LatentSpec(c.d, c.rope, c.page, hr.QSpec("int", 4, c.group, c.sym, c.sdt))


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def randn(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(shape, generator=g)).to(dtype)


def make_table(c, lens, seed, max_pages=None, spare=2):
    rng = np.random.default_rng(seed)
    need = [-(-n // c.page) for n in lens]
    n_pages = sum(need) + spare
    ids = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(lens), max_pages or max(max(need), 1)), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at: at + k]
        at += k
    return table, n_pages


def poison_unseen(pool, c, table, lens):
    """NaN scales and rotary keys past each length and in pages that nobody holds."""
    held = set()
    for b, n in enumerate(lens):
        for j in range(-(-n // c.page)):
            p = int(table[b, j])
            if 0 <= p < len(pool):
                held.add(p)
                for s in range(c.page):
                    if j * c.page + s >= n:
                        O.poison(pool, c, p, s)
    for p in set(range(len(pool))) - held:
        for s in range(c.page):
            O.poison(pool, c, p, s)


def cu_of(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


FORMATS = [(512, 128, False, "bf16"), (512, 256, False, "f32"), (512, 512, False, "bf16"), (512, 128, True, "f32"),
           (512, 512, True, "bf16"), (256, 128, False, "bf16"), (256, 256, False, "f32"), (256, 256, True, "bf16")]


# ---------------------------------------------------------------------------
# append and read

@pytest.mark.parametrize("d,group,sym,sdt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rotate", [True, False])
def test_append_formats(d, group, sym, sdt, dtype, rotate):
    """What is written equals the definition by the rules of rotate_quantize_act,
    nothing else changes, and latent_read gives it back."""
    c = O.LatentDef(d, 16, group, sym, sdt)
    say("append", c, dtype, rotate)
    seqs = [(5, 5), (1, 40), (0, 20), (17, 50), (2, 33)]
    new, lens = [n for n, _ in seqs], [n for _, n in seqs]
    table, n_pages = make_table(c, lens, d)
    cu = cu_of(new)
    x, rope = randn((int(cu[-1]), d), dtype, d), randn((int(cu[-1]), 64), dtype, d + 1)
    pool = torch.randint(0, 256, (n_pages, c.page_bytes), dtype=torch.uint8, generator=torch.Generator().manual_seed(1))
    before = pool.numpy().copy()
    gp = pool.to(DEV)
    hr.latent_append(gp, spec_of(c), x.to(DEV), rope.to(DEV), gpu(table), ints(lens), cu_q=gpu(cu), rotate=rotate)
    after = gp.cpu().numpy()
    y = oracle.rotate(x, d, d) if rotate else x.double().numpy()
    codes, scales, zeros, want_rope = [], [], [], []
    touched = np.zeros(before.shape, dtype=bool)
    es = 4 if sdt == "f32" else 2
    for b, (n, length) in enumerate(seqs):
        for i in range(n):
            pos = length - n + i
            p, s = table[b, pos // 16], pos % 16
            row = after[p]
            codes.append(O.section(row, c, "codes").reshape(16, -1)[s])
            scales.append(O.section(row, c, "scales").reshape(16, -1)[s])
            want_rope.append(O.section(row, c, "rope").reshape(16, -1)[s])
            off = c.offsets()[0]
            for name, width in (("codes", d // 2), ("scales", c.ng * es), ("rope", 128)):
                touched[p, off[name][0] + s * width: off[name][0] + (s + 1) * width] = True
            if not sym:
                for g in range(c.ng):
                    at = s * c.ng + g
                    zeros.append(O.section(row, c, "zeros")[at // 2] >> (4 * (at % 2)) & 15)
                    touched[p, off["zeros"][0] + at // 2] = True
    # (a byte of zero points that holds a neighbour's too keeps that half)
    if not sym and c.ng == 1:
        for b, (n, length) in enumerate(seqs):
            if n and (length - n) % 2:
                at, p = length - n - 1, table[b, (length - n) // 16]
                assert O.section(after[p], c, "zeros")[at % 16 // 2] & 15 == O.section(before[p], c, "zeros")[at % 16 // 2] & 15
            if n and length % 2:
                at, p = length - 1, table[b, (length - 1) // 16]
                assert O.section(after[p], c, "zeros")[at % 16 // 2] >> 4 == O.section(before[p], c, "zeros")[at % 16 // 2] >> 4
    assert np.array_equal(after[~touched], before[~touched])
    z = np.array(zeros, dtype=np.uint8)
    z = np.concatenate((z, np.zeros(z.size % 2, dtype=np.uint8)))
    out = {"codes": torch.from_numpy(np.stack(codes)), "zeros": None if sym else torch.from_numpy(z[0::2] | (z[1::2] << 4)),
           "scales": torch.from_numpy(np.stack(scales)).view(F32 if sdt == "f32" else BF)}
    check_int(out, y, group, sym, sdt, Report())
    assert np.array_equal(np.stack(want_rope).reshape(-1), rope.to(BF).contiguous().view(torch.uint8).numpy().reshape(-1))
    # read it back: every position of every sequence, one past the end, as the oracle has it
    ck = cu_of([n + 1 for n in lens])
    got, got_rope = hr.latent_read(gp, spec_of(c), gpu(np.pad(table, ((0, 0), (0, 1)), constant_values=-1)), ints(lens), gpu(ck), int(ck[-1]),
                                   dtype=dtype, rotate=rotate)
    for b, n in enumerate(lens):
        v, _, r, _ = O.gather(after, c, table[b], n)
        # positions that were not appended hold any bytes, scales near float32's end among
        # them: a partial sum of 512 such values, at most sum |v|, need not fit float32
        with np.errstate(invalid="ignore"):
            fits = np.abs(v).sum(1, keepdims=True) < 2.0 ** 127
        if rotate:
            v = oracle.rotate(torch.from_numpy(v), d, d)
        g = got[ck[b]: ck[b] + n].cpu().double().numpy()
        norm = np.linalg.norm(v, axis=1, keepdims=True)
        with np.errstate(invalid="ignore"):
            lim = np.abs(v) * (2.0 ** -8 if dtype is BF else 2.0 ** -23) + (math.log2(d) + 2) * 2.0 ** -24 * norm
            # (and subnormal numbers by half a step: bfloat16's is 2^-133, float32's 2^-149, in each of the transform's
            # log2(d) + 2 roundings, of d elements at most)
            lim = lim + (2.0 ** -134 if dtype is BF else 0) + (math.log2(d) + 2) * d * 2.0 ** -150
            assert ((np.abs(g - v) <= lim) | ~fits).all()
        gr = got_rope[ck[b]: ck[b] + n].cpu().double().numpy()
        assert np.array_equal(gr, r, equal_nan=True)
        assert (got[ck[b] + n] == 0).all() and (got_rope[ck[b] + n] == 0).all()


def test_append_strides_absent_pages_and_nan():
    c = O.LatentDef(512, 16, 128, False, "bf16")
    x = randn((6, 512 + 64 + 32), BF, 1)
    x[2, 130] = float("nan")
    xd = x.to(DEV)
    table = np.array([[1, -1, 2]], dtype=np.int32)
    pool = torch.zeros((4, c.page_bytes), dtype=torch.uint8, device=DEV)
    hr.latent_append(pool, spec_of(c), xd[:, :512], xd[:, 512:576], gpu(table), ints([34]))   # positions 28 to 33
    v, s, r, _ = O.gather(pool.cpu().numpy(), c, table[0], 34)
    want = oracle.rotate(x[4:, :512].contiguous(), 512, 512)
    assert np.linalg.norm(v[32:] - want) < 0.2 * np.linalg.norm(want)
    assert np.array_equal(r[32:], x[4:, 512:576].double().numpy())
    assert (pool[[0, 3]] == 0).all()
    pool.zero_()
    hr.latent_append(pool, spec_of(c), xd[:, :512], xd[:, 512:576], gpu(table), ints([6]), rotate=False)
    v, s, r, _ = O.gather(pool.cpu().numpy(), c, table[0], 6)
    assert np.isnan(v[2, 128:256]).all() and np.isfinite(v[2, :128]).all() and np.isfinite(np.delete(v, 2, 0)).all()


def test_read_without_bounds_and_into_buffers():
    c = O.LatentDef(256, 32, 256, True, "f32")
    table, n_pages = make_table(c, [40, 40], 3)
    pool = O.random_pool(c, n_pages, 3)
    buf = torch.full((80, 400), 7.0, dtype=BF, device=DEV)
    out = (buf[:, :256], buf[:, 320:384])
    got = hr.latent_read(gpu(pool), spec_of(c), gpu(table), ints([40, 40]), None, 80, out=out, rotate=False)
    assert got is out and (buf[:, 256:320] == 7).all() and (buf[:, 384:] == 7).all()
    for b in range(2):
        v, _, r, _ = O.gather(pool, c, table[b], 40)
        assert np.array_equal(out[0][40 * b: 40 * b + 40].cpu().double().numpy(), torch.from_numpy(v).to(BF).double().numpy())
        assert np.array_equal(out[1][40 * b: 40 * b + 40].cpu().double().numpy(), r)
    one = hr.latent_read(gpu(pool), spec_of(c), gpu(table), ints([40, 0]), None, 2, dtype=F32)
    assert (one[0][1] == 0).all() and (one[0][0] != 0).any()
    assert hr.latent_read(gpu(pool), spec_of(c), gpu(table), ints([40, 0]), None, 0)[0].shape == (0, 256)


# ---------------------------------------------------------------------------
# absorbed attention

def run_attention(c, seqs, heads, dtype=BF, causal=True, rotate=True, seed=0, absent=(), scale=0.07, max_q=None, use_cu=True, std=1.0,
                  rms=True, prepare=None, poisoned=True):
    say("latent attention", c, seqs if len(seqs) < 9 else len(seqs), "heads", heads, dtype, "causal", causal, "rotate", rotate)
    new, lens = [n for n, _ in seqs], [n for _, n in seqs]
    table, n_pages = make_table(c, lens, seed)
    pool = O.random_pool(c, n_pages, seed)
    if poisoned:
        poison_unseen(pool, c, table, lens)
    for b, j, v in absent:
        table[b, j] = v
    if prepare:
        prepare(pool, table)
    cu = cu_of(new)
    q, qr = randn((int(cu[-1]), heads, c.d), dtype, seed, std), randn((int(cu[-1]), heads, 64), dtype, seed + 1)
    ref, rlse, need = O.attention(q.double().numpy(), qr.double().numpy(), pool, c, table, lens, cu, scale, causal, rotate)
    out, lse = hr.latent_attention(q.to(DEV), qr.to(DEV), gpu(pool), spec_of(c), gpu(table), ints(lens), scale,
                                   cu_q=gpu(cu) if use_cu else None, max_q=max(new) if max_q is None else max_q, causal=causal,
                                   rotate=rotate, lse=True)
    torch.cuda.synchronize()
    check(out, lse, ref, rlse, need, c, dtype, max(lens), rms)
    return out


def check(out, lse, ref, rlse, need, c, dtype, keys, rms):
    wide = dtype is F32
    u, step = (2.0 ** -22, 2.0 ** -23) if wide else (2.0 ** -11, 2.0 ** -8)
    e = (u + (c.d + 8) * 2.0 ** -24) * need["score"] + 72 * 2.0 ** -24 * need["rope"] + math.log2(c.d) * 2.0 ** -24 * need["norm"] + 2.0 ** -20
    lim = (np.expm1(2 * e) + 2 * u + (keys / 32 + 64) * 2.0 ** -24) * need["value"] + keys * 2.0 ** -33 * need["unit"]
    lim = (lim + math.log2(c.d) * 2.0 ** -24 * need["size"])[..., None] + np.abs(ref) * step + 1e-30
    g = out.cpu().double().numpy()
    bad = ~((np.abs(g - ref) <= lim) | (np.isnan(g) & np.isnan(ref)))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("output %s: gpu %r oracle %r, bound %r; %d of %d off" % (i, g[i], ref[i], lim[i], bad.sum(), bad.size))
    fine = np.isfinite(ref)
    if rms and np.linalg.norm(ref[fine]) > 0:
        rel = np.linalg.norm((g - ref)[fine]) / np.linalg.norm(ref[fine])
        say("  relative error %.3g" % rel)
        assert rel <= (2e-6 if wide else 1.3 * 2.0 ** -9)
    if lse is not None:
        l, inf = lse.cpu().double().numpy(), rlse == -np.inf
        assert (l[inf] == -np.inf).all()
        ok = (np.abs(l - rlse) <= e + 2.0 ** -18 * (1 + np.abs(rlse))) | (np.isnan(l) & np.isnan(rlse))
        assert ok[~inf].all()


@pytest.mark.parametrize("d,group,sym,sdt", FORMATS)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [4, 20, 48], ids=["h4", "h20", "h48"])
def test_attention_formats(d, group, sym, sdt, dtype, heads):
    """Every format, type and kernel; lengths that end inside a page, a 16-key tile
    and a 64-key step, and one-token caches."""
    run_attention(O.LatentDef(d, 32, group, sym, sdt), [(1, 1), (1, 77), (2, 130), (3, 16), (1, 160)], heads, dtype, seed=d + group + heads)


@pytest.mark.parametrize("seqs", [[(1, 1)], [(1, 1500)], [(40, 40)], [(33, 300), (1, 5)], [(0, 20), (2, 2), (0, 0), (5, 64)], [(3, 2), (1, 70)]],
                         ids=["one", "long", "prompt", "chunk", "empty-rows", "before-0"])
@pytest.mark.parametrize("kw", [dict(), dict(causal=False), dict(rotate=False)], ids=["causal", "full", "plain"])
@pytest.mark.parametrize("heads", [3, 16])
def test_attention_masks(seqs, kw, heads):
    run_attention(O.LatentDef(256, 16, 128, False, "bf16"), seqs, heads, seed=len(seqs), **kw)


def test_attention_absent_pages():
    c = O.LatentDef(512, 16, 128, False, "bf16")
    run_attention(c, [(2, 170), (5, 40), (1, 16)], 4, absent=[(0, 1, -1), (0, 5, 1 << 20), (1, 2, -7), (2, 0, -1)], seed=3)
    run_attention(c, [(1, 640)], 16, absent=[(0, j, -1) for j in range(4, 20)], seed=4)


def test_attention_many_sequences_and_parts():
    """More sequences than the numbering takes at once; sequences cut into parts of every kind."""
    run_attention(O.LatentDef(256, 16, 256, True, "bf16"), [(i % 3, 3 + i % 90) for i in range(600)], 2, seed=8)
    run_attention(O.LatentDef(256, 64, 128, False, "bf16"), [(1, 5000), (1, 64), (2, 3000), (1, 1)], 17, seed=9)
    run_attention(O.LatentDef(512, 64, 128, False, "bf16"), [(1, 9000)], 16, seed=10)


def test_attention_without_bounds():
    c = O.LatentDef(512, 64, 512, False, "bf16")
    run_attention(c, [(2, 100), (2, 40), (2, 2)], 8, use_cu=False, max_q=0, seed=5)
    run_attention(c, [(40, 100), (1, 40)], 8, max_q=1, seed=6)     # more than max_q says
    run_attention(c, [(1, 100), (1, 40)], 8, max_q=1000, seed=7)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_attention_scales_far_apart(dtype):
    """Latents 2^40 times as large or small as their neighbours, seen and unseen:
    what a row does not see has no influence, and the others keep their bits."""
    c = O.LatentDef(512, 16, 128, False, "f32")

    def far(pool, table):
        rng = np.random.default_rng(1)
        for p in range(len(pool)):
            s = O.section(pool[p], c, "scales").view("<f4")
            s *= np.where(rng.random(s.shape) < 0.1, np.float32(2.0 ** -40), np.float32(1)).astype(np.float32)
        last = pool[table[0, 4]]                       # positions 64 to 79: seen by some of the tokens
        O.section(last, c, "scales").view("<f4").reshape(16, -1)[8:] *= np.float32(2.0 ** 40)
    run_attention(c, [(8, 72)], 5, dtype, prepare=far, seed=2, scale=0.02)


def test_attention_nan_and_infinity_stay_with_their_keys():
    """A NaN latent or rotary key gives NaN to the tokens that see it, and to no other."""
    c = O.LatentDef(256, 16, 128, False, "bf16")

    def bad(pool, table):
        O.section(pool[table[0, 2]], c, "scales").reshape(16, -1)[5] = 0xFF     # position 37
        O.section(pool[table[1, 0]], c, "rope").reshape(16, -1)[9] = 0xFF       # position 9
    out = run_attention(c, [(6, 40), (10, 12), (1, 70)], 4, prepare=bad, poisoned=False, seed=3, rms=False)
    seen = torch.isnan(out.float()).all(-1).all(-1).cpu().tolist()
    assert seen == [False] * 3 + [True] * 3 + [False] * 7 + [True] * 3 + [False]


@pytest.mark.parametrize("std,scale", [(30.0, 0.3), (1e4, 1.0), (1e-4, 1.0), (0.0, 1.0)])
def test_attention_sharp_and_flat(std, scale):
    """Scores of hundreds and of millions (one key has all of the weight), and none at all."""
    c = O.LatentDef(256, 16, 128, False, "bf16")
    new, lens = [2], [200]
    table, n_pages = make_table(c, lens, 1)
    pool = O.random_pool(c, n_pages, 1)
    cu = cu_of(new)
    q, qr = randn((2, 4, 256), BF, 1, std), randn((2, 4, 64), BF, 2, min(std, 1.0))
    ref, rlse, need = O.attention(q.double().numpy(), qr.double().numpy(), pool, c, table, lens, cu, scale)
    out, lse = hr.latent_attention(q.to(DEV), qr.to(DEV), gpu(pool), spec_of(c), gpu(table), ints(lens), scale, lse=True)
    # where rounding of a score could pick another key nothing can be said but that it is an average of values
    top = need["score"] * (2.0 ** -10)
    calm = top < 0.05
    g = out.cpu().double().numpy()
    assert np.isfinite(g).all() and torch.isfinite(lse).all()
    assert (np.linalg.norm(g, axis=-1) <= need["value"] * 3 + 15 * 256).all()
    if calm.all():
        check(out, lse, ref, rlse, need, c, BF, 200, True)
    # scores err by need["score"] 2^-10 and 2^-17 of their own size (float32 in the exponent)
    assert (np.abs(lse.cpu().double().numpy() - rlse) <= top + 2.0 ** -17 * (1 + np.abs(rlse))).all()


def test_attention_strides_and_in_place():
    c = O.LatentDef(512, 64, 128, False, "bf16")
    table, n_pages = make_table(c, [150, 30], 1)
    pool = gpu(O.random_pool(c, n_pages, 1))
    args = (pool, spec_of(c), gpu(table), ints([150, 30]), 0.07)
    both = randn((2, 8, 512 + 64), BF, 1).to(DEV)
    want = hr.latent_attention(both[..., :512].contiguous(), both[..., 512:].contiguous(), *args)
    got = hr.latent_attention(both[..., :512], both[..., 512:], *args)
    assert torch.equal(got, want)
    heads_first = torch.empty((8, 2, 512), dtype=BF, device=DEV).transpose(0, 1)
    assert torch.equal(hr.latent_attention(both[..., :512], both[..., 512:], *args, out=heads_first), want)
    rope = both[..., 512:].clone()
    assert torch.equal(hr.latent_attention(both[..., :512], both[..., 512:], *args, out=both[..., :512]), want)   # into q itself
    assert torch.equal(both[..., 512:], rope)


def test_attention_rotation_fused_into_the_maps():
    """q in the rotated space with rotate off gives the rotated result."""
    c = O.LatentDef(256, 16, 256, False, "f32")
    table, n_pages = make_table(c, [90], 1)
    pool = gpu(O.random_pool(c, n_pages, 1))
    q, qr = randn((1, 4, 256), F32, 1).to(DEV), randn((1, 4, 64), F32, 2).to(DEV)
    args = (pool, spec_of(c), gpu(table), ints([90]), 0.1)
    a = hr.latent_attention(q, qr, *args)
    b = hr.latent_attention(hr.rotate(q), qr, *args, rotate=False)
    assert torch.allclose(hr.rotate(b), a, rtol=0, atol=2e-5 * a.abs().max().item())


# ---------------------------------------------------------------------------
# expanded attention

def run_prompt(seqs, heads, nope, causal=True, scale=None, seed=0, std=1.5, prepare=None, rms=True):
    say("prompt", seqs if len(seqs) < 9 else len(seqs), "heads", heads, "nope", nope, "causal", causal)
    cu_q, cu_k = cu_of([n for n, _ in seqs]), cu_of([n for _, n in seqs])
    t, p = int(cu_q[-1]), int(cu_k[-1])
    q, kv, rope = randn((t, heads, nope + 64), BF, seed, std), randn((p, heads, 2 * nope), BF, seed + 1), randn((p, 64), BF, seed + 2)
    if prepare:
        prepare(kv, rope)
    k, v = kv[..., :nope], kv[..., nope:]
    ref, rlse, score, value = O.prompt(q.double().numpy(), k.double().numpy(), rope.double().numpy(), v.double().numpy(), cu_q, cu_k, scale, causal)
    kvd = kv.to(DEV)
    out, lse = hr.latent_prompt_attention(q.to(DEV), kvd[..., :nope], rope.to(DEV), kvd[..., nope:], gpu(cu_q), gpu(cu_k), scale=scale,
                                          causal=causal, lse=True)
    torch.cuda.synchronize()
    keys = max(n for _, n in seqs)
    e = (nope + 72) * 2.0 ** -24 * score + 2.0 ** -20
    g, l, inf = out.cpu().double().numpy(), lse.cpu().double().numpy(), rlse == -np.inf
    with np.errstate(invalid="ignore"):
        lim = (np.expm1(2 * e) + 2.0 ** -8 + (keys / 32 + 64) * 2.0 ** -24)[..., None] * value + np.abs(ref) * 2.0 ** -8 + 1e-30
        bad = ~((np.abs(g - ref) <= lim) | (g == ref) | (np.isnan(g) & np.isnan(ref)))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("output %s: gpu %r oracle %r, bound %r; %d of %d off" % (i, g[i], ref[i], lim[i], bad.sum(), bad.size))
    fine = np.isfinite(ref)
    if rms and np.linalg.norm(ref[fine]) > 0:
        rel = np.linalg.norm((g - ref)[fine]) / np.linalg.norm(ref[fine])
        say("  relative error %.3g" % rel)
        # (a row of few keys may have all of its probabilities rounded the same way)
        assert rel <= (1.3 * math.sqrt(2) * 2.0 ** -9 if min(n - m for m, n in seqs) >= 64 else 2.0 ** -8 + 2.0 ** -9)
    assert (l[inf] == -np.inf).all() and (g[inf] == 0).all()
    ok = (np.abs(l - rlse) <= e + 2.0 ** -18 * (1 + np.abs(rlse))) | (np.isnan(l) & np.isnan(rlse))
    assert ok[~inf].all()
    return g


@pytest.mark.parametrize("nope", [64, 128])
@pytest.mark.parametrize("seqs", [[(1, 1)], [(1, 300)], [(77, 77)], [(130, 200), (1, 5), (64, 64)], [(0, 20), (2, 2), (0, 0), (129, 129), (5, 64)],
                                  [(3, 2), (5, 0), (1, 70)], [(200, 700)]],
                         ids=["one", "long", "prompt", "ragged", "empty-rows", "before-0", "chunk"])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_masks(nope, seqs, causal):
    run_prompt(seqs, 3, nope, causal, seed=len(seqs) + nope)


def test_prompt_many_sequences_heads_and_scale():
    run_prompt([(i % 4, 2 + i % 50) for i in range(300)], 2, 64, seed=1)
    run_prompt([(20, 30)], 40, 128, scale=0.01, seed=2)


@pytest.mark.parametrize("nope", [64, 128])
def test_prompt_infinities_and_nan_where_they_are_not_seen(nope):
    """Values and keys that are infinite or NaN reach the tokens that see them, and no
    other: inside a step that is masked, past the sequence, and in another one's."""
    def bad(kv, rope):
        kv[100, 0, nope + 3] = float("inf")      # a value of the first sequence, position 100
        kv[70, 1, nope + 9] = float("nan")
        kv[90, 2, 5] = float("nan")              # a key
        kv[150:, :, nope:] = float("nan")        # all values of the second
    g = run_prompt([(150, 150), (20, 30)], 3, nope, seed=4, prepare=bad, rms=False)
    assert np.isfinite(g[:70]).all() and np.isfinite(g[:100, 0]).all() and not np.isfinite(g[101:150, 0, 3]).any()
    assert np.isnan(g[70:150, 1, 9]).all() and np.isfinite(np.delete(g[70:150, 1], 9, 1)).all() and np.isnan(g[150:]).all()

    def rope_nan(kv, rope):
        rope[40, 7] = float("nan")
    g = run_prompt([(60, 60)], 2, nope, seed=5, prepare=rope_nan, rms=False)
    assert np.isfinite(g[:40]).all() and np.isnan(g[40:]).all()


@pytest.mark.parametrize("std", [1e4, 200.0, 0.0])
def test_prompt_sharp_and_flat(std):
    g = run_prompt([(90, 170)], 2, 64, seed=6, std=std, rms=False)
    assert np.isfinite(g).all()


def test_prompt_strides():
    q, kv, rope = randn((70, 4, 192), BF, 1).to(DEV), randn((100, 4, 256), BF, 2).to(DEV), randn((100, 64), BF, 3).to(DEV)
    cu_q, cu_k = ints([0, 70]), ints([0, 100])
    want = hr.latent_prompt_attention(q, kv[..., :128].contiguous(), rope, kv[..., 128:].contiguous(), cu_q, cu_k)
    wide = torch.zeros((70, 4, 400), dtype=BF, device=DEV)
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)
    ropes = torch.zeros((100, 96), dtype=BF, device=DEV)
    ropes[:, 16:80] = rope
    got = hr.latent_prompt_attention(heads_first, kv[..., :128], ropes[:, 16:80], kv[..., 128:], cu_q, cu_k, out=wide[..., 100 - 4: 224])
    assert torch.equal(got, want) and (wide[..., :96] == 0).all() and (wide[..., 224:] == 0).all()


# ---------------------------------------------------------------------------
# together

def test_the_forms_agree_and_pages_move():
    """A prompt and a step over a pool that is updated, forked and compacted: the
    absorbed form over the cache and the expanded one over what latent_read gives
    are the same attention, within the rounding of expanded keys and values."""
    heads, nope, d = 4, 128, 512
    spec = hr.LatentSpec(d, 64, 16, hr.QSpec("int", 4, 128, False, "bf16"))
    pool = hr.cache_pool(spec, 40)
    table, lens = torch.full((3, 12), -1, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    w = randn((d, heads * 2 * nope), F32, 1).to(DEV) / math.sqrt(d)
    wk, wv = (x.contiguous() for x in w.view(d, heads, 2, nope).permute(2, 1, 3, 0))       # [heads, nope, d]

    def step(parents, grow, seed):
        nonlocal table, lens
        s = hr.cache_update(pool, spec, table, lens, ints(parents), ints(grow))
        table, lens = s["table"], s["lens"]
        t = sum(grow)
        cu = gpu(cu_of(grow))
        c, rope = randn((t, d), BF, seed).to(DEV), randn((t, 64), BF, seed + 1).to(DEV)
        q = randn((t, heads, nope + 64), BF, seed + 2).to(DEV)
        hr.latent_append(pool, spec, c, rope, table, lens, cu_q=cu)
        scale = 1 / math.sqrt(nope + 64)
        qc = torch.bmm(q[..., :nope].float().transpose(0, 1).contiguous(), wk).transpose(0, 1).to(BF)
        o = hr.latent_attention(qc, q[..., nope:], pool, spec, table, lens, scale, cu_q=cu)
        a = torch.bmm(o.float().transpose(0, 1).contiguous(), wv.transpose(1, 2).contiguous()).transpose(0, 1)
        n = lens.tolist()
        ck = gpu(cu_of(n))
        lat, r = hr.latent_read(pool, spec, table, lens, ck, sum(n))
        kv = (lat.float() @ w).to(BF).view(-1, heads, 2 * nope)
        b = hr.latent_prompt_attention(q, kv[..., :nope], r, kv[..., nope:], cu, ck).float()
        # q_c, o, the latents read and kv are each rounded to bfloat16 once (rms 2^-9 at
        # most each), scores of size 1 turn that into as much again
        assert torch.linalg.vector_norm(a - b) <= 8 * 2.0 ** -9 * torch.linalg.vector_norm(b)
        return o
    step([-1, -1, -1], [50, 7, 33], 10)
    step([0, 0, 2], [1, 3, 1], 20)          # the second row gives way to a fork of the first
    before = hr.latent_read(pool, spec, table, lens, None, 3 * 30)
    s = hr.cache_compact(pool, spec, table, lens)
    table = s["table"]
    assert s["status"][0].item() == int((s["refs"] > 0).sum())
    after = hr.latent_read(pool, spec, table, lens, None, 3 * 30)
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    other = hr.cache_pool(spec, 20)
    s = hr.cache_compact(pool, spec, table, lens, into=other)
    assert torch.equal(hr.latent_read(other, spec, s["table"], lens, None, 90)[0], after[0])
    step([0, 1, 2], [1, 1, 1], 30)


@pytest.mark.parametrize("heads,dtype", [(8, BF), (40, BF), (20, F32)])
def test_captured_steps_replay(heads, dtype):
    """A captured step (append, attention) replays over changed lengths, with eager
    work between the replays."""
    c = O.LatentDef(512, 64, 128, False, "bf16")
    spec = spec_of(c)
    table, n_pages = make_table(c, [400, 90], 1)
    table = gpu(table)
    pool = gpu(O.random_pool(c, n_pages, 1))
    lens = ints([300, 70])
    x, rope = randn((2, 512), dtype, 1).to(DEV), randn((2, 64), dtype, 2).to(DEV)
    q, qr = randn((2, heads, 512), dtype, 3).to(DEV), randn((2, heads, 64), dtype, 4).to(DEV)
    out = torch.empty_like(q)


    def step(into):
        hr.latent_append(pool, spec, x, rope, table, lens)
        hr.latent_attention(q, qr, pool, spec, table, lens, 0.07, max_q=1, out=into)
    step(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    for k in range(4):
        lens += 3
        x.copy_(randn((2, 512), dtype, 10 + k))
        q.copy_(randn((2, heads, 512), dtype, 20 + k))
        graph.replay()
        torch.cuda.synchronize()
        got, eager = out.clone(), torch.empty_like(q)
        step(eager)
        torch.cuda.synchronize()
        assert torch.equal(got, eager)


def test_another_stream():
    c = O.LatentDef(512, 64, 128, False, "bf16")
    table, n_pages = make_table(c, [700], 1)
    pool = gpu(O.random_pool(c, n_pages, 1))
    q, qr = randn((1, 32, 512), BF, 3).to(DEV), randn((1, 32, 64), BF, 4).to(DEV)
    args = (pool, spec_of(c), gpu(table), ints([700]), 0.07)
    want = hr.latent_attention(q, qr, *args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [hr.latent_attention(q, qr, *args) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)
