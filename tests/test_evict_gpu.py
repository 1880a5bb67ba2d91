"""Eviction from the paged 4-bit cache on the GPU against its definition in
float64 (oracle/evict.py) at the sizes, masks and layouts where it can go wrong.

Tolerances.  An eviction moves bytes: everything is equal.  Weights are sums of
p = exp(x - lse) with x = scale q'.k, and err by the arithmetic of x: the query is
a pair of float16 (relative 2^-22), products with codes are exact and summed in
float32 in 2 D steps at most (2 D 2^-24), the rotation rounds log2(D) times
(2^-24 of the vector's norm each), and the scales, the factor and the exponent's
own rounding are six more roundings of x and of lse; then
    |dp| <= p (exp(e) - 1 + 2^-22),  e = (2^-22 + (2 D + 6) 2^-24) scale |q'|.|k|
                                         + 8 2^-24 scale ||q|| ||k|| + 6 2^-24 (|lse| + 1)
with e below 0.01, where exp(e) - 1 <= 1.01 e; sums of n rows add log-like parts,
at most (n / 16 + 40) 2^-24 of the sum, and decay and the last addition 2 2^-24 of
the result.
"""
import sys

import numpy as np
import pytest
import torch

import hadamard_rotation_preprocessing_amd as hr
from oracle import cache as O
from oracle import evict as E
from test_cache_gpu import gpu, ints, make_q, make_table, spec_of

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


def poison_unseen(pool, c, table, lens):
    """NaN scales in positions past each length and in pages that nobody holds."""
    held = set()
    for b, n in enumerate(lens):
        for j in range(-(-n // c.page)):
            p = int(table[b, j])
            if not 0 <= p < len(pool):
                continue
            held.add(p)
            for s in range(c.page):
                if j * c.page + s >= n:
                    O.poison(pool, c, p, s)
    for p in set(range(len(pool))) - held:
        for s in range(c.page):
            O.poison(pool, c, p, s)


def run_weights(c, seqs, hq, dtype=BF, window=0, causal=True, rotate=True, seed=0, decay=0.9, absent=(), scale=None, extra=0, max_q=0):
    say("weights", c, seqs if len(seqs) < 9 else len(seqs), "hq", hq, dtype, "window", window, "causal", causal, "rotate", rotate)
    new, lens = [n for n, _ in seqs], [n for _, n in seqs]
    table, n_pages = make_table(c, lens, seed)
    pool = O.random_pool(c, n_pages, seed)
    poison_unseen(pool, c, table, lens)
    for b, j, v in absent:
        table[b, j] = v
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = make_q(int(cu[-1]), hq, c.d, dtype, seed)
    _, lse, _ = O.attention(q.double().numpy(), pool, c, table, lens, cu, scale, causal, window, rotate)
    lse = lse.astype(np.float32)
    width = table.shape[1] * c.page + extra
    old = np.random.default_rng(seed).random((len(seqs), c.heads, width)).astype(np.float32)
    for b, n in enumerate(lens):       # what new positions held before does not matter
        old[b, :, max(n - new[b], 0):n] = np.nan if new[b] else old[b, :, max(n - new[b], 0):n]
    ref, need = E.weights(q.double().numpy(), pool, c, table, lens, cu, lse, old, scale, causal, window, rotate, decay)
    w = gpu(old)
    got = hr.cache_weights(q.to(DEV), gpu(pool), spec_of(c), gpu(table), ints(lens), gpu(lse), w, cu_q=gpu(cu), max_q=max_q,
                           scale=scale, causal=causal, window=window, rotate=rotate, decay=decay)
    assert got is w
    torch.cuda.synchronize()
    check_weights(w, ref, need, c, max(new) * (hq // c.heads))
    return w


def check_weights(w, ref, need, c, rows):
    e = (2.0 ** -22 + (2 * c.d + 6) * 2.0 ** -24) * need[1] + 8 * 2.0 ** -24 * need[2] + 6 * 2.0 ** -24 * need[3]
    lim = 1.01 * e + need[0] * (2.0 ** -22 + (rows / 16 + 40) * 2.0 ** -24) + 2 * 2.0 ** -24 * np.abs(ref) + 1e-30
    g = w.cpu().double().numpy()
    bad = ~((np.abs(g - ref) <= lim) | (np.isnan(g) & np.isnan(ref)))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("weight %s: gpu %r oracle %r, bound %r; %d of %d off" % (i, g[i], ref[i], lim[i], bad.sum(), bad.size))
    fine = np.isfinite(ref)
    say("  relative error %.3g" % (np.linalg.norm((g - ref)[fine]) / max(np.linalg.norm(ref[fine]), 1e-30)))


@pytest.mark.parametrize("d,group", [(64, 64), (64, 32), (128, 128), (128, 64), (128, 32), (256, 256), (256, 128), (256, 64), (256, 32)])
@pytest.mark.parametrize("sym,sdt", [(False, "bf16"), (True, "f32")], ids=["asym-bf16", "sym-f32"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_weights_formats(d, group, sym, sdt, dtype):
    """Every head dimension, group size, symmetry and type; lengths that end
    inside a page and a 16-key tile, and one-token caches."""
    c = O.CacheDef(2, d, 32, group, sym, sdt)
    run_weights(c, [(1, 1), (1, 77), (2, 130), (3, 16), (1, 160)], 6, dtype, seed=d + group)


@pytest.mark.parametrize("seqs", [[(1, 1)], [(1, 700)], [(40, 40)], [(33, 300), (1, 5)], [(0, 20), (2, 2), (0, 0), (5, 64)]],
                         ids=["one", "long", "prompt", "chunk", "empty-rows"])
@pytest.mark.parametrize("kw", [dict(), dict(window=17), dict(causal=False), dict(rotate=False, scale=0.05)],
                         ids=["causal", "window", "full", "plain"])
def test_weights_masks(seqs, kw):
    run_weights(O.CacheDef(3, 64, 16, 64, False, "bf16"), seqs, 9, seed=len(seqs), **kw)


@pytest.mark.parametrize("hq", [1, 4, 16, 64])
def test_weights_grouped_heads(hq):
    run_weights(O.CacheDef(1, 128, 64, 128, False, "bf16"), [(3, 200), (1, 90)], hq, seed=hq)


def test_weights_absent_pages_and_more_tokens_than_positions():
    c = O.CacheDef(2, 64, 16, 64, False, "bf16")
    run_weights(c, [(2, 70), (5, 40)], 4, absent=[(0, 1, -1), (1, 2, 1 << 20)], seed=3)
    run_weights(c, [(6, 4), (2, 40)], 4, seed=4)       # two of the tokens lie before position 0


def test_weights_width_beyond_the_table_is_left():
    run_weights(O.CacheDef(2, 64, 16, 64, False, "bf16"), [(2, 70), (5, 40)], 4, extra=37)


def test_weights_many_rows_and_long_prompts():
    """More rows than a workgroup numbers at once; sums over thousands of rows."""
    run_weights(O.CacheDef(1, 64, 16, 64, True, "bf16"), [(i % 3, 3 + i % 40) for i in range(600)], 2, seed=8)
    run_weights(O.CacheDef(1, 64, 64, 64, False, "bf16"), [(700, 900)], 4, seed=9, decay=0.0)


def test_weights_nan_scale_reaches_only_its_position():
    """A NaN key gives NaN to its own position alone (lse is the caller's)."""
    c = O.CacheDef(1, 64, 16, 64, False, "bf16")
    table, n_pages = make_table(c, [40], 1)
    pool = O.random_pool(c, n_pages, 1)
    cu = np.array([0, 1], dtype=np.int32)
    q = make_q(1, 2, 64, BF, 1)
    _, lse, _ = O.attention(q.double().numpy(), pool, c, table, [40], cu)
    O.poison(pool, c, int(table[0, 1]), 3)
    w = torch.zeros((1, 1, 48), device=DEV)
    hr.cache_weights(q.to(DEV), gpu(pool), spec_of(c), gpu(table), ints([40]), gpu(lse.astype(np.float32)), w)
    bad = torch.isnan(w[0, 0]).cpu().numpy()
    assert bad[19] and bad.sum() == 1


def test_weights_sum_to_the_rows_and_follow_cache_attention():
    """With cache_attention's own log-sum-exp each row's weights sum to 1."""
    c = O.CacheDef(2, 128, 64, 128, False, "bf16")
    lens, new, hq = [500, 37], [3, 2], 8
    table, n_pages = make_table(c, lens, 5)
    pool, cu = gpu(O.random_pool(c, n_pages, 5)), np.array([0, 3, 5], dtype=np.int32)
    q = make_q(5, hq, 128, BF, 5).to(DEV)
    _, lse = hr.cache_attention(q, pool, spec_of(c), gpu(table), ints(lens), cu_q=gpu(cu), lse=True)
    w = torch.zeros((2, 2, table.shape[1] * 64), device=DEV)
    hr.cache_weights(q, pool, spec_of(c), gpu(table), ints(lens), lse, w, cu_q=gpu(cu))
    # (the log-sum-exp errs by up to 2^-12 of rounded probabilities, and its queries by 2^-11 an element)
    assert torch.allclose(w.sum(-1).cpu(), torch.tensor([[12.0, 12.0], [8.0, 8.0]]), rtol=4e-3)


def run_evict(c, lens, budget, sinks=0, recent=0, layers=1, share=(), spare=3, seed=0, w=None, absent=(), max_pages=None, extra=0):
    say("evict", c, lens if len(lens) < 9 else len(lens), "budget", budget, "sinks", sinks, "recent", recent, "layers", layers, share)
    rng = np.random.default_rng(seed)
    table, n_pages = make_table(c, lens, seed, max_pages=max_pages, spare=spare)
    for b, j, v in absent:
        table[b, j] = v
    for b, other, k in share:          # row b starts with `other`'s first k pages
        table[b, :k] = table[other, :k]
    pool = rng.integers(0, 256, (layers, n_pages, c.page_bytes), dtype=np.uint8)
    if w is None:
        w = (rng.random((layers, len(lens), c.heads, table.shape[1] * c.page + extra)) ** 6).astype(np.float32)
        w = np.round(w * 64) / 64      # ties
    w = w.astype(np.float32)
    gp, gw = gpu(pool), gpu(w)
    if layers == 1:
        gp, gw = gp[0].contiguous(), gw[0].contiguous()
    got = hr.cache_evict(gp, spec_of(c), gpu(table), ints(lens), gw, budget, sinks, recent)
    torch.cuda.synchronize()
    ref_w = w.copy()
    ref = E.evict(pool, c, table, lens, ref_w, budget, sinks, recent)
    for name, r in zip(("table", "lens", "refs", "status"), ref):
        assert np.array_equal(got[name].cpu().numpy(), r), (name, got[name].cpu().numpy(), r)
    assert np.array_equal(gw.cpu().numpy().reshape(ref_w.shape).view(np.uint32), ref_w.view(np.uint32)), "weights"
    g = gp.cpu().numpy().reshape(pool.shape)
    if not np.array_equal(g, pool):
        bad = np.argwhere(g != pool)
        raise AssertionError("pool: %d of %d bytes differ, first %s" % (len(bad), pool.size, bad[:4].tolist()))
    return got


@pytest.mark.parametrize("d,group", [(64, 64), (64, 32), (128, 128), (128, 64), (128, 32), (256, 256), (256, 64), (256, 32)])
@pytest.mark.parametrize("sym,sdt", [(False, "bf16"), (True, "bf16"), (False, "f32"), (True, "f32")])
def test_evict_formats(d, group, sym, sdt):
    run_evict(O.CacheDef(2, d, 16, group, sym, sdt), [100, 30, 77], 41, sinks=3, recent=8, layers=2, seed=d + group)


@pytest.mark.parametrize("lens,budget,sinks,recent", [
    ([1], 1, 0, 0), ([2], 1, 0, 0), ([2], 1, 1, 0), ([2], 1, 0, 1), ([0, 5, 0], 4, 1, 1), ([50, 50], 49, 0, 0), ([50, 50], 50, 0, 0),
    ([64], 16, 16, 0), ([64], 16, 0, 16), ([64], 17, 8, 9), ([64], 15, 2, 3), ([65, 63, 200], 33, 1, 2), ([31], 1000, 0, 0)])
def test_evict_sizes(lens, budget, sinks, recent):
    for sym in (False, True):
        run_evict(O.CacheDef(1, 64, 16, 64, sym, "bf16"), lens, budget, sinks, recent, seed=budget)


@pytest.mark.parametrize("length,budget", [(4095, 1023), (4097, 4096), (9000, 5000), (9000, 4)])
def test_evict_long_rows(length, budget):
    """More positions than a chunk takes, budgets of more than a step's moves."""
    run_evict(O.CacheDef(1, 64, 64, 64, False, "bf16"), [length, length // 2], budget, 2, 1, seed=length)
    run_evict(O.CacheDef(1, 128, 64, 32, False, "f32"), [length], budget, 2, 1, seed=length)


def test_evict_equal_and_extreme_weights():
    """All equal; zeros of both signs; infinities, NaN, negative numbers, subnormals."""
    c = O.CacheDef(2, 64, 16, 64, False, "bf16")
    same = np.full((1, 2, 2, 112), 0.25)
    run_evict(c, [100, 70], 33, 2, 4, w=same)
    rng = np.random.default_rng(3)
    odd = rng.choice([0.0, -0.0, 1e-42, -1.0, np.inf, -np.inf, np.nan, 2.0, 1e-30], size=(1, 2, 2, 112))
    run_evict(c, [100, 70], 33, 2, 4, w=odd)
    bits = rng.integers(0, 1 << 32, (1, 2, 2, 112), dtype=np.uint64).astype(np.uint32).view(np.float32)
    run_evict(c, [100, 70], 50, 0, 1, w=bits)


def test_evict_shared_and_absent_pages():
    c = O.CacheDef(2, 64, 16, 64, False, "bf16")
    run_evict(c, [100, 90, 40], 41, 2, 4, layers=2, share=[(1, 0, 3)], spare=8)                 # two rows share, both are cut
    run_evict(c, [100, 30, 100], 41, 2, 4, share=[(1, 0, 1), (2, 0, 2)], spare=8)               # one that shares is short
    got = run_evict(c, [100, 100, 100, 100], 41, 2, 4, share=[(1, 0, 3), (2, 0, 3)], spare=0)   # not enough free pages
    assert got["status"][1].item() == 3 and got["status"][2].item() == 3
    got = run_evict(c, [100, 100], 41, absent=[(0, 5, -1), (1, 6, 1 << 20)])
    assert got["lens"].tolist() == [100, 41] or got["status"][2].item() <= 1
    run_evict(c, [64, 64], 20, share=[(1, 0, 4)], spare=1)                                      # one free page of four


def test_evict_large_pools_and_many_rows():
    """More pages than the plan's counters fit in LDS; more rows than it scans at once."""
    run_evict(O.CacheDef(1, 64, 16, 64, False, "bf16"), [40] * 8, 20, 1, 2, spare=12400, share=[(3, 2, 2)])
    run_evict(O.CacheDef(1, 64, 16, 64, True, "bf16"), [17 + i % 30 for i in range(1100)], 20, 1, 2)


def test_evict_wide_tables_and_caller_buffers():
    c = O.CacheDef(1, 64, 16, 64, False, "bf16")
    run_evict(c, [40, 33], 20, max_pages=37, extra=5)
    table, n = make_table(c, [40, 33], 0)
    pool = torch.zeros((n, c.page_bytes), dtype=torch.uint8, device=DEV)
    w = torch.rand((2, 1, table.shape[1] * 16), device=DEV)
    out = {"table": torch.full(table.shape, 7, dtype=torch.int32, device=DEV), "lens": ints([0, 0]), "refs": ints([9] * n), "status": ints([0] * 4)}
    got = hr.cache_evict(pool, spec_of(c), gpu(table), ints([40, 33]), w, 20, out=out)
    assert got is out and out["lens"].tolist() == [20, 20] and (out["table"][:, 2:] == -1).all()
