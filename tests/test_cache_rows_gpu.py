"""Attention over the paged 4-bit cache with many query rows, where a
workgroup's waves share the operands of the same keys (256 or 128 rows to a
workgroup).  Which kernel a call takes goes by its rows and by the keys that its
page table can hold, so the tables here are made wide: small calls take the
kernel of large ones.  Oracle and bounds as in test_cache_gpu.py."""
import numpy as np
import pytest
import torch

import hadamard_rotation_preprocessing_amd as hr
import test_cache_gpu as T
from oracle import cache as O
from test_cache_gpu import BF, DEV, F32, check_attention, gpu, gpu_ready, ints, make_q, run_attention, spec_of  # noqa: F401

pytestmark = pytest.mark.gpu
FORMATS = [(64, 64), (64, 32), (128, 128), (128, 64), (128, 32), (256, 256), (256, 128), (256, 64), (256, 32)]


@pytest.fixture(autouse=True)
def wide_tables(monkeypatch):
    """Tables of 2^22 positions, their further pages absent."""
    plain = T.make_table

    def make(c, lens, seed, max_pages=None, spare=2):
        table, n_pages = plain(c, lens, seed, max_pages, spare)
        wide = np.full((len(lens), (1 << 22) // c.page), -1, dtype=np.int32)
        wide[:, :table.shape[1]] = table
        return wide, n_pages
    monkeypatch.setattr(T, "make_table", make)


@pytest.mark.parametrize("d,group", FORMATS)
@pytest.mark.parametrize("sym", [False, True], ids=["asym", "sym"])
@pytest.mark.parametrize("sdt", ["bf16", "f32"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_formats(d, group, sym, sdt, dtype):
    c = O.CacheDef(2, d, 32, group, sym, sdt)
    run_attention(c, [(70, 70), (1, 77), (33, 130), (0, 16), (50, 161), (16, 16)], 4, dtype, seed=d + group)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("rep", [1, 3, 7, 16])
def test_pages_and_heads(page, rep):
    """Query heads per kv head that do not divide a block of rows."""
    c = O.CacheDef(1, 128, page, 128, False, "bf16")
    run_attention(c, [(130, 300), (1, 15), (97, 97), (40, 511)], rep, seed=page + rep)


@pytest.mark.parametrize("d,group,dtype", [(128, 128, BF), (128, 32, BF), (256, 256, BF), (64, 64, F32), (256, 32, F32)])
@pytest.mark.parametrize("length", [1, 31, 32, 33, 127, 128, 129, 255, 257, 900])
def test_lengths(d, group, dtype, length):
    """Lengths around a tile and a pass; fewer positions than new tokens."""
    c = O.CacheDef(1, d, 16, group, False, "bf16")
    run_attention(c, [(100, length)], 2, dtype, seed=length)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_units_cut_and_whole(dtype):
    """A long sequence whose row block is cut over many workgroups, and one
    among many short ones."""
    c = O.CacheDef(1, 128, 64, 128, False, "bf16")
    run_attention(c, [(50, 9000)], 4, dtype, seed=1)
    c = O.CacheDef(4, 64, 64, 64, False, "bf16")
    rng = np.random.default_rng(5)
    seqs = [(int(n), int(n + rng.integers(0, 40))) for n in rng.integers(0, 40, 90)]
    seqs[40] = (30, 3001)
    run_attention(c, seqs, 16, dtype, seed=2, max_q=40)


@pytest.mark.parametrize("rows", [1, 3, 70, 300, 520])
def test_sequences_per_thread(rows):
    """As many, fewer and more sequences than a workgroup has threads."""
    c = O.CacheDef(1, 64, 16, 64, False, "bf16")
    rng = np.random.default_rng(rows)
    seqs = [(int(rng.integers(0, 4)), int(rng.integers(0, 40))) for _ in range(rows)]
    seqs[rows // 2] = (45, 1200)
    run_attention(c, seqs, 4, seed=rows)


@pytest.mark.parametrize("window", [1, 33, 100, 5000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_window(window, dtype):
    c = O.CacheDef(2, 128, 16, 128, False, "bf16")
    run_attention(c, [(90, 400), (60, 60), (1, 97)], 4, dtype, window=window, seed=window)


def test_not_causal_rotation_and_scale():
    c = O.CacheDef(2, 128, 32, 64, True, "f32")
    run_attention(c, [(90, 170), (30, 1), (140, 33)], 4, causal=False, seed=8)
    run_attention(c, [(90, 500), (2, 64)], 4, F32, rotate=False, scale=0.25, seed=5)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_that_see_nothing(dtype):
    c = O.CacheDef(2, 64, 16, 64, False, "bf16")
    run_attention(c, [(100, 0), (0, 50), (70, 3), (1, 20), (60, 0), (90, 140)], 4, dtype, seed=4,
                  absent=[(3, 0, -1), (3, 1, 10 ** 6), (5, 1, -7), (5, 8, 1 << 30)])
    out, _ = run_attention(c, [(99, 0), (99, 0)], 4, dtype, seed=1)
    assert (out == 0).all()


def test_large_scores_and_zero_queries():
    c = O.CacheDef(1, 128, 32, 128, False, "bf16")
    run_attention(c, [(40, 400), (2, 100)], 4, std=1e-9, seed=2)
    run_attention(c, [(40, 400), (2, 100)], 4, std=0.0, seed=2)
    run_attention(c, [(40, 300), (2, 90)], 4, F32, std=1e6, scale=1e-6, seed=2)
    run_attention(c, [(40, 300)], 4, BF, std=40.0, seed=2, rms=False)


@pytest.mark.parametrize("group", [128, 32])
@pytest.mark.parametrize("what", ["k", "v"])
def test_scales_of_all_sizes(group, what):
    """Scales that grow by powers of two along the sequence."""
    c = O.CacheDef(1, 128, 16, group, False, "f32")
    lens = [400]
    table, n_pages = T.make_table(c, lens, 1)
    pool = O.random_pool(c, n_pages, 1)
    for j in range(400):
        row = O.section(pool[table[0, j // 16]], c, 0, what + "_scales").reshape(16, -1)
        row[j % 16] = O.f32_to_bytes(np.full(c.ng, 2.0 ** (j / 8 - 25) * 1.37), "f32")
    q = make_q(60, 4, 128, F32, 5) * (2.0 ** -26 if what == "k" else 1.0)
    cu = np.array([0, 60], dtype=np.int32)
    ref, rlse, err = O.attention(q.double().numpy(), pool, c, table, lens, cu)
    out, lse = hr.cache_attention(q.to(DEV), gpu(pool), spec_of(c), gpu(table), ints(lens), lse=True)
    check_attention(out, lse, ref, rlse, err, q, c, 400)


@pytest.mark.parametrize("group", [64, 32])
@pytest.mark.parametrize("what", ["v", "k"])
def test_bad_scales_reach_only_those_who_see_them(group, what):
    c = O.CacheDef(2, 64, 16, group, False, "bf16")
    table, n_pages = T.make_table(c, [160], 2)
    pool = O.random_pool(c, n_pages, 2)
    q = make_q(120, 4, 64, BF, 6)
    cu = np.array([0, 120], dtype=np.int32)
    ref, _, _ = O.attention(q.double().numpy(), pool, c, table, [160], cu)
    O.section(pool[table[0, 90 // 16]], c, 1, what + "_scales").reshape(16, -1)[90 % 16] = 0xFF
    out = hr.cache_attention(q.to(DEV), gpu(pool), spec_of(c), gpu(table), ints([160]), cu_q=gpu(cu), max_q=120).cpu()
    assert torch.isnan(out[50:, 2:]).any(-1).all()
    fine = np.ones((120, 4), dtype=bool)
    fine[50:, 2:] = False
    assert not torch.isnan(out[torch.from_numpy(fine)]).any()
    g = out.double().numpy()[fine]
    assert np.linalg.norm(g - ref[fine]) / np.linalg.norm(ref[fine]) < 1.3 * 2.0 ** -9


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_in_place_and_streams(dtype):
    c = O.CacheDef(2, 128, 32, 128, False, "bf16")
    lens = [700, 90, 300]
    table, n_pages = T.make_table(c, lens, 3)
    pool, tab, n, cu = gpu(O.random_pool(c, n_pages, 3)), gpu(table), ints(lens), ints([0, 150, 160, 260])
    q = make_q(260, 8, 128, dtype, 7).to(DEV)
    want = hr.cache_attention(q, pool, spec_of(c), tab, n, cu)
    assert torch.equal(want, hr.cache_attention(q, pool, spec_of(c), tab, n, cu))
    wide = torch.zeros((260, 12, 128), dtype=dtype, device=DEV)
    wide[:, 2:10] = q
    assert torch.equal(want, hr.cache_attention(wide[:, 2:10], pool, spec_of(c), tab, n, cu))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = hr.cache_attention(q, pool, spec_of(c), tab, n, cu)
    s.synchronize()
    assert torch.equal(want, other)
    hr.cache_attention(q, pool, spec_of(c), tab, n, cu, out=q)
    assert torch.equal(want, q)
