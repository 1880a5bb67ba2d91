"""The paged 4-bit cache on the GPU where one sequence, key or row could reach
another's result: idle sequences, scales and queries of very different sizes.
Oracle and bounds as in test_cache_gpu.py."""
import numpy as np
import pytest
import torch

import oracle
import test_cache_gpu as T
from oracle import cache as O
from test_cache_gpu import BF, F32, gpu_ready  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,group,dtype", [(64, 64, BF), (128, 128, BF), (256, 32, BF), (128, 32, F32)])
@pytest.mark.parametrize("sym", [False, True], ids=["asym", "sym"])
def test_append_idle_sequences(d, group, dtype, sym):
    """Sequences without new tokens before, between and after the others, of
    lengths that end inside a block of positions."""
    c = O.CacheDef(3, d, 16, group, sym, "bf16")
    T.run_append(c, [(0, 101), (0, 50), (3, 21), (0, 9), (5, 31), (0, 7)], dtype, seed=d)
    T.run_append(c, [(0, 1), (1, 3)], dtype, seed=d)


def test_calls_without_tokens():
    c = O.CacheDef(2, 64, 16, 64, False, "bf16")
    T.run_append(c, [(0, 33), (0, 5)])
    q = T.make_q(0, 4, 64, BF, 1).to(T.DEV)
    pool = T.gpu(O.random_pool(c, 4, 1))
    out, lse = T.hr.cache_attention(q, pool, T.spec_of(c), T.ints([[0, 1]]), T.ints([20]), cu_q=T.ints([0, 0]), lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def definition(v, c):
    """Codes, scale bytes and zero points of float32 vectors [tokens, d] by the
    definition, step for step in float32."""
    y = v.reshape(len(v), c.ng, c.group)
    with np.errstate(all="ignore"):
        if c.sym:
            lo, s = None, np.abs(y).max(-1) / np.float32(7)
        else:
            lo, hi = np.minimum(y.min(-1), np.float32(0)), np.maximum(y.max(-1), np.float32(0))
            s = (hi - lo) / np.float32(15)
        s = np.where(s == 0, np.float32(1), s).astype(np.float32)
        stored = torch.from_numpy(s) if c.sdt == "f32" else torch.from_numpy(s).to(BF)
        s = stored.float().numpy()
        q = np.rint(y / s[..., None])
        z = np.zeros(s.shape, dtype=np.float32) if c.sym else np.clip(np.rint(-lo / s), 0, 15)
        q = np.clip(q, -8, 7) if c.sym else np.clip(q + z[..., None], 0, 15)
    return q, stored, z


@pytest.mark.parametrize("sdt", ["bf16", "f32"])
@pytest.mark.parametrize("sym", [False, True], ids=["asym", "sym"])
@pytest.mark.parametrize("d,group", [(64, 64), (128, 32), (256, 256)])
def test_append_at_the_ends_of_float32(d, group, sym, sdt):
    """Vectors whose scale is subnormal, next to it, next to the largest number
    or infinite: the definition's codes; a NaN marks the scale of its group."""
    c = O.CacheDef(1, d, 16, group, sym, sdt)
    rng = np.random.default_rng(d)
    v = rng.standard_normal((48, 1, d)).astype(np.float32)
    for i, e in enumerate([-149, -146, -140, -133, -130, -128, -127, -126, -125, -120, -110, -100, -70, -66, -64, -62, -60, -30,
                           30, 60, 64, 66, 100, 120, 123, 124, 125]):
        v[i] = np.ldexp(v[i] / np.abs(v[i]).max(), e)
    v[30, 0, 3] = np.inf
    v[31, 0, d - 1] = -np.inf
    nan = [(35, 0), (36, 17), (37, d - 1), (38, d // 2 + 5), (39, d // 2 - 1)]
    for t, i in nan:
        v[t, 0, i] = np.nan
    v[40, 0, 5:9] = np.nan, np.inf, -np.inf, 1.0
    k = torch.zeros((48, 1, d)).to(T.DEV)
    pool = T.hr.cache_pool(T.spec_of(c), 3)
    T.hr.cache_append(pool, T.spec_of(c), k, torch.from_numpy(v).to(T.DEV), T.ints([[2, 0, 1]]), T.ints([48]))
    out, zeros = T.read_rows(pool.cpu().numpy(), c, np.array([[2, 0, 1]]), 0, 0, "v", 0, 48)
    q, s, z = definition(v[:, 0], c)
    want_nan = np.zeros((48, c.ng), dtype=bool)
    for t, i in nan + [(40, 5)]:
        want_nan[t, i // group] = True
    got = out["scales"].float()
    assert (torch.isnan(got).numpy() == want_nan).all()
    s = s.float().numpy()
    same = ~want_nan
    assert (got.numpy()[same] == s[same]).all()
    # codes of groups whose elements and scale are finite
    fine = same & np.isfinite(v[:, 0].reshape(48, c.ng, group)).all(-1)
    codes = oracle.unpack_nibbles(out["codes"].numpy().reshape(-1), 48 * d, sym).reshape(48, c.ng, group)
    # (a scale that bfloat16 rounds to 0 leaves 0 / 0 without a code)
    assert ((codes == q) | np.isnan(q))[fine].all(), np.argwhere(((codes != q) & ~np.isnan(q)).any(-1) & fine)
    if not sym:
        assert (zeros.reshape(48, c.ng)[fine] == z[fine]).all()


def test_a_nan_that_was_appended_is_seen():
    """A NaN in one key, or value, reaches the rows that see it and no others."""
    c = O.CacheDef(2, 128, 16, 32, False, "bf16")
    for x in range(2):
        kv = [T.make_q(40, 2, 128, BF, 3 + y, 1.0).to(T.DEV) for y in range(2)]
        kv[x][20, 1, 77] = float("nan")
        pool, table = T.hr.cache_pool(T.spec_of(c), 3), T.ints([[1, 2, 0]])
        T.hr.cache_append(pool, T.spec_of(c), *kv, table, T.ints([40]))
        out = T.hr.cache_attention(T.make_q(30, 4, 128, BF, 9).to(T.DEV), pool, T.spec_of(c), table, T.ints([40])).cpu()
        assert torch.isnan(out[10:, 2:]).any(-1).all()
        assert not torch.isnan(out[:10]).any() and not torch.isnan(out[:, :2]).any()


# ---------------------------------------------------------------------------
# attention: nothing of another row or of an unseen key in a row's result

KERNELS = ["few", "shared"]
SHAPES = [(64, 32), (128, 128), (128, 32), (256, 256), (256, 64)]


def attend(many, c, pool, table, lens, cu, q, **kw):
    """One call, by the kernel of few rows or by that of many (which a table of
    2^22 positions and a large bound of new tokens ask for)."""
    if many == "shared":
        wide = np.full((len(lens), (1 << 22) // c.page), -1, dtype=np.int32)
        wide[:, :table.shape[1]] = table
        table = wide
    return T.hr.cache_attention(q.to(T.DEV), T.gpu(pool), T.spec_of(c), T.gpu(table), T.ints(lens), cu_q=T.ints(cu),
                                max_q=1 << 20 if many == "shared" else 1, lse=True, **kw)


def row_errors(out, ref):
    """Relative error of each (token, head)."""
    g = out.detach().cpu().double().numpy()
    return np.linalg.norm(g - ref, axis=-1) / np.maximum(np.linalg.norm(ref, axis=-1), 1e-30)


# A row's error where nothing cancels: rounding the result once leaves at most
# 2^-8 / sqrt(3) in the root mean square (bfloat16, of elements at the lower end of
# their binades), times 1.3.  float32: as in test_cache_gpu.py.
ROW = {BF: 1.5 * 2.0 ** -9, F32: 2e-5}


@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("many", KERNELS)
def test_no_row_loses_a_pair_of_float16(many, d, group):
    """float32 rows, each by itself: one key whose probability, scale or query
    is a pair of float16 that do not belong together errs by 2^-11."""
    c = O.CacheDef(2, d, 16, group, False, "f32")
    lens, cu = [300, 90], np.array([0, 150, 240], dtype=np.int32)
    table, n_pages = T.make_table(c, lens, 4)
    pool = O.random_pool(c, n_pages, 4)
    q = T.make_q(240, 4, d, F32, 6)
    ref, rlse, err = O.attention(q.double().numpy(), pool, c, table, lens, cu)
    out, lse = attend(many, c, pool, table, lens, cu, q)
    T.check_attention(out, lse, ref, rlse, err, q, c, 300)
    e = row_errors(out, ref)
    T.say("  largest row error %.3g" % e.max())
    assert e.max() <= ROW[F32], np.unravel_index(e.argmax(), e.shape)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("many", KERNELS)
def test_scores_beyond_the_bits_of_float32(many, d, group, dtype):
    """Scores of 1e9 to 1e31, whose unit in the last place is large: one key
    takes a row, and the result is finite."""
    c = O.CacheDef(1, d, 16, group, False, "bf16")
    lens, cu = [150, 70], np.array([0, 40, 60], dtype=np.int32)
    table, n_pages = T.make_table(c, lens, 3)
    pool = O.random_pool(c, n_pages, 3)
    for size in (1e9, 1e20, 1e30):
        q = (size * T.make_q(60, 4, d, F32, 5)).to(dtype)
        ref, _, (mag, _) = O.attention(q.double().numpy(), pool, c, table, lens, cu)
        out, _ = attend(many, c, pool, table, lens, cu, q)
        assert torch.isfinite(out).all()
        # rows whose best key leads by more than twice what a score errs by
        y = oracle.rotate(q.double().numpy().reshape(-1, d), d, 0).reshape(60, 4, d)
        lead = np.zeros((60, 4))
        for b in range(2):
            k = np.concatenate([O.vectors(pool[p], c, 0, "k")[0] for p in table[b] if p >= 0])[: lens[b]]
            for t in range(cu[b], cu[b + 1]):
                seen = lens[b] - (cu[b + 1] - t) + 1
                s = np.sort(y[t] @ k[:seen].T / np.sqrt(d), -1)
                lead[t] = s[:, -1] - s[:, -2] if seen > 1 else np.inf
        sure = lead > 2 * (2.0 ** -21 if dtype == F32 else 2.0 ** -11) * mag + 2 * d * 2.0 ** -24 * mag
        assert sure.mean() > 0.5
        e = np.where(sure, row_errors(out, ref), 0)
        assert e.max() <= ROW[dtype], np.unravel_index(e.argmax(), e.shape)


@pytest.mark.parametrize("sdt", ["bf16", "f32"])
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("many", KERNELS)
def test_a_key_is_not_scaled_as_a_whole(many, d, group, sdt):
    """Rows that see one key: the log-sum-exp is the score.  Queries of the
    key's signs, so that nothing cancels.  A float16 operand is rounded by a unit
    in the last place / sqrt(12) in the root mean square, 2^-10 / sqrt(12) of a
    number at the lower end of its binade and less of others.  What is left of
    these errors in a score: independent ones of the queries, and of the keys one
    for every odd part of c - z (powers of two are rounded alike).  A scale that
    is rounded for a whole key, or a rounded factor of all scores, has one error
    for the score as a whole and leaves more."""
    c = O.CacheDef(2, d, 16, group, False, sdt)
    rows, hq = 96, 4
    rng = np.random.default_rng(d + group)
    table = rng.permutation(rows).astype(np.int32)[:, None]
    pool = O.random_pool(c, rows, 7)
    q = np.abs(rng.standard_normal((rows, hq, d))) + 0.2
    want, sigma = np.zeros((rows, hq)), np.zeros((rows, hq))
    for b in range(rows):
        for h in range(hq):
            k, n, _ = (x[0] for x in O.vectors(pool[table[b, 0]], c, h // 2, "k"))
            x = torch.from_numpy(q[b, h] * np.where(k < 0, -1, 1)).to(BF).double().numpy()
            q[b, h] = x
            w = np.abs(x * k)
            want[b, h] = w.sum() / np.sqrt(d)
            odd = np.abs(n).astype(int)
            while ((odd > 0) & (odd % 2 == 0)).any():
                odd = np.where((odd > 0) & (odd % 2 == 0), odd // 2, odd)
            classes = [w[g * group: (g + 1) * group][odd[g * group: (g + 1) * group] == v].sum() for g in range(c.ng) for v in range(1, 16, 2)]
            sigma[b, h] = np.sqrt((w ** 2).sum() + (np.array(classes) ** 2).sum()) / w.sum()
    out, lse = attend(many, c, pool, table, [1] * rows, np.arange(rows + 1), torch.from_numpy(q).to(BF), rotate=False)
    e = (lse.cpu().double().numpy() / want - 1) / sigma / (2.0 ** -10 / 12 ** 0.5)
    T.say("  root mean square of the errors, of its bound: %.3g; largest %.3g" % (np.sqrt((e ** 2).mean()), np.abs(e).max()))
    assert np.sqrt((e ** 2).mean()) <= 1


def check_rows(many, out, lse, ref, rlse, err, q, c, keys, rows):
    """check_attention of some (token, head) rows.  The log-sum-exp of a bfloat16
    call by the kernel of many rows is that of probabilities rounded to float16:
    2^-11 more."""
    mag, vabs = (x[rows] for x in err)
    loose = many == "shared" and q.dtype == BF
    T.check_attention(out.cpu()[rows], None if loose else lse.cpu()[rows], ref[rows], rlse[rows], (mag, vabs), q, c, keys, rms=False)
    if loose:
        e = (2.0 ** -11 + c.d * 2.0 ** -24) * mag + 2.0 ** -20 + 2.0 ** -18 * (1 + np.abs(rlse[rows])) + 2.0 ** -11
        assert (np.abs(lse.cpu().double().numpy()[rows] - rlse[rows]) <= e).all()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("many", KERNELS)
def test_rows_of_all_sizes(many, d, group, dtype):
    """Queries of sizes from 1e-30 to 1e30 in one block of rows: each is as
    precise as its own size allows."""
    c = O.CacheDef(1, d, 16, group, False, "bf16")
    lens, cu = [150, 70], np.array([0, 40, 60], dtype=np.int32)
    table, n_pages = T.make_table(c, lens, 3)
    pool = O.random_pool(c, n_pages, 3)
    rng = np.random.default_rng(d)
    for top in (100.0, 1e4, 1e7, 1e30):
        size = rng.choice([1e-4, 1e-2, 0.3, 1.0, top], (60, 4))
        size[5:9] = 1e-30
        size[9, 1] = 0.0
        q = (T.make_q(60, 4, d, F32, 5) * torch.from_numpy(size[..., None]).float()).to(dtype)
        ref, rlse, err = O.attention(q.double().numpy(), pool, c, table, lens, cu)
        out, lse = attend(many, c, pool, table, lens, cu, q)
        assert torch.isfinite(out).all()
        small = size <= 1.0
        check_rows(many, out, lse, ref, rlse, err, q, c, 150, small)
        if dtype == F32:
            assert row_errors(out, ref)[small].max() <= ROW[F32]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("many", KERNELS)
def test_rows_of_infinities(many, dtype):
    """A query with an infinity or a NaN gives NaN, and changes no other row."""
    c = O.CacheDef(1, 128, 16, 128, False, "bf16")
    lens, cu = [150], np.array([0, 60], dtype=np.int32)
    table, n_pages = T.make_table(c, lens, 3)
    pool = O.random_pool(c, n_pages, 3)
    q = T.make_q(60, 4, 128, dtype, 5)
    ref, rlse, err = O.attention(q.double().numpy(), pool, c, table, lens, cu)
    fine = np.ones((60, 4), dtype=bool)
    for t, h, x in ((3, 0, float("inf")), (17, 2, float("nan")), (40, 3, -float("inf"))):
        q[t, h, 70] = x
        fine[t, h] = False
    out, lse = attend(many, c, pool, table, lens, cu, q)
    assert torch.isnan(out.cpu()[torch.from_numpy(~fine)]).all()
    check_rows(many, out, lse, ref, rlse, err, q, c, 150, fine)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("below", [1e3, 1e5, 1e7])
@pytest.mark.parametrize("many", KERNELS)
def test_scores_far_above_the_first_ones(many, below, dtype):
    """A sequence whose first keys have scores far below all others': the result
    is that without them."""
    c = O.CacheDef(1, 128, 16, 128, True, "f32")
    lens, cu = [200], np.array([0, 60], dtype=np.int32)
    table, n_pages = T.make_table(c, lens, 3)
    pool = O.random_pool(c, n_pages, 3)
    q = T.make_q(60, 4, 128, F32, 5).abs().to(dtype)
    without = table.copy()
    without[0, :2] = -1
    ref, rlse, err = O.attention(q.double().numpy(), pool, c, without, lens, cu, rotate=False)
    for pos in range(32):                     # codes of -8: their scores are -8 s sum(q) / sqrt(128)
        O.section(pool[table[0, pos // 16]], c, 0, "k_codes").reshape(16, -1)[pos % 16] = 0x88
        row = O.section(pool[table[0, pos // 16]], c, 0, "k_scales").reshape(16, -1)
        row[pos % 16] = O.f32_to_bytes(np.full(1, below / 100, dtype=np.float32), "f32")
    out, lse = attend(many, c, pool, table, lens, cu, q, rotate=False)
    check_rows(many, out, lse, ref, rlse, err, q, c, 200, np.ones((60, 4), dtype=bool))
    if dtype == F32:
        assert row_errors(out, ref).max() <= ROW[F32]


def set_scales(pool, c, table, b, head, x, pos, values):
    """Sets the scales [ng] of one position."""
    row = O.section(pool[table[b, pos // c.page]], c, head, x + "_scales").reshape(c.page, -1)
    row[pos % c.page] = O.f32_to_bytes(np.broadcast_to(np.asarray(values, dtype=np.float32), (c.ng,)), c.sdt)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("many", KERNELS)
def test_unseen_keys_have_no_influence(many, what, d, group, dtype):
    """Scales of 1e10, 1e30, 1e-30 and infinity in keys after a row's own, before
    its window and past the length: the rows that do not see them are the same
    as without them, and as precise."""
    c = O.CacheDef(2, d, 16, group, False, "f32")
    lens, cu = [170, 70], np.array([0, 60, 130], dtype=np.int32)
    table, n_pages = T.make_table(c, lens, 3)
    plain = O.random_pool(c, n_pages, 3)
    q = T.make_q(130, 4, d, dtype, 5)
    later, before = ((0, 150), (0, 151), (0, 169), (1, 40), (1, 41), (1, 69)), ((0, 75), (0, 100), (1, 0), (1, 3))
    for window in (0, 33):
        ref, rlse, err = O.attention(q.double().numpy(), plain, c, table, lens, cu, window=window)
        for extreme in (1e4, 1e10, 1e30, 1e-30, np.inf):
            pool = plain.copy()
            unseen = np.ones((130, 4), dtype=bool)
            for b, pos in later + (before if window else ()):
                set_scales(pool, c, table, b, 1, what, pos, 2.0 ** 0.3 * extreme)
                first = lens[b] - (cu[b + 1] - cu[b])
                t = np.arange(cu[b], cu[b + 1])
                sees = (pos <= first + t - cu[b]) & ((window == 0) | (pos > first + t - cu[b] - window))
                unseen[t[sees], 2:] = False
            for pos in (170, 171, 175):
                set_scales(pool, c, table, 0, 1, what, pos, extreme)
            out, lse = attend(many, c, pool, table, lens, cu, q, window=window)
            assert unseen[:, 2:].sum() >= 40
            check_rows(many, out, lse, ref, rlse, err, q, c, 170, unseen)
            if dtype == F32:
                assert row_errors(out, ref)[unseen].max() <= ROW[F32]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("what", ["k", "v", "both"])
@pytest.mark.parametrize("many", KERNELS)
def test_scales_far_apart(many, what, d, group, dtype):
    """Neighbouring keys whose scales are up to 2^70 apart, all of them seen: a
    key of little weight takes no bits from the others."""
    c = O.CacheDef(1, d, 16, group, False, "f32")
    lens, cu = [200, 90], np.array([0, 40, 100], dtype=np.int32)
    table, n_pages = T.make_table(c, lens, 3)
    rng = np.random.default_rng(d + group)
    q = T.make_q(100, 4, d, dtype, 5)
    for spread in (8.0, 35.0):
        pool = O.random_pool(c, n_pages, 3)
        for b, n in enumerate(lens):
            for pos in range(n):
                x = 2.0 ** rng.uniform(-spread, spread, c.ng if pos % 3 else 1)
                if what != "k":
                    set_scales(pool, c, table, b, 0, "v", pos, x)
                if what != "v":
                    set_scales(pool, c, table, b, 0, "k", pos, 2.0 ** rng.uniform(-spread, 0))
        ref, rlse, err = O.attention(q.double().numpy(), pool, c, table, lens, cu)
        out, lse = attend(many, c, pool, table, lens, cu, q)
        check_rows(many, out, lse, ref, rlse, err, q, c, 200, np.ones((100, 4), dtype=bool))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("many", KERNELS)
def test_a_large_value_of_no_weight(many, dtype):
    """A value 2^40 times the others', whose probability is 2^-60 or 0: the
    others keep their bits."""
    c = O.CacheDef(1, 128, 16, 128, True, "f32")
    lens, cu = [100], np.array([0, 60], dtype=np.int32)
    table, n_pages = T.make_table(c, lens, 3)
    pool = O.random_pool(c, n_pages, 3)
    q = T.make_q(60, 2, 128, F32, 5).abs().to(dtype)
    for pos, size in ((20, 30.0), (21, 3000.0)):   # codes of -8: scores far below the others'
        O.section(pool[table[0, 1]], c, 0, "k_codes").reshape(16, -1)[pos % 16] = 0x88
        set_scales(pool, c, table, 0, 0, "k", pos, size / 128)
        set_scales(pool, c, table, 0, 0, "v", pos, 2.0 ** 40)
    ref, rlse, err = O.attention(q.double().numpy(), pool, c, table, lens, cu, rotate=False)
    out, lse = attend(many, c, pool, table, lens, cu, q, rotate=False)
    check_rows(many, out, lse, ref, rlse, err, q, c, 100, np.ones((60, 2), dtype=bool))
    if dtype == F32:
        assert row_errors(out, ref).max() <= ROW[F32]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,group", [(64, 64), (128, 32)])
@pytest.mark.parametrize("many", KERNELS)
def test_keys_set_aside_anywhere(many, d, group, dtype):
    """Extreme scales in a long sequence, whose units are cut over workgroups,
    and in many short ones, several to a workgroup; the same bits in place."""
    c = O.CacheDef(2, d, 64, group, False, "f32")
    rng = np.random.default_rng(d)
    new = rng.integers(1, 12, 90)
    lens = new + rng.integers(0, 90, 90)
    new[7], lens[7] = 9, 4000
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    table, n_pages = T.make_table(c, [int(n) for n in lens], 3)
    pool = O.random_pool(c, n_pages, 3)
    for b in rng.permutation(90)[:60].tolist() + [7] * 12:
        pos = int(rng.integers(0, lens[b]))
        set_scales(pool, c, table, b, int(rng.integers(0, 2)), "v" if rng.random() < 0.7 else "k", pos,
                   2.0 ** rng.choice([-45.0, -20.0, 24.0, 40.0]) if rng.random() < 0.8 else 0.0)
    # the same extremes everywhere in one sequence, and nothing but them
    for pos in range(lens[8]):
        set_scales(pool, c, table, 8, 0, "v", pos, 2.0 ** rng.uniform(35, 60))
        set_scales(pool, c, table, 8, 1, "v", pos, 0.0)
    q = T.make_q(int(cu[-1]), 6, d, dtype, 5)
    ref, rlse, err = O.attention(q.double().numpy(), pool, c, table, lens, cu)
    out, lse = attend(many, c, pool, table, [int(n) for n in lens], cu, q)
    check_rows(many, out, lse, ref, rlse, err, q, c, 4000, np.ones((int(cu[-1]), 6), dtype=bool))
    x = q.to(T.DEV)
    assert torch.equal(attend(many, c, pool, table, [int(n) for n in lens], cu, x, out=x)[0], out)
