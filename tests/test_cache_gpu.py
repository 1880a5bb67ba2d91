"""The paged 4-bit cache on the GPU against its definitions in float64
(oracle/cache.py) at the sizes, masks and layouts where it can go wrong.

Tolerances.  Pages that are written follow the rules of tests/parity.py for
rotate_quantize_act.  Attention's follow from its arithmetic: with u the
rounding of a float16 operand (2^-11; pairs of float16 for float32
activations: 2^-21) and S = D 2^-24 the float32 sums of a score, a score errs
by at most
    e = (u + S) scale sum_i |q_i| 15 s_i  (the codes enter unshifted, up to 15)
and the base-2 exponent's own rounding adds 2^-20; probabilities then err by a
factor exp(2 e) at most, and an output by
    (exp(2 e) - 1 + 2 u + (keys / 32 + 64) 2^-24) sum_j p_j 15 s_j  + its own rounding.
These bounds are worst cases; the root mean square over a case is also held to
what rounding the result once leaves (bf16: 2^-9 / sqrt(3) = 1.13e-3 of each
value on average over a binade's mantissas, at most 2^-9 = 1.95e-3), times 1.3.
"""
import sys

import numpy as np
import pytest
import torch

import oracle
import hadamard_rotation_preprocessing_amd as hr
from oracle import cache as O
from parity import Report, check_int

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the gpu-marked tests need an MI355X")
    hr.lib()


def spec_of(c: O.CacheDef):
    return hr.CacheSpec(c.heads, c.d, c.page, hr.QSpec("int", 4, c.group, c.sym, c.sdt))


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


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


def make_q(tokens, hq, d, dtype, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn((tokens, hq, d), generator=g)).to(dtype)


def check_attention(got, lse, ref, rlse, err, q, c, keys, rms=True):
    mag, vabs = err
    wide = q.dtype == torch.float32
    u = 2.0 ** -21 if wide else 2.0 ** -11
    e = (u + c.d * 2.0 ** -24) * mag + 2.0 ** -20
    lim = (np.expm1(2 * e) + 2 * u + (keys / 32 + 64) * 2.0 ** -24)[..., None] * vabs
    lim = lim + np.abs(ref) * (2.0 ** -23 if wide else 2.0 ** -8) + 1e-30
    g = got.detach().cpu().double().numpy()
    bad = ~(np.abs(g - ref) <= lim)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("output %s: gpu %r oracle %r, bound %r; %d of %d off" % (i, g[i], ref[i], lim[i], bad.sum(), bad.size))
    if rms and np.linalg.norm(ref) > 0:
        rel = np.linalg.norm(g - ref) / np.linalg.norm(ref)
        say("  relative error %.3g" % rel)
        assert rel <= (2e-5 if wide else 1.3 * 2.0 ** -9)
    if lse is not None:
        l = lse.detach().cpu().double().numpy()
        inf = np.isinf(rlse)
        assert (l[inf] == -np.inf).all()
        assert (np.abs(l[~inf] - rlse[~inf]) <= e[~inf] + 2.0 ** -18 * (1 + np.abs(rlse[~inf]))).all()


def run_attention(c, seqs, hq, dtype=torch.bfloat16, window=0, causal=True, rotate=True, seed=0, std=1.5, use_cu=True,
                  max_q=None, poisoned=True, absent=(), scale=None, rms=True):
    """One call against the oracle; seqs = [(new tokens, length)]."""
    say("attention", c, seqs if len(seqs) < 9 else len(seqs), "hq", hq, dtype, "window", window, "causal", causal, "rotate", rotate)
    lens = [n for _, n in seqs]
    new = [n for n, _ in seqs]
    table, n_pages = make_table(c, lens, seed)
    pool = O.random_pool(c, n_pages, seed)
    if poisoned:  # positions past each length, pages nobody holds
        held = set()
        for b, n in enumerate(lens):
            for j in range(-(-n // c.page)):
                held.add(int(table[b, j]))
                for s in range(c.page):
                    if j * c.page + s >= n:
                        O.poison(pool, c, int(table[b, j]), s)
        for p in set(range(n_pages)) - held:
            for s in range(c.page):
                O.poison(pool, c, p, s)
    for b, j, v in absent:
        table[b, j] = v
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = make_q(int(cu[-1]), hq, c.d, dtype, seed)
    q = (q * (std / 1.5)).to(dtype)
    ref, rlse, err = O.attention(q.double().numpy(), pool, c, table, lens, cu, scale, causal, window, rotate)
    out, lse = hr.cache_attention(q.to(DEV), gpu(pool), spec_of(c), gpu(table), ints(lens), cu_q=gpu(cu) if use_cu else None,
                                  max_q=max(new) if max_q is None else max_q, scale=scale, causal=causal, window=window,
                                  rotate=rotate, lse=True)
    torch.cuda.synchronize()
    check_attention(out, lse, ref, rlse, err, q, c, max(lens), rms)
    return out, ref


BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("d,group", [(64, 64), (64, 32), (128, 128), (128, 64), (128, 32), (256, 256), (256, 128), (256, 64), (256, 32)])
@pytest.mark.parametrize("sym", [False, True], ids=["asym", "sym"])
@pytest.mark.parametrize("sdt", ["bf16", "f32"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_attention_formats(d, group, sym, sdt, dtype):
    """Every head dimension, group size, symmetry and type; lengths that end
    inside a page, a 16-key tile and a 32-key step, and one-token caches."""
    c = O.CacheDef(2, d, 32, group, sym, sdt)
    run_attention(c, [(1, 1), (1, 77), (2, 130), (3, 16), (1, 160)], 6, dtype, seed=d + group)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("rep", [1, 4, 7, 16])
def test_attention_pages_and_heads(page, rep):
    c = O.CacheDef(2, 128, page, 128, False, "bf16")
    run_attention(c, [(1, 300), (1, 15), (4, 65), (1, 16), (2, 511)], 2 * rep, seed=page + rep)


@pytest.mark.parametrize("d,dtype", [(64, BF), (128, BF), (256, BF), (64, F32), (128, F32), (256, F32)])
@pytest.mark.parametrize("new,length,rep", [(17, 17, 1), (33, 200, 2), (100, 100, 1), (50, 333, 3), (5, 5, 7)])
def test_attention_prompts(d, dtype, new, length, rep):
    """Many rows: the kernels with row blocks, from the first token and behind
    a prefix, at odd sizes."""
    c = O.CacheDef(1, d, 16, d, False, "bf16")
    run_attention(c, [(new, length), (1, 40), (new // 2, length)], rep, dtype, seed=new)


@pytest.mark.parametrize("group", [128, 32])
def test_attention_whole_units(group):
    """Enough rows that every workgroup has a unit of its own, ragged."""
    c = O.CacheDef(32, 128, 64, group, False, "bf16")
    run_attention(c, [(350, 350), (1, 90), (0, 30), (260, 300), (500, 500), (130, 131), (77, 200)], 32 * 4, seed=3)


@pytest.mark.parametrize("window", [1, 5, 16, 33, 100, 5000])
@pytest.mark.parametrize("new", [1, 20])
def test_attention_window(window, new):
    c = O.CacheDef(2, 128, 16, 128, False, "bf16")
    run_attention(c, [(new, 200), (new, 32), (new, max(new, 1)), (1, 97)], 4, window=window, seed=window)


def test_attention_not_causal():
    c = O.CacheDef(2, 128, 32, 128, True, "bf16")
    run_attention(c, [(9, 70), (3, 1), (40, 33)], 4, causal=False, seed=8)


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_rotation_and_scale(rotate, dtype):
    c = O.CacheDef(2, 128, 64, 64, False, "f32")
    run_attention(c, [(1, 500), (2, 64)], 4, dtype, rotate=rotate, scale=0.25, seed=5)


def test_attention_rows_that_see_nothing():
    """Empty sequences, rows without new tokens, more new tokens than
    positions, absent pages: zeros and -inf, whatever the bytes are."""
    c = O.CacheDef(2, 64, 16, 64, False, "bf16")
    run_attention(c, [(1, 0), (0, 50), (5, 3), (1, 20), (2, 0), (3, 40)], 4, seed=4,
                  absent=[(3, 0, -1), (3, 1, 10 ** 6), (5, 1, -7)])
    run_attention(c, [(40, 8), (30, 0), (1, 1)], 4, seed=4)  # the kernels with row blocks
    out, _ = run_attention(c, [(1, 0), (1, 0)], 2, seed=1)
    assert (out == 0).all()


@pytest.mark.parametrize("max_q", [0, 1, 2, 1000])
def test_attention_max_q_is_only_a_hint(max_q):
    c = O.CacheDef(2, 128, 32, 128, False, "bf16")
    run_attention(c, [(3, 90), (40, 64), (1, 200)], 8, max_q=max_q, seed=9)


def test_attention_uniform_rows_without_cu():
    c = O.CacheDef(2, 128, 32, 128, False, "bf16")
    run_attention(c, [(3, 90), (3, 3), (3, 200)], 8, use_cu=False, seed=9)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_many_ragged_sequences(dtype):
    """More sequences than a workgroup has threads, most of them short."""
    c = O.CacheDef(1, 64, 16, 64, False, "bf16")
    rng = np.random.default_rng(12)
    seqs = [(int(rng.integers(0, 3)), int(rng.integers(0, 50))) for _ in range(600)]
    seqs[37], seqs[599] = (2, 1500), (1, 3000)
    run_attention(c, seqs, 2, dtype, seed=6)


def test_attention_large_scores_and_zero_queries():
    """Queries far outside float16's range, queries of zeros, and score spreads
    that leave one key: the running maximum moves in every step."""
    c = O.CacheDef(1, 128, 32, 128, False, "bf16")
    run_attention(c, [(1, 400), (2, 100)], 4, std=1e-9, seed=2)
    run_attention(c, [(1, 400), (2, 100)], 4, std=0.0, seed=2)
    run_attention(c, [(1, 300), (2, 90)], 4, F32, std=1e6, scale=1e-6, seed=2)
    run_attention(c, [(1, 300)], 4, BF, std=40.0, seed=2, rms=False)


def test_attention_value_scales_of_all_sizes():
    """Value scales that grow by powers of two along the sequence."""
    for group in (128, 32):
        c = O.CacheDef(1, 128, 16, group, False, "f32")
        run_attention(c, [(1, 600), (2, 333)], 4, F32, seed=3)
        lens = [200]
        table, n_pages = make_table(c, lens, 1)
        pool = O.random_pool(c, n_pages, 1)
        for j in range(200):
            row = O.section(pool[table[0, j // 16]], c, 0, "v_scales").reshape(16, -1)
            row[j % 16] = O.f32_to_bytes(np.full(c.ng, 2.0 ** (j / 4 - 30) * 1.37), "f32")
        q = make_q(1, 4, 128, F32, 5)
        cu = np.array([0, 1], dtype=np.int32)
        ref, rlse, err = O.attention(q.double().numpy(), pool, c, table, lens, cu)
        out, lse = hr.cache_attention(q.to(DEV), gpu(pool), spec_of(c), gpu(table), ints(lens), lse=True)
        check_attention(out, lse, ref, rlse, err, q, c, 200)


@pytest.mark.parametrize("group", [64, 32])
@pytest.mark.parametrize("what", ["v", "k"])
def test_attention_bad_scales_reach_only_those_who_see_them(group, what):
    """A NaN scale at a visible position makes the rows that see it NaN and
    leaves earlier rows (causal) and other heads alone."""
    c = O.CacheDef(2, 64, 16, group, False, "bf16")
    table, n_pages = make_table(c, [60], 2)
    pool = O.random_pool(c, n_pages, 2)
    q = make_q(20, 4, 64, BF, 6)
    cu = np.array([0, 20], dtype=np.int32)
    ref, rlse, err = O.attention(q.double().numpy(), pool, c, table, [60], cu)
    j = 50
    O.section(pool[table[0, j // 16]], c, 1, what + "_scales").reshape(16, -1)[j % 16] = 0xFF
    for new in (20,):
        out, lse = hr.cache_attention(q.to(DEV), gpu(pool), spec_of(c), gpu(table), ints([60]), cu_q=gpu(cu), max_q=new, lse=True)
        out, lse = out.cpu(), lse.cpu()
        blind = 50 - 40
        assert torch.isnan(out[blind:, 2:]).any(-1).all()
        fine = np.ones((20, 4), dtype=bool)
        fine[blind:, 2:] = False
        assert not torch.isnan(out[torch.from_numpy(fine)]).any()
        g = out.double().numpy()[fine]
        assert np.linalg.norm(g - ref[fine]) / np.linalg.norm(ref[fine]) < 1.3 * 2.0 ** -9


def test_attention_strides_in_place_and_streams():
    """q as a slice of a wider projection, out in place, another stream than
    the default one: the same bits as the plain call; twice the same bits."""
    c = O.CacheDef(2, 128, 32, 128, False, "bf16")
    table, n_pages = make_table(c, [700, 90, 300], 3)
    pool, tab, lens = gpu(O.random_pool(c, n_pages, 3)), gpu(table), ints([700, 90, 300])
    q = make_q(6, 8, 128, BF, 7).to(DEV)
    want = hr.cache_attention(q, pool, spec_of(c), tab, lens)
    assert torch.equal(want, hr.cache_attention(q, pool, spec_of(c), tab, lens))
    wide = torch.zeros((6, 12, 128), dtype=BF, device=DEV)
    wide[:, 2:10] = q
    assert torch.equal(want, hr.cache_attention(wide[:, 2:10], pool, spec_of(c), tab, lens))
    by_head = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(want, hr.cache_attention(by_head, pool, spec_of(c), tab, lens, out=torch.empty_like(by_head)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = hr.cache_attention(q, pool, spec_of(c), tab, lens)
    s.synchronize()
    assert torch.equal(want, other)
    hr.cache_attention(q, pool, spec_of(c), tab, lens, out=q)
    assert torch.equal(want, q)


def test_attention_long_cache_beyond_32_bits():
    """A pool of more than 2^32 bytes: the pages that count lie at its end."""
    c = O.CacheDef(8, 128, 256, 128, False, "bf16")
    spec = spec_of(c)
    n_pages = (1 << 32) // spec.page_bytes + 9
    pool = torch.zeros((n_pages, spec.page_bytes), dtype=torch.uint8, device=DEV)
    small = O.random_pool(c, 3, 11)
    pool[-3:] = gpu(small)
    q = make_q(1, 8, 128, BF, 3)
    cu = np.array([0, 1], dtype=np.int32)
    ref, rlse, err = O.attention(q.double().numpy(), small, c, [[0, 1, 2]], [700], cu)
    table = ints([[n_pages - 3, n_pages - 2, n_pages - 1]])
    out, lse = hr.cache_attention(q.to(DEV), pool, spec, table, ints([700]), lse=True)
    check_attention(out, lse, ref, rlse, err, q, c, 700)
    # and appends there
    before = pool[-2:].clone()
    k = torch.ones((1, 8, 128), dtype=BF, device=DEV)
    hr.cache_append(pool, spec, k, k, ints([[n_pages - 1, n_pages - 2]]), ints([257]))
    assert not torch.equal(pool[-2], before[0]) and torch.equal(pool[-1], before[1])


# ---------------------------------------------------------------------------
# append

def read_rows(pool, c, table, b, head, x, lo, hi):
    """The framework's quantized tensors of positions [lo, hi) of one head."""
    codes, scales, zeros = [], [], []
    for p in range(lo, hi):
        row, s = pool[table[b, p // c.page]], p % c.page
        codes.append(O.section(row, c, head, x + "_codes").reshape(c.page, -1)[s])
        scales.append(O.section(row, c, head, x + "_scales").reshape(c.page, -1)[s])
        if not c.sym:
            zeros.append(oracle.unpack_nibbles(O.section(row, c, head, x + "_zeros"), c.page * c.ng).reshape(c.page, c.ng)[s])
    s = O.bytes_to_f64(np.stack(scales), c.sdt)
    out = {"codes": torch.from_numpy(np.stack(codes)), "scales": torch.from_numpy(s), "zeros": None}
    return out, (np.stack(zeros) if zeros else None)


def run_append(c, seqs, dtype=BF, rotate=True, seed=0, use_cu=True, std=1.0):
    say("append", c, seqs if len(seqs) < 9 else len(seqs), dtype, "rotate", rotate)
    lens, new = [n for _, n in seqs], [n for n, _ in seqs]
    table, n_pages = make_table(c, lens, seed)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    t = int(cu[-1])
    rng = np.random.default_rng(seed)
    k = torch.from_numpy(rng.standard_normal((t, c.heads, c.d), dtype=np.float32) * np.float32(std)).to(dtype)
    v = torch.from_numpy(rng.standard_t(3, (t, c.heads, c.d)).astype(np.float32) * np.float32(std)).to(dtype)
    before = rng.integers(0, 256, (n_pages, c.page_bytes), dtype=np.uint8)
    pool = gpu(before.copy())
    hr.cache_append(pool, spec_of(c), k.to(DEV), v.to(DEV), gpu(table), ints(lens), cu_q=gpu(cu) if use_cu else None, rotate=rotate)
    after = pool.cpu().numpy()
    touched = np.zeros(after.shape, dtype=bool)   # whole bytes that belong to new positions
    shared = np.zeros(after.shape, dtype=np.uint8)  # bits of them in shared bytes
    rep = Report()
    for b, (n, length) in enumerate(seqs):
        lo = max(length - n, 0)
        skip = max(n - length, 0)
        for h in range(c.heads):
            for x, src in (("k", k), ("v", v)):
                if length == lo:
                    continue
                y = src[cu[b] + skip: cu[b + 1], h].double().numpy()
                if x == "k" and rotate:
                    y = oracle.rotate(y, c.d, 0)
                out, zeros = read_rows(after, c, table, b, h, x, lo, length)
                check_int(out, y, c.group, c.sym, c.sdt, rep, zeros_gpu=zeros)
                for p in range(lo, length):
                    row, s = table[b, p // c.page], p % c.page
                    for name, width in (("codes", None), ("scales", None)):
                        O.section(touched[row], c, h, "%s_%s" % (x, name)).reshape(c.page, -1)[s] = True
                    if not c.sym:
                        z = O.section(shared[row], c, h, x + "_zeros")
                        for i in range(s * c.ng, (s + 1) * c.ng):
                            z[i // 2] |= 0xF0 if i & 1 else 0x0F
    assert ((after == before) | touched | (shared > 0)).all(), "bytes of other positions changed"
    keep = ~shared
    assert ((after & keep) == (before & keep))[~touched].all(), "another position's zero point changed"
    return pool


@pytest.mark.parametrize("d,group", [(64, 64), (64, 32), (128, 128), (128, 64), (128, 32), (256, 256), (256, 128), (256, 64), (256, 32)])
@pytest.mark.parametrize("sym", [False, True], ids=["asym", "sym"])
@pytest.mark.parametrize("sdt,dtype", [("bf16", BF), ("f32", BF), ("bf16", F32), ("f32", F32)])
def test_append_formats(d, group, sym, sdt, dtype):
    c = O.CacheDef(3, d, 16, group, sym, sdt)
    run_append(c, [(1, 1), (5, 22), (0, 9), (33, 33), (1, 16), (2, 19)], dtype, seed=d + group)


@pytest.mark.parametrize("heads,page", [(1, 16), (5, 32), (8, 64), (2, 256)])
@pytest.mark.parametrize("rotate", [False, True])
def test_append_heads_pages(heads, page, rotate):
    c = O.CacheDef(heads, 128, page, 128, False, "bf16")
    run_append(c, [(1, 100), (70, 70), (3, 3), (9, 300)], rotate=rotate, seed=heads)


def test_append_uniform_and_clamped():
    c = O.CacheDef(2, 128, 16, 128, False, "bf16")
    run_append(c, [(2, 7), (2, 2), (2, 33)], use_cu=False)
    run_append(c, [(6, 4), (3, 0), (1, 5)])          # more new tokens than positions: the last ones
    run_append(c, [(7, 31)], std=1e-20, dtype=F32)
    run_append(c, [(7, 31)], std=0.0)


def test_append_matches_the_contiguous_quantizer():
    """The same codes, scales and zero points as rotate_quantize_act writes for
    the same rows, but for its scale (range times 1 / 15, an ulp of float32)."""
    c = O.CacheDef(2, 128, 64, 128, False, "bf16")
    k = make_q(64, 2, 128, BF, 1, 1.0).to(DEV)
    pool = hr.cache_pool(spec_of(c), 1)
    hr.cache_append(pool, spec_of(c), k, k, ints([[0]]), ints([64]))
    sec = hr.cache_sections(pool, spec_of(c))
    for h in range(2):
        for x, block in (("k", 0), ("v", 1)):
            want = hr.rotate_quantize_act(k[:, h].contiguous(), block, hr.QSpec("int", 4, 128, False, "bf16"))
            same = (sec[x + "_codes"][0, h].reshape(64, 64) == want["codes"]).float().mean().item()
            assert same > 0.999
            got = {"codes": sec[x + "_codes"][0, h].contiguous(), "zeros": sec[x + "_zeros"][0, h].contiguous(),
                   "scales": sec[x + "_scales"][0, h].contiguous().view(torch.bfloat16)}
            y = oracle.rotate(k[:, h].double().cpu().numpy(), 128, block)
            deq, st = hr.dequant_check(got, hr.QSpec("int", 4, 128, False, "bf16"), 64, 128, ref=torch.from_numpy(y).float().to(DEV))
            assert st["max_err_steps"] < 1.1 and abs(deq.double().cpu().numpy() - y).max() < 0.5


def test_append_strides():
    c = O.CacheDef(2, 64, 16, 64, False, "bf16")
    spec = spec_of(c)
    qkv = make_q(30, 8, 64, BF, 4, 1.0).to(DEV)
    table, lens = ints([[1, 0]]), ints([30])
    a, b = hr.cache_pool(spec, 2), hr.cache_pool(spec, 2)
    hr.cache_append(a, spec, qkv[:, 4:6], qkv[:, 6:8], table, lens)
    hr.cache_append(b, spec, qkv[:, 4:6].contiguous(), qkv[:, 6:8].contiguous(), table, lens)
    assert torch.equal(a, b) and a.any()


def test_append_absent_pages_and_token_by_token():
    c = O.CacheDef(2, 128, 16, 128, False, "bf16")
    spec = spec_of(c)
    k, v = (make_q(40, 2, 128, BF, s, 1.0).to(DEV) for s in (1, 2))
    whole, one = hr.cache_pool(spec, 3), hr.cache_pool(spec, 3)
    table = ints([[2, 0, 1]])
    hr.cache_append(whole, spec, k, v, table, ints([40]))
    for i in range(40):
        hr.cache_append(one, spec, k[i: i + 1], v[i: i + 1], table, ints([i + 1]))
    assert torch.equal(whole, one)
    gap = hr.cache_pool(spec, 3)
    hr.cache_append(gap, spec, k, v, ints([[2, -1, 99]]), ints([40]))
    assert torch.equal(gap[2], whole[2]) and not gap[:2].any()


# ---------------------------------------------------------------------------
# pages

def random_state(rows, n_pages, max_pages, page, seed, share=True):
    rng = np.random.default_rng(seed)
    ids = list(rng.permutation(n_pages))
    table = np.full((rows, max_pages), -1, dtype=np.int32)
    lens = np.zeros(rows, dtype=np.int32)
    for i in range(rows):
        k = int(rng.integers(0, max_pages + 1))
        k = min(k, max(0, len(ids) - n_pages // 4))
        own = [ids.pop() for _ in range(k)]
        if share and i % 3 == 1:
            m = int(min(k, lens[i - 1] // page))
            ids += own[:m]
            own[:m] = [int(x) for x in table[i - 1, :m]]
        table[i, :k] = own
        lens[i] = 0 if k == 0 else (k - 1) * page + int(rng.integers(1, page + 1))
    return table, lens


def run_update(rows, new_rows, n_pages, max_pages, page, layers, seed, grow_to=40, state=None, parents=None, grow=None):
    say("update", rows, new_rows, n_pages, max_pages, page, layers, seed)
    c = O.CacheDef(1, 64, page, 64, False, "bf16")
    rng = np.random.default_rng(seed + 1)
    table, lens = random_state(rows, n_pages, max_pages, page, seed) if state is None else state
    if parents is None:
        parents = rng.integers(-1, rows + 1, new_rows)
    if grow is None:
        grow = rng.integers(-grow_to // 2, grow_to, new_rows)
        grow[rng.random(new_rows) < 0.2] = 0
    nt, nl, refs, status, copies = O.update(page, max_pages, n_pages, table, lens, parents, grow)
    before = rng.integers(0, 256, (layers, n_pages, c.page_bytes), dtype=np.uint8)
    pool = gpu(before.copy())
    out = hr.cache_update(pool, spec_of(c), gpu(table), ints(lens), ints(parents), ints(grow))
    for s, t in copies:
        before[:, t] = before[:, s]
    assert out["table"].cpu().numpy().tolist() == nt.tolist()
    assert out["lens"].cpu().numpy().tolist() == nl.tolist()
    assert out["refs"].cpu().numpy().tolist() == refs.tolist()
    assert out["status"].cpu().tolist() == status
    assert (pool.cpu().numpy() == before).all()
    return nt, nl


@pytest.mark.parametrize("rows,new_rows,n_pages,max_pages,page,layers", [
    (1, 1, 4, 2, 16, 1), (5, 8, 40, 6, 16, 2), (30, 20, 100, 7, 32, 1), (64, 64, 500, 9, 16, 3), (3, 700, 900, 5, 16, 1),
    (700, 40, 3000, 5, 16, 1), (300, 1500, 9000, 8, 16, 1), (20, 20, 33, 6, 16, 1), (40, 1100, 12288, 30, 16, 1),
    (40, 1100, 13001, 30, 16, 1)])
def test_update(rows, new_rows, n_pages, max_pages, page, layers):
    for seed in range(3):
        run_update(rows, new_rows, n_pages, max_pages, page, layers, seed)


def test_update_forks_of_one_row():
    """Forks of a partly filled page: all grow, some do not, cut into the middle
    of a full page, and a row of no parent."""
    table = np.array([[5, 2, -1, -1], [5, 7, -1, -1]], dtype=np.int32)
    lens = np.array([20, 16], dtype=np.int32)
    state = (table, lens)
    run_update(2, 3, 10, 4, 16, 2, 0, state=state, parents=np.array([0, 0, 0]), grow=np.array([1, 1, 30]))
    run_update(2, 3, 10, 4, 16, 2, 0, state=state, parents=np.array([0, 0, 0]), grow=np.array([1, 0, 1]))
    run_update(2, 3, 10, 4, 16, 2, 0, state=state, parents=np.array([0, 1, 0]), grow=np.array([-10, 5, 100]))
    run_update(2, 2, 10, 4, 16, 2, 0, state=state, parents=np.array([-1, 9]), grow=np.array([70, -3]))
    run_update(2, 2, 3, 4, 16, 2, 0, state=(np.array([[0, 2, -1, -1], [0, 1, -1, -1]], dtype=np.int32), lens),
               parents=np.array([0, 0]), grow=np.array([40, 3]))   # the pool runs out
    run_update(2, 0, 10, 4, 16, 1, 0, state=state, parents=np.array([], dtype=int), grow=np.array([], dtype=int))


def run_compact(rows, n_pages, max_pages, page, layers, seed, into=None):
    say("compact", rows, n_pages, max_pages, page, layers, "into", into)
    c = O.CacheDef(1, 64, page, 64, True, "bf16")
    rng = np.random.default_rng(seed)
    table, lens = random_state(rows, n_pages, max_pages, page, seed)
    nt, refs, status, moves = O.compact(page, max_pages, n_pages, table, lens, into)
    before = rng.integers(0, 256, (layers, n_pages, c.page_bytes), dtype=np.uint8)
    pool = gpu(before.copy())
    dst = None if into is None else torch.zeros((layers, into, c.page_bytes), dtype=torch.uint8, device=DEV)
    out = hr.cache_compact(pool, spec_of(c), gpu(table), ints(lens), into=dst)
    want = before.copy() if into is None else np.zeros((layers, into, c.page_bytes), dtype=np.uint8)
    for s, t in moves:
        want[:, t] = before[:, s]
    assert out["table"].cpu().numpy().tolist() == nt.tolist()
    assert out["refs"].cpu().numpy().tolist() == refs.tolist()
    assert out["status"].cpu().tolist() == status
    assert ((pool if dst is None else dst).cpu().numpy() == want).all()
    if dst is not None:
        assert (pool.cpu().numpy() == before).all()


@pytest.mark.parametrize("into", [None, 1, 17, 4000])
@pytest.mark.parametrize("rows,n_pages,max_pages,layers", [(1, 1, 1, 1), (4, 30, 5, 2), (50, 400, 9, 1), (600, 5000, 7, 2), (3, 9000, 4, 1),
                                                           (300, 12288, 30, 1), (300, 12290, 30, 1)])
def test_compact(rows, n_pages, max_pages, layers, into):
    for seed in range(2):
        run_compact(rows, n_pages, max_pages, 16, layers, seed, into)


# ---------------------------------------------------------------------------
# the path together

def test_decode_loop_equals_prefill_and_survives_forks():
    """Two sequences are filled, forked, grown token by token and compacted;
    attention over the cache equals that over one filled in a single call, and a
    captured graph of a decoding step replays to the eager result."""
    spec = hr.CacheSpec(2, 128, 16, hr.QSpec("int", 4, 128, False, "bf16"))
    dev = dict(device=DEV)
    layers, n_pages, width = 2, 40, 6
    pool = hr.cache_pool(spec, n_pages, layers)
    k, v, q = (make_q(80, h, 128, BF, s, 1.0).to(DEV) for s, h in ((1, 2), (2, 2), (3, 8)))
    empty = (torch.full((2, width), -1, dtype=torch.int32, **dev), torch.zeros(2, dtype=torch.int32, **dev))
    st = hr.cache_update(pool, spec, *empty, ints([-1, -1]), ints([20, 37]))
    cu = ints([0, 20, 57])
    for l in range(layers):
        hr.cache_append(pool[l], spec, k[:57], v[:57], st["table"], st["lens"], cu_q=cu)
    st = hr.cache_update(pool, spec, st["table"], st["lens"], ints([0, 1, 0]), ints([1, 1, 1]))
    assert st["status"].tolist()[2] == 1   # the partly filled page of row 0 was copied
    for l in range(layers):
        hr.cache_append(pool[l], spec, k[57:60], v[57:60], st["table"], st["lens"])
    cp = hr.cache_compact(pool, spec, st["table"], st["lens"])
    st["table"] = cp["table"]
    got = hr.cache_attention(q[:3], pool[1], spec, st["table"], st["lens"])
    # the three sequences from scratch
    idx = [list(range(20)) + [57], list(range(20, 57)) + [58], list(range(20)) + [59]]
    flat = torch.tensor(sum(idx, []), **dev)
    ref_pool = hr.cache_pool(spec, 20)
    st2 = hr.cache_update(ref_pool, spec, *empty, ints([-1, -1, -1]), ints([21, 38, 21]))
    hr.cache_append(ref_pool, spec, k[flat], v[flat], st2["table"], st2["lens"], cu_q=ints([0, 21, 59, 80]))
    want = hr.cache_attention(q[:3], ref_pool, spec, st2["table"], st2["lens"])
    assert torch.equal(got, want)
    # a decoding step in a graph
    s = torch.cuda.Stream()
    kk, vv, qq = k[60:63].clone(), v[60:63].clone(), q[60:63].clone()
    work = torch.empty(max(hr.cache_attention_work(BF, 3, 8, spec, 3, 1), 16), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(qq)
    upd = hr.cache_update(pool, spec, st["table"], st["lens"], ints([0, 1, 2]), ints([1, 1, 1]))
    uw = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    par, gr = ints([0, 1, 2]), ints([1, 1, 1])

    def one():
        hr.cache_update(pool, spec, st["table"], st["lens"], par, gr, out=upd, work=uw)
        hr.cache_append(pool[1], spec, kk, vv, upd["table"], upd["lens"])
        hr.cache_attention(qq, pool[1], spec, upd["table"], upd["lens"], max_q=1, out=out, work=work)

    one()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        one()
    for i in range(4):
        kk.copy_(k[60 + i: 63 + i])
        qq.copy_(q[60 + i: 63 + i])
        one()
        torch.cuda.synchronize()
        want = out.clone()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and out.any()
