"""Bytes, numbers and tokens at the edge of what the eviction and the latent cache
take, on the GPU against their definitions in float64 (oracle/).  Tolerances are
those of test_latent_gpu.py and test_evict_gpu.py."""
import numpy as np
import pytest
import torch

import hadamard_rotation_preprocessing_amd as hr
from oracle import cache as OC
from oracle import evict as OE
from oracle import latent as OL
from test_cache_gpu import make_q, make_table
from test_cache_gpu import spec_of as cache_spec
from test_evict_gpu import check_weights, run_evict, run_weights
from test_latent_gpu import gpu, ints, run_attention

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the gpu-marked tests need an MI355X")
    hr.lib()


# the upper halves of a NaN, both infinities, the largest numbers of both signs, -1, both zeros and a subnormal number
ODD = np.array([0x7FC0, 0x7F80, 0xFF80, 0xFF7F, 0x7F7F, 0xBF80, 0x0000, 0x8000, 0x8001], dtype=np.uint16)


def odd_bytes(n, rng, wide):
    """n scales (float32 where wide, else bfloat16) of any bits, extremes most often, as bytes."""
    v = np.where(rng.random(n) < 0.7, rng.choice(ODD, n), rng.integers(0, 1 << 16, n).astype(np.uint16)).astype(np.uint16)
    return ((v.astype(np.uint32) << 16) if wide else v).view(np.uint8)


def unseen_slots(c, table, lens, n_pages):
    """(page, slot) of positions past each length and of pages that nobody holds."""
    held = {int(table[b, j]) for b, n in enumerate(lens) for j in range(-(-n // c.page))}
    out = [(p, s) for p in range(n_pages) if p not in held for s in range(c.page)]
    return out + [(int(table[b, n // c.page]), s) for b, n in enumerate(lens) if n % c.page for s in range(n % c.page, c.page)]


# ---------------------------------------------------------------------------
# bytes that nobody sees

@pytest.mark.parametrize("d,group,sym,sdt", [(512, 128, False, "bf16"), (512, 512, True, "f32"), (512, 256, False, "bf16"),
                                             (256, 128, False, "f32"), (256, 256, True, "bf16")])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("heads", [4, 20, 48], ids=["h4", "h20", "h48"])
def test_latents_that_nobody_sees_may_be_any_bytes(d, group, sym, sdt, dtype, heads):
    c = OL.LatentDef(d, 32, group, sym, sdt)
    seqs = [(1, 1), (1, 77), (2, 130), (3, 17)]

    def odd(pool, table):
        rng = np.random.default_rng(heads)
        for p, s in unseen_slots(c, table, [n for _, n in seqs], len(pool)):
            OL.section(pool[p], c, "scales").reshape(c.page, -1)[s] = odd_bytes(c.ng, rng, sdt == "f32")
            OL.section(pool[p], c, "rope").reshape(c.page, -1)[s] = odd_bytes(c.rope, rng, False)
    run_attention(c, seqs, heads, dtype, prepare=odd, poisoned=False, seed=d + group + heads)


def test_a_later_latent_of_minus_infinity_leaves_the_tokens_before_it():
    """Of tokens in one workgroup's rows only those that see the key may be other than without it."""
    c = OL.LatentDef(512, 16, 128, False, "bf16")
    spec = hr.LatentSpec(512, 64, 16, hr.QSpec("int", 4, 128, False, "bf16"))
    pool = OL.random_pool(c, 3, 1)
    g = torch.Generator().manual_seed(1)
    q, qr = (torch.randn((6, 3, n), generator=g).to(BF).to(DEV) for n in (512, 64))
    table = ints([[2, 0, 1]])
    want = hr.latent_attention(q, qr, gpu(pool), spec, table, ints([40]), 0.07)
    OL.section(pool[1], c, "scales").reshape(16, -1)[5] = np.full(4, 0xFF80, dtype=np.uint16).view(np.uint8)   # position 37
    got = hr.latent_attention(q, qr, gpu(pool), spec, table, ints([40]), 0.07)
    assert torch.isfinite(want.float()).all() and torch.equal(got[:3], want[:3])      # tokens 34, 35, 36


@pytest.mark.parametrize("sym,sdt", [(False, "bf16"), (True, "bf16"), (True, "f32")])
@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("heads,dtype", [(1, BF), (5, BF), (40, BF), (4, F32), (20, F32)])
def test_an_infinite_latent_gives_nan_to_the_tokens_that_see_it(sym, sdt, rotate, heads, dtype):
    """Its scale is infinite and its codes are anything: no score may come out as a number
    that drops the position.  In a step that not all tokens see whole, and in one that they do."""
    spec = hr.LatentSpec(512, 64, 16, hr.QSpec("int", 4, 128, sym, sdt))
    g = torch.Generator().manual_seed(heads)
    table, lens = ints([[2, 0, 1, 3, 5, 4]]), ints([90])

    def draw(*shape):
        return torch.randn(shape, generator=g).to(dtype).to(DEV)
    c, rope, q, qr = draw(90, 512), draw(90, 64), draw(14, heads, 512), draw(14, heads, 64)
    for at, sees in ((80, 4), (10, 0)):           # the tokens are at 76 to 89
        for bad in (float("inf"), -float("inf")):
            out = []
            for x in (0.0, bad):
                pool = hr.cache_pool(spec, 6)
                v = c.clone()
                v[at, 7] = x
                hr.latent_append(pool, spec, v, rope, table, lens, rotate=rotate)
                out.append(hr.latent_attention(q, qr, pool, spec, table, lens, 0.07, rotate=rotate))
            assert torch.isfinite(out[0].float()).all() and torch.equal(out[0][:sees], out[1][:sees])
            assert torch.isnan(out[1][sees:]).all()


# ---------------------------------------------------------------------------
# tokens that are masked out

@pytest.mark.parametrize("d,group", [(64, 64), (128, 32), (256, 256)])
@pytest.mark.parametrize("new,hq,max_q", [(1, 4, 1), (5, 8, 5), (6, 8, 1), (70, 8, 70)], ids=["step", "draft", "more-than-bound", "chunk"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_tokens_without_a_log_sum_exp_add_nothing(d, group, new, hq, max_q, dtype):
    """A padded batch: tokens whose lse is -inf add nothing, whatever their queries
    are and though they see keys, and the rows beside them keep their weights."""
    c = OC.CacheDef(2, d, 16, group, False, "bf16")
    lens = [250, 97, 150]
    table, n_pages = make_table(c, lens, d)
    pool = OC.random_pool(c, n_pages, d)
    cu = np.arange(4, dtype=np.int32) * new
    q = make_q(3 * new, hq, d, dtype, d)
    _, lse, _ = OC.attention(q.double().numpy(), pool, c, table, lens, cu)
    lse = lse.astype(np.float32)
    lse[:new, 1] = -np.inf                    # one head of the first sequence's tokens, some tokens of the second, all of the third
    lse[new: 2 * new][::3] = -np.inf
    lse[2 * new:] = -np.inf
    fine = q.clone()
    out = torch.from_numpy(lse == -np.inf)
    fine[out] = 0.0
    old = np.random.default_rng(1).random((3, 2, table.shape[1] * 16)).astype(np.float32)
    ref, need = OE.weights(fine.double().numpy(), pool, c, table, lens, cu, lse, old, decay=0.5)
    odd = torch.tensor([float("nan"), float("inf"), -float("inf"), 3.0])
    q[out] = odd[torch.arange(int(out.sum()) * d) % 4].view(-1, d).to(dtype)
    for x in (q, fine):
        w = gpu(old)
        hr.cache_weights(x.to(DEV), gpu(pool), cache_spec(c), gpu(table), ints(lens), gpu(lse), w, cu_q=gpu(cu), max_q=max_q, decay=0.5)
        check_weights(w, ref, need, c, new * hq // 2)


@pytest.mark.parametrize("d,group,sym,sdt", [(64, 64, False, "bf16"), (128, 32, True, "f32"), (128, 64, False, "f32"), (256, 256, True, "bf16")])
@pytest.mark.parametrize("new,max_q", [(1, 1), (3, 3), (40, 40)], ids=["step", "draft", "chunk"])
@pytest.mark.parametrize("window", [0, 29])
def test_weights_of_keys_that_nobody_sees_may_be_any_bytes(d, group, sym, sdt, new, max_q, window):
    """Scales past each length and in pages that nobody holds, and in positions that a
    window has left (whose weights only decay)."""
    c = OC.CacheDef(2, d, 16, group, sym, sdt)
    lens, cu = [205, 77], np.array([0, new, 2 * new], dtype=np.int32)
    table, n_pages = make_table(c, lens, d)
    pool = OC.random_pool(c, n_pages, d)
    rng = np.random.default_rng(d + new)
    slots = unseen_slots(c, table, lens, n_pages)
    if window:
        slots += [(int(table[b, j // 16]), j % 16) for b, n in enumerate(lens) for j in range(max(n - new - window + 1, 0))]
    for p, s in slots:
        for h in range(2):
            OC.section(pool[p], c, h, "k_scales").reshape(16, -1)[s] = odd_bytes(c.ng, rng, sdt == "f32")
    q = make_q(2 * new, 6, d, BF, d)
    _, lse, _ = OC.attention(q.double().numpy(), pool, c, table, lens, cu, window=window)
    lse = lse.astype(np.float32)
    old = rng.random((2, 2, table.shape[1] * 16)).astype(np.float32)
    ref, need = OE.weights(q.double().numpy(), pool, c, table, lens, cu, lse, old, window=window, decay=0.9)
    assert np.isfinite(ref).all()
    w = gpu(old)
    hr.cache_weights(q.to(DEV), gpu(pool), cache_spec(c), gpu(table), ints(lens), gpu(lse), w, cu_q=gpu(cu), max_q=max_q, window=window, decay=0.9)
    check_weights(w, ref, need, c, new * 3)


# ---------------------------------------------------------------------------
# many sequences, of which few have much work

@pytest.mark.parametrize("seqs", [[(1, 20)] * 300 + [(700, 900)] + [(0, 5)] * 40, [(700, 900)] + [(1, 20 + i % 60) for i in range(400)],
                                  [(i % 2, 40) for i in range(255)] + [(600, 700), (500, 500)] + [(2, 300)] * 300],
                         ids=["in-the-second-256", "first", "around-256"])
def test_weights_shared_out_among_many_sequences(seqs):
    """A prompt's chunk among hundreds of single tokens: rows are numbered over more
    sequences than a workgroup takes at once.  (Not in whole blocks: 4 times the
    heaviest, of 24 stages of 32 rows at least, is above 5 times the mean.)"""
    blocks = [2 + -(-4 * n // 32) for n, length in seqs if n for _ in range(-(-length // 256))]
    assert 4 * max(blocks) * 512 * -(-len(blocks) // 512) > 5 * sum(blocks)
    run_weights(OC.CacheDef(1, 64, 16, 64, False, "bf16"), seqs, 4, max_q=700, seed=len(seqs))


# ---------------------------------------------------------------------------
# pages that are absent, or held twice by the same row

def test_evict_leaves_the_row_with_the_absent_page_and_cuts_the_other():
    c = OC.CacheDef(2, 64, 16, 64, False, "bf16")
    got = run_evict(c, [100, 100], 41, absent=[(0, 5, -1), (1, 6, 1 << 20)])
    assert got["lens"].tolist() == [100, 100] and got["status"][2].item() == 0
    got = run_evict(c, [100, 100], 41, absent=[(0, 5, -1)])
    assert got["lens"].tolist() == [100, 41] and got["status"][2].item() == 1
    got = run_evict(c, [100, 100], 41, absent=[(1, 0, 1 << 20)], layers=2)
    assert got["lens"].tolist() == [41, 100] and got["status"][2].item() == 1


def test_evict_of_a_page_that_a_row_holds_twice():
    """Each of its places that stays gets a page of its own, and reads what was there."""
    c = OC.CacheDef(2, 64, 16, 64, False, "bf16")
    table, _ = make_table(c, [100, 90], 0)
    twice = [(0, 1, int(table[0, 0])), (1, 5, int(table[1, 2]))]     # both places stay, and one of two
    got = run_evict(c, [100, 90], 41, 2, 4, layers=2, absent=twice, spare=6)
    assert got["lens"].tolist() == [41, 41] and got["status"][1].item() == 0
    got = run_evict(c, [100, 90], 41, 2, 4, absent=twice, spare=0)    # (the pages that left the table are free)
    assert got["lens"].tolist()[0] == 41


# ---------------------------------------------------------------------------
# queries near the end of float32

def small_keys(pool, c, heads=None):
    """Scales 2^-80 as large."""
    for p in range(len(pool)):
        for s in [OL.section(pool[p], c, "scales")] if heads is None else [OC.section(pool[p], c, h, "k_scales") for h in range(heads)]:
            s.view("<f4")[:] *= np.float32(2.0 ** -80)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d,group,heads", [(512, 128, 20), (256, 256, 4), (512, 512, 48)])
def test_latent_attention_of_the_largest_queries(dtype, d, group, heads):
    """Elements of 2^126 and more over small latents: scores of ordinary size."""
    c = OL.LatentDef(d, 16, group, False, "f32")
    run_attention(c, [(2, 100), (1, 37)], heads, dtype, rotate=False, std=2.0 ** 125, scale=2.0 ** -51, seed=d,
                  prepare=lambda pool, table: small_keys(pool, c))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 40], ids=["few", "many"])
@pytest.mark.parametrize("d,group", [(64, 64), (128, 32), (256, 128)])
def test_weights_of_the_largest_queries(dtype, new, d, group):
    c = OC.CacheDef(2, d, 16, group, False, "f32")
    lens, cu = [130, 77], np.array([0, new, 2 * new], dtype=np.int32)
    table, n_pages = make_table(c, lens, d)
    pool = OC.random_pool(c, n_pages, d)
    small_keys(pool, c, 2)
    q = make_q(2 * new, 8, d, dtype, d, std=2.0 ** 125)
    q[:, :, 0] = 1.875 * 2.0 ** 127           # (every row's largest element)
    scale = 2.0 ** -52
    _, lse, _ = OC.attention(q.double().numpy(), pool, c, table, lens, cu, scale, rotate=False)
    lse = lse.astype(np.float32)
    old = np.zeros((2, 2, table.shape[1] * 16), dtype=np.float32)
    ref, need = OE.weights(q.double().numpy(), pool, c, table, lens, cu, lse, old, scale, rotate=False)
    w = gpu(old)
    hr.cache_weights(q.to(DEV), gpu(pool), cache_spec(c), gpu(table), ints(lens), gpu(lse), w, cu_q=gpu(cu), max_q=new, scale=scale, rotate=False)
    check_weights(w, ref, need, c, new * 4)
