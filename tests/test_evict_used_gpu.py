"""Eviction as it is used: kernels chosen by a bound that does not hold, captured
steps, streams, and append, attention, weights, eviction and attention over what
is left, against their definitions in float64 (oracle/)."""
import math
import os
import sys

import numpy as np
import pytest
import torch

import hadamard_rotation_preprocessing_amd as hr
from oracle import cache as O
from test_cache_gpu import gpu, ints, make_q, make_table, spec_of
from test_evict_gpu import BF, DEV, F32, run_weights, say

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def gpu_ready():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: the gpu-marked tests need an MI355X")
    hr.lib()


@pytest.mark.parametrize("max_q", [1, 3, 5, 1 << 40])
@pytest.mark.parametrize("kw", [dict(), dict(window=9), dict(causal=False)], ids=["causal", "window", "full"])
def test_weights_with_any_bound(max_q, kw):
    """max_q chooses the kernel, and no result: rows of 8 and 32, more than a pass
    takes, and none."""
    run_weights(O.CacheDef(2, 64, 16, 32, False, "bf16"), [(40, 200), (1, 130), (0, 9), (7, 7), (9, 5)], 16, max_q=max_q, seed=3, **kw)


@pytest.mark.parametrize("d,group", [(64, 64), (128, 128), (128, 32), (256, 64)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_weights_of_single_tokens(d, group, dtype):
    """One and two tiles of rows, odd lengths, symmetric and not."""
    seqs = [(1, 1), (1, 63), (1, 64), (1, 65), (1, 1000), (1, 17)]
    run_weights(O.CacheDef(2, d, 32, group, False, "bf16"), seqs, 14, dtype=dtype, max_q=1, seed=d, absent=[(4, 3, -1)])
    run_weights(O.CacheDef(1, d, 64, group, True, "f32"), seqs, 24, dtype=dtype, max_q=1, seed=d + 1)


def test_weights_of_many_short_rows():
    rng = np.random.default_rng(5)
    run_weights(O.CacheDef(1, 64, 16, 64, False, "bf16"), [(1, int(n)) for n in rng.integers(1, 90, 600)], 4, max_q=1, seed=7)


def setup(layers=2, spare=30):
    c = O.CacheDef(2, 64, 16, 64, False, "bf16")
    lens = [150, 33, 90]
    table, n_pages = make_table(c, lens, 11, max_pages=12, spare=spare)
    pool = gpu(np.stack([O.random_pool(c, n_pages, 11 + i) for i in range(layers)]))
    return c, spec_of(c), pool, gpu(table), ints(lens)


def test_a_captured_step_with_eviction_replays():
    """Attention, its weights and an eviction in one graph, over lengths that change,
    against the same calls made one by one, with eager work between the replays."""
    c, spec, pool, table, lens = setup()
    q = torch.randn((3, 8, 64), device=DEV).bfloat16()
    w = torch.rand((2, 3, 2, 12 * 16 + 3), device=DEV)
    fixed = dict(table=torch.empty_like(table), lens=torch.empty_like(lens), refs=ints([0] * pool.shape[1]), status=ints([0] * 4))

    def step(pool, w, out):
        o, lse = hr.cache_attention(q, pool[1], spec, table, lens, max_q=1, lse=True)
        hr.cache_weights(q, pool[1], spec, table, lens, lse, w[1], max_q=1, decay=0.5)
        return o, hr.cache_evict(pool, spec, table, lens, w, 40, 2, 8, out=out)
    step(pool.clone(), w.clone(), None)          # (once outside the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, got = step(pool, w, fixed)
    for k in range(5):
        q.copy_(torch.randn((3, 8, 64), device=DEV))
        pool.random_(0, 60)
        w.uniform_()
        lens.copy_(ints([150 - 20 * k, 33 + 9 * k, 90]))
        other_pool, other_w = pool.clone(), w.clone()
        graph.replay()
        want, eager = step(other_pool, other_w, None)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(pool, other_pool) and torch.equal(w, other_w)
        assert all(torch.equal(got[n], eager[n]) for n in eager)


def test_streams_and_scratch_of_the_caller():
    c, spec, pool, table, lens = setup()
    q = torch.randn((3, 8, 64), device=DEV).bfloat16()
    _, lse = hr.cache_attention(q, pool[0], spec, table, lens, lse=True)
    w0 = torch.rand((2, 3, 2, 192), device=DEV)
    want = hr.cache_weights(q, pool[0], spec, table, lens, lse, w0[0].clone())
    wp, ww = pool.clone(), w0.clone()
    cut = hr.cache_evict(wp, spec, table, lens, ww, 50, 1, 3)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            work = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
            a = hr.cache_weights(q, pool[0], spec, table, lens, lse, w0[0].clone(), work=work)
            p, x = pool.clone(), w0.clone()
            got.append((a, p, x, hr.cache_evict(p, spec, table, lens, x, 50, 1, 3, work=work)))
    torch.cuda.synchronize()
    for a, p, x, r in got:
        assert torch.equal(a, want) and torch.equal(p, wp) and torch.equal(x, ww)
        assert all(torch.equal(r[n], cut[n]) for n in cut)
    with pytest.raises(hr.HadarotError, match="work_bytes"):
        hr.cache_evict(pool, spec, table, lens, w0, 50, work=torch.empty(64, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("share", [False, True])
def test_decoding_with_a_budget(share):
    """Two steps of two rows (one, or both over the pages of the same prompt): what is
    attended to after an eviction is what the definition keeps."""
    c = O.CacheDef(2, 64, 16, 64, False, "bf16")
    spec, budget, sinks, recent = spec_of(c), 30, 2, 6
    pool = hr.cache_pool(spec, 40)
    table, lens = gpu(np.full((2, 8), -1, np.int32)), ints([0, 0])
    weights = torch.full((2, 2, 128), float("nan"), device=DEV)
    rng = torch.Generator().manual_seed(4)

    def draw(n, h):
        return torch.randn((n, h, 64), generator=rng).bfloat16().to(DEV)

    def step(parents, grow):
        nonlocal table, lens, weights
        r = hr.cache_update(pool, spec, table, lens, ints(parents), ints(grow))
        table, lens = r["table"], r["lens"]
        weights = weights[:, :].index_select(0, ints([max(p, 0) for p in parents]).long())
        cu, n = gpu(np.concatenate([[0], np.cumsum(grow)]).astype(np.int32)), sum(grow)
        q = draw(n, 8)
        hr.cache_append(pool, spec, draw(n, 2), draw(n, 2), table, lens, cu_q=cu)
        o, lse = hr.cache_attention(q, pool, spec, table, lens, cu_q=cu, lse=True)
        hr.cache_weights(q, pool, spec, table, lens, lse, weights, cu_q=cu)
        ref, _, bound = O.attention(q.double().cpu().numpy(), pool.cpu().numpy(), c, table.cpu().numpy(), lens.tolist(), cu.cpu().numpy())
        # (within 2^-7 of the values' size: rounded queries, probabilities and results)
        assert np.abs(o.double().cpu().numpy() - ref).max() < 2.0 ** -6 * max(1.0, np.abs(ref).max())
        return q
    if share:
        step([-1, -1], [70, 0])
        step([0, 0], [1, 3])
    else:
        step([-1, -1], [70, 50])
        step([0, 1], [1, 3])
    assert torch.isfinite(weights[0, :, :71]).all()
    before = {k: v.clone() for k, v in dict(pool=pool, w=weights, table=table, lens=lens).items()}
    r = hr.cache_evict(pool, spec, table, lens, weights, budget, sinks, recent)
    assert r["lens"].tolist() == [budget, budget] and r["status"].tolist()[1:3] == [0, 2]
    from oracle import evict as E
    p, w = before["pool"].cpu().numpy()[None].copy(), before["w"].cpu().numpy()[None].copy()
    ref = E.evict(p, c, before["table"].cpu().numpy(), before["lens"].tolist(), w, budget, sinks, recent)
    assert np.array_equal(pool.cpu().numpy(), p[0]) and np.array_equal(r["table"].cpu().numpy(), ref[0])
    # the heads' kept positions, by the weights
    for b in range(2):
        n = int(before["lens"][b])
        for h in range(2):
            x = before["w"][b, h, sinks:n - recent]
            kept = torch.sort(torch.topk(x, budget - sinks - recent).values).values
            assert torch.equal(torch.sort(weights[b, h, sinks:budget - recent]).values, kept)
    table, lens = r["table"], r["lens"]
    step([0, 1], [1, 1])
    step([1, 0], [2, 1])
    assert lens.tolist() == [budget + 3, budget + 2]


@pytest.mark.parametrize("rows,prompt,steps,budget", [(1, 40, 9, 16), (3, 100, 20, 64)])
def test_decode_example_with_a_budget(rows, prompt, steps, budget, capsys):
    import decode_cache
    args = ["--rows", rows, "--prompt", prompt, "--steps", steps, "--layers", 2, "--q-heads", 4, "--kv-heads", 2, "--head-dim", 64,
            "--budget", budget]
    error, logits = decode_cache.main([str(x) for x in args])
    assert error < 0.26 and math.isfinite(error)
    assert logits.shape == (rows, 256) and torch.isfinite(logits).all()
    left = budget + (steps - 1) % 8 + 1
    assert "lengths %s" % ([left] * rows) in capsys.readouterr().out


@pytest.mark.parametrize("d,group,page", [(64, 64, 16), (128, 32, 64), (256, 128, 32), (256, 32, 16)])
@pytest.mark.parametrize("kw", [dict(), dict(window=50), dict(causal=False)], ids=["causal", "window", "full"])
def test_weights_of_few_blocks_with_many_rows(d, group, page, kw):
    """Blocks whose rows are shared out among workgroups: some with a whole block, some
    with a part, sequences without tokens and with more tokens than positions, and
    blocks that no row sees."""
    seqs = [(500, 700), (0, 40), (130, 900), (300, 280), (1, 1)]
    run_weights(O.CacheDef(2, d, page, group, False, "bf16"), seqs, 4, seed=d, absent=[(2, 3, -1)], **kw)


def test_weights_of_blocks_that_stay_whole():
    """As many blocks as workgroups take without a cut, of one length and of two."""
    c = O.CacheDef(1, 64, 16, 64, False, "bf16")
    run_weights(c, [(12, 60)] * 1000, 4, seed=1)
    run_weights(c, [(12, 60), (0, 5), (14, 300)] * 170, 4, seed=2)
