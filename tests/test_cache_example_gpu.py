"""The decoding example, small: append, attention, update and compaction as they
are used together.

Its attention against exact attention over unquantized keys and values: 4-bit
codes over a vector of 64 normal numbers leave steps of about 4.8 / 15 of a
standard deviation, so 0.09 of a value's size as noise on the values, and scores
of unit size that are off by as much: together 0.13, held to twice that."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("rows,prompt,steps,kv", [(1, 40, 3, 1), (3, 100, 20, 2)])
def test_decode_example(rows, prompt, steps, kv, capsys):
    import decode_cache
    args = ["--rows", rows, "--prompt", prompt, "--steps", steps, "--layers", 2, "--q-heads", 4, "--kv-heads", kv, "--head-dim", 64]
    error, logits = decode_cache.main([str(x) for x in args])
    assert error < 0.26 and math.isfinite(error)
    assert logits.shape == (rows, 256) and torch.isfinite(logits).all()
    assert "%d steps" % steps in capsys.readouterr().out


def test_a_captured_step_replays():
    """Append and attention in a graph, at lengths that grow between replays,
    against the same calls made one by one."""
    import hadamard_rotation_preprocessing_amd as hr
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(3)
    spec = hr.CacheSpec(2, 128, 16, hr.QSpec("int", 4, 128, False, "bf16"))
    pool = torch.randint(0, 60, (40, spec.page_bytes), generator=g, device=dev, dtype=torch.uint8)
    other = pool.clone()
    table = torch.randperm(36, generator=g, device=dev).to(torch.int32).view(3, 12)
    lens = torch.tensor([14, 100, 31], dtype=torch.int32, device=dev)
    x = torch.randn((3, 12, 128), generator=g, device=dev).bfloat16()

    def step(p, y):
        hr.cache_append(p, spec, y[:, 8:10], y[:, 10:], table, lens)
        return hr.cache_attention(y[:, :8], p, spec, table, lens, max_q=1, lse=True)
    step(other.clone(), x)          # (once outside the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(pool, x)
    for _ in range(6):
        x.normal_(generator=g)
        graph.replay()
        want, wlse = step(other, x)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wlse) and torch.equal(pool, other)
        lens += 1
