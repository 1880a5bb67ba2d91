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
