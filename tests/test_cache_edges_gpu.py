"""The paged 4-bit cache on the GPU where one sequence, key or row could reach
another's result: idle sequences, scales and queries of very different sizes.
Oracle and bounds as in test_cache_gpu.py."""
import pytest

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
