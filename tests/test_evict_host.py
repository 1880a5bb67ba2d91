"""CPU tests of the eviction's C ABI and binding (no GPU): exports, scratch sizes
and every refusal, with its status and before anything touches the device.
Pointers are fake, aligned addresses far apart: every case fails validation."""
import ctypes
import os
import re

import pytest
import torch

import hadamard_rotation_preprocessing_amd as hr
from hadamard_rotation_preprocessing_amd import _lib as L
from hadamard_rotation_preprocessing_amd import evict as E
from test_cache_host import CU, LENS, LSE, OUT, POOL, Q, ROOT, TAB, WORK, X1, X2, X3, X4, cspec, refused, seqs

W = X1
BIG = 1 << 36


def test_exports_every_header_symbol():
    text = open(os.path.join(ROOT, "include", "hadarot_evict.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M)
    assert set(names) == set(E.EXPORTS)
    for n in names:
        assert hasattr(E._evict_lib(), n), n


def weights(q=Q, st=4096, sh=128, dt=L.HR_BF16, tokens=8, hq=32, pool=POOL, n_pages=100, spec=None, sq=None, lse=LSE, scale=0.0,
            causal=1, window=0, decay=1.0, w=W, width=640, max_q=0, work=WORK, bytes_=BIG):
    return E._evict_lib().hr_cache_weights(q, st, sh, dt, tokens, hq, pool, n_pages, ctypes.byref(spec or cspec()),
                                           ctypes.byref(sq or seqs()), lse, scale, causal, window, 1, decay, w, width, max_q, work,
                                           bytes_, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(spec=cspec(d=96)), L.HR_EUNSUPPORTED, "head_dim"),
    (dict(dt=9), L.HR_EINVAL, "dtype"),
    (dict(tokens=-1), L.HR_EINVAL, "tokens"),
    (dict(hq=0), L.HR_EINVAL, "q_heads"),
    (dict(hq=12), L.HR_EINVAL, "multiple of kv_heads"),
    (dict(max_q=-1), L.HR_EINVAL, "max_q"),
    (dict(tokens=1 << 28), L.HR_EINVAL, "2^31"),
    (dict(n_pages=0), L.HR_EINVAL, "n_pages"),
    (dict(sq=seqs(rows=0)), L.HR_EINVAL, "no rows"),
    (dict(sq=seqs(cu=None), tokens=9), L.HR_EINVAL, "multiple of rows"),
    (dict(sq=seqs(lens=None)), L.HR_EINVAL, "lens is NULL"),
    (dict(sq=seqs(max_pages=(1 << 25) - 1), width=(1 << 31) - 1), L.HR_EUNSUPPORTED, "2^31 - 2^16"),
    (dict(scale=-1.0), L.HR_EINVAL, "scale"),
    (dict(scale=float("nan")), L.HR_EINVAL, "scale"),
    (dict(window=-1), L.HR_EINVAL, "window"),
    (dict(window=4, causal=0), L.HR_EINVAL, "window needs causal"),
    (dict(decay=-0.5), L.HR_EINVAL, "decay"),
    (dict(decay=float("nan")), L.HR_EINVAL, "decay"),
    (dict(decay=float("inf")), L.HR_EINVAL, "decay"),
    (dict(width=639), L.HR_EINVAL, "width"),
    (dict(width=1 << 31), L.HR_EINVAL, "width"),
    (dict(q=None), L.HR_EINVAL, "q is NULL"),
    (dict(q=Q + 8), L.HR_EINVAL, "q is not 16-byte"),
    (dict(st=100), L.HR_EINVAL, "q rows"),
    (dict(sh=64), L.HR_EINVAL, "smaller than a row"),
    (dict(pool=None), L.HR_EINVAL, "pool is NULL"),
    (dict(lse=None), L.HR_EINVAL, "lse is NULL"),
    (dict(w=None), L.HR_EINVAL, "weights is NULL"),
    (dict(w=W + 2), L.HR_EINVAL, "weights is not 4-byte"),
    (dict(work=None), L.HR_EINVAL, "work is NULL"),
    (dict(bytes_=1000), L.HR_EINVAL, "work_bytes"),
    (dict(w=LSE), L.HR_EINVAL, "weights overlaps lse"),
    (dict(w=POOL + 64), L.HR_EINVAL, "weights overlaps pool"),
    (dict(work=Q), L.HR_EINVAL, "work overlaps q"),
    (dict(sq=seqs(table=W)), L.HR_EINVAL, "weights overlaps table"),
    (dict(sq=seqs(cu=WORK)), L.HR_EINVAL, "work overlaps cu_q"),
])
def test_weights_refusals(kw, status, text):
    refused(weights(**kw), status, text)


def evict(pool=POOL, layers=2, n_pages=100, spec=None, table=TAB, lens=LENS, rows=4, max_pages=10, w=W, width=640, budget=64, sinks=4,
          recent=16, new_table=X3, new_lens=X4, refs=OUT, status=LSE, work=WORK, bytes_=1 << 20):
    return E._evict_lib().hr_cache_evict(pool, layers, n_pages, ctypes.byref(spec or cspec()), table, lens, rows, max_pages, w, width,
                                         budget, sinks, recent, new_table, new_lens, refs, status, work, bytes_, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(spec=cspec(g=8)), L.HR_EUNSUPPORTED, "group_size"),
    (dict(layers=0), L.HR_EINVAL, "layers"),
    (dict(n_pages=0), L.HR_EINVAL, "n_pages"),
    (dict(rows=-1), L.HR_EINVAL, "rows"),
    (dict(max_pages=0), L.HR_EINVAL, "max_pages"),
    (dict(rows=1 << 10, max_pages=1 << 21, width=(1 << 31) - 1), L.HR_EUNSUPPORTED, "2^31"),
    (dict(width=600), L.HR_EINVAL, "width"),
    (dict(budget=0), L.HR_EINVAL, "budget"),
    (dict(budget=1 << 31), L.HR_EINVAL, "budget"),
    (dict(sinks=-1), L.HR_EINVAL, "sinks"),
    (dict(recent=-1), L.HR_EINVAL, "recent"),
    (dict(sinks=40, recent=25), L.HR_EINVAL, "at most budget"),
    (dict(sinks=1 << 62, recent=1 << 62), L.HR_EINVAL, "at most budget"),
    (dict(pool=None), L.HR_EINVAL, "pool"),
    (dict(refs=None), L.HR_EINVAL, "refs"),
    (dict(status=LSE + 1), L.HR_EINVAL, "status"),
    (dict(table=None), L.HR_EINVAL, "table"),
    (dict(lens=LENS + 2), L.HR_EINVAL, "lens"),
    (dict(w=None), L.HR_EINVAL, "weights"),
    (dict(new_table=None), L.HR_EINVAL, "new_table"),
    (dict(new_lens=None), L.HR_EINVAL, "new_lens"),
    (dict(work=None), L.HR_EINVAL, "work"),
    (dict(bytes_=100), L.HR_EINVAL, "work_bytes"),
    (dict(new_table=TAB), L.HR_EINVAL, "overlaps"),
    (dict(new_lens=LENS), L.HR_EINVAL, "overlaps"),
    (dict(w=POOL + 1024), L.HR_EINVAL, "overlaps"),
    (dict(refs=X3 + 40), L.HR_EINVAL, "overlaps"),
    (dict(work=LENS), L.HR_EINVAL, "overlaps"),
])
def test_evict_refusals(kw, status, text):
    refused(evict(**kw), status, text)


def test_scratch_sizes_and_empty_calls():
    l, n = E._evict_lib(), ctypes.c_int64()
    assert weights(tokens=0, q=None, lse=None, w=None, work=None, bytes_=0) == L.HR_OK
    assert l.hr_cache_weights_work(L.HR_BF16, 0, 32, ctypes.byref(cspec()), 4, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert l.hr_cache_weights_work(L.HR_BF16, 5, 32, ctypes.byref(cspec()), 3, 0, ctypes.byref(n)) == 0
    assert n.value == 4 * 8 + 5 * 32 * 8 + 5 * 32 * 128 * 4
    assert l.hr_cache_evict_work(100, 4, ctypes.byref(n)) == 0 and n.value >= 4 * (3 * 100 + 4)
    refused(l.hr_cache_weights_work(L.HR_BF16, 5, 32, ctypes.byref(cspec()), 3, 0, None), L.HR_EINVAL, "bytes")
    refused(l.hr_cache_weights_work(L.HR_BF16, 5, 33, ctypes.byref(cspec()), 3, 0, ctypes.byref(n)), L.HR_EINVAL, "q_heads")
    refused(l.hr_cache_weights_work(L.HR_BF16, 5, 32, ctypes.byref(cspec()), -1, 0, ctypes.byref(n)), L.HR_EINVAL, "rows")
    refused(l.hr_cache_evict_work(0, 4, ctypes.byref(n)), L.HR_EINVAL, "n_pages")
    refused(l.hr_cache_evict_work(4, -4, ctypes.byref(n)), L.HR_EINVAL, "rows")
    refused(l.hr_cache_evict_work(4, 4, None), L.HR_EINVAL, "bytes")


def test_binding_refusals():
    spec = hr.CacheSpec(2, 64, 16, hr.QSpec("int", 4, 64, False, "bf16"))
    pool = hr.cache_pool(spec, 4, device="cpu")
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q, lse, w = torch.zeros((1, 4, 64)), torch.zeros((1, 4)), torch.zeros((1, 2, 32))
    two = hr.cache_pool(spec, 4, 2, "cpu")
    bad = [
        lambda: hr.cache_weights(q, pool, spec, table, lens, lse.half(), w),
        lambda: hr.cache_weights(q, pool, spec, table, lens, lse[:, :3], w),
        lambda: hr.cache_weights(q, pool, spec, table, lens, torch.zeros((1, 8))[:, ::2], w),
        lambda: hr.cache_weights(q, pool, spec, table, lens, lse, w.double()),
        lambda: hr.cache_weights(q, pool, spec, table, lens, lse, w[0]),
        lambda: hr.cache_weights(q, pool, spec, table, lens, lse, torch.zeros((1, 2, 64))[..., ::2]),
        lambda: hr.cache_weights(q, pool, spec, table, lens, lse, torch.zeros((2, 2, 32))),
        lambda: hr.cache_weights(q.half(), pool, spec, table, lens, lse, w),
        lambda: hr.cache_weights(q, pool, spec, table.long(), lens, lse, w),
        lambda: hr.cache_weights(q, pool, spec, table, lens, lse, w, cu_q=lens),
        lambda: hr.cache_weights(q, pool, spec, table, lens, lse, w, scale=1e-60),
        lambda: hr.cache_weights(q, two, spec, table, lens, lse, w),
        lambda: hr.cache_evict(pool, spec, table, lens, w[None], 16),
        lambda: hr.cache_evict(two, spec, table, lens, w, 16),
        lambda: hr.cache_evict(pool, spec, table, lens, w.to("meta"), 16),
        lambda: hr.cache_evict(pool, spec, table, lens[:0], w, 16),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError("case %d was accepted" % i)
