"""CPU tests of the paged cache's C ABI (no GPU): exports, the page layout and
every refusal, with its status and before anything touches the device.
Pointers are fake, aligned addresses far apart: every case fails validation."""
import ctypes
import os
import re

import pytest
import torch

import hadamard_rotation_preprocessing_amd as hr
from hadamard_rotation_preprocessing_amd import _lib as L
from hadamard_rotation_preprocessing_amd import cache as K
from oracle import cache as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x7F0000000000
POOL, KP, VP, TAB, LENS, CU, Q, OUT, WORK, LSE, X1, X2, X3, X4 = (P + i * (1 << 40) for i in range(14))
BIG = 1 << 40


def msg():
    return L.lib().hr_last_error().decode()


def refused(status, want, text):
    assert status == want, (status, msg())
    assert text in msg(), msg()


def cspec(heads=8, d=128, page=64, fmt=L.HR_Q_INT, bits=4, g=128, sym=0, sd=L.HR_BF16):
    return K.hr_cache_spec(heads, d, page, L.hr_qspec(fmt, bits, g, sym, sd, 0.0))


def test_exports_every_header_symbol():
    text = open(os.path.join(ROOT, "include", "hadarot_cache.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M)
    assert set(names) == set(K.EXPORTS)
    for n in names:
        assert hasattr(K._cache_lib(), n), n


@pytest.mark.parametrize("kw,status,text", [
    (dict(heads=0), L.HR_EINVAL, "kv_heads"),
    (dict(heads=1 << 20), L.HR_EINVAL, "kv_heads"),
    (dict(d=0), L.HR_EINVAL, "head_dim"),
    (dict(d=96), L.HR_EUNSUPPORTED, "head_dim"),
    (dict(d=512), L.HR_EUNSUPPORTED, "head_dim"),
    (dict(page=0), L.HR_EINVAL, "page_size"),
    (dict(page=8), L.HR_EUNSUPPORTED, "page_size"),
    (dict(page=48), L.HR_EUNSUPPORTED, "page_size"),
    (dict(page=512), L.HR_EUNSUPPORTED, "page_size"),
    (dict(fmt=L.HR_Q_MXFP4, g=32, sd=L.HR_E8M0), L.HR_EUNSUPPORTED, "MXFP4"),
    (dict(fmt=L.HR_Q_NVFP4, g=16, sd=L.HR_E4M3), L.HR_EUNSUPPORTED, "NVFP4"),
    (dict(fmt=9), L.HR_EINVAL, "format"),
    (dict(bits=8), L.HR_EUNSUPPORTED, "bits"),
    (dict(sym=2), L.HR_EINVAL, "sym"),
    (dict(sd=L.HR_E8M0), L.HR_EINVAL, "scales"),
    (dict(g=0), L.HR_EINVAL, "group_size"),
    (dict(g=48), L.HR_EINVAL, "group_size"),
    (dict(g=256), L.HR_EINVAL, "group_size"),
    (dict(g=16), L.HR_EUNSUPPORTED, "group_size"),
])
def test_spec_refusals(kw, status, text):
    out = K.hr_cache_page()
    refused(K._cache_lib().hr_cache_page_layout(ctypes.byref(cspec(**kw)), ctypes.byref(out)), status, text)


def test_null_spec_and_out():
    l = K._cache_lib()
    refused(l.hr_cache_page_layout(None, ctypes.byref(K.hr_cache_page())), L.HR_EINVAL, "spec")
    refused(l.hr_cache_page_layout(ctypes.byref(cspec()), None), L.HR_EINVAL, "out")
    refused(l.hr_cache_update_work(10, 1, None), L.HR_EINVAL, "bytes")
    refused(l.hr_cache_compact_work(10, None), L.HR_EINVAL, "bytes")
    refused(l.hr_cache_compact_work(0, ctypes.byref(ctypes.c_int64())), L.HR_EINVAL, "n_pages")
    refused(l.hr_cache_update_work(10, -1, ctypes.byref(ctypes.c_int64())), L.HR_EINVAL, "new_rows")


@pytest.mark.parametrize("heads", [1, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("sym", [False, True])
@pytest.mark.parametrize("sdt", ["bf16", "f32"])
def test_layout_matches_the_definition(heads, d, page, sym, sdt):
    for g in (32, d):
        lay = hr.CacheSpec(heads, d, page, hr.QSpec("int", 4, g, sym, sdt)).layout()
        off, head = O.CacheDef(heads, d, page, g, sym, sdt).offsets()
        assert lay["head_bytes"] == head and lay["page_bytes"] == head * heads and head % 128 == 0
        for name in ("k_codes", "v_codes", "k_scales", "v_scales", "k_zeros", "v_zeros"):
            assert lay[name] == off.get(name, (0, 0))[0]
            assert lay[name] % 16 == 0
        assert hr.cache_pool(hr.CacheSpec(heads, d, page, hr.QSpec("int", 4, g, sym, sdt)), 3, 2, "cpu").shape == (2, 3, head * heads)


def seqs(table=TAB, lens=LENS, cu=CU, rows=4, max_pages=10):
    return K.hr_cache_seqs(table, lens, cu, rows, max_pages)


def append(pool=POOL, n_pages=100, spec=None, sq=None, k=KP, kst=1024, ksh=128, v=VP, vst=1024, vsh=128, dt=L.HR_BF16, tokens=8):
    return K._cache_lib().hr_cache_append(pool, n_pages, ctypes.byref(spec or cspec()), ctypes.byref(sq or seqs()), k, kst, ksh,
                                          v, vst, vsh, dt, tokens, 1, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(spec=cspec(d=96)), L.HR_EUNSUPPORTED, "head_dim"),
    (dict(dt=7), L.HR_EINVAL, "dtype"),
    (dict(tokens=-1), L.HR_EINVAL, "tokens"),
    (dict(n_pages=0), L.HR_EINVAL, "n_pages"),
    (dict(sq=seqs(rows=-1)), L.HR_EINVAL, "rows"),
    (dict(sq=seqs(rows=0)), L.HR_EINVAL, "no rows"),
    (dict(sq=seqs(max_pages=0)), L.HR_EINVAL, "max_pages"),
    (dict(sq=seqs(max_pages=1 << 26)), L.HR_EINVAL, "max_pages"),
    (dict(sq=seqs(cu=None), tokens=9), L.HR_EINVAL, "multiple of rows"),
    (dict(sq=seqs(table=None)), L.HR_EINVAL, "table is NULL"),
    (dict(sq=seqs(lens=LENS + 2)), L.HR_EINVAL, "lens is not 4-byte"),
    (dict(sq=seqs(cu=CU + 1)), L.HR_EINVAL, "cu_q is not 4-byte"),
    (dict(pool=None), L.HR_EINVAL, "pool is NULL"),
    (dict(pool=POOL + 8), L.HR_EINVAL, "pool is not 16-byte"),
    (dict(k=None), L.HR_EINVAL, "k is NULL"),
    (dict(v=VP + 2), L.HR_EINVAL, "v is not 16-byte"),
    (dict(kst=1020), L.HR_EINVAL, "k rows"),
    (dict(ksh=130), L.HR_EINVAL, "k rows"),
    (dict(vsh=64), L.HR_EINVAL, "smaller than a row"),
    (dict(vst=0), L.HR_EINVAL, "smaller than a row"),
    (dict(kst=-1024), L.HR_EINVAL, "strides"),
    (dict(k=POOL + 4096), L.HR_EINVAL, "pool overlaps k"),
    (dict(sq=seqs(table=POOL)), L.HR_EINVAL, "pool overlaps table"),
    (dict(tokens=1 << 29, kst=1024, vst=1024), L.HR_EUNSUPPORTED, "one launch"),
])
def test_append_refusals(kw, status, text):
    refused(append(**kw), status, text)


def attention(q=Q, st=4096, sh=128, dt=L.HR_BF16, tokens=8, hq=32, pool=POOL, n_pages=100, spec=None, sq=None, scale=0.0,
              causal=1, window=0, out=OUT, ost=4096, osh=128, lse=None, max_q=4096, work=WORK, bytes_=0):
    return K._cache_lib().hr_cache_attention(q, st, sh, dt, tokens, hq, pool, n_pages, ctypes.byref(spec or cspec()),
                                             ctypes.byref(sq or seqs()), scale, causal, window, 1, out, ost, osh, lse, max_q,
                                             work, bytes_, None)


WHOLE = dict(tokens=4096, hq=32)   # enough rows that no scratch (and so no device query) is needed


@pytest.mark.parametrize("kw,status,text", [
    (dict(spec=cspec(page=8)), L.HR_EUNSUPPORTED, "page_size"),
    (dict(dt=L.HR_E8M0), L.HR_EINVAL, "dtype"),
    (dict(tokens=-3), L.HR_EINVAL, "tokens"),
    (dict(hq=0), L.HR_EINVAL, "q_heads"),
    (dict(hq=12), L.HR_EINVAL, "multiple of kv_heads"),
    (dict(max_q=-1), L.HR_EINVAL, "max_q"),
    (dict(tokens=1 << 28, hq=32), L.HR_EINVAL, "2^31"),
    (dict(scale=-1.0), L.HR_EINVAL, "scale"),
    (dict(scale=float("nan")), L.HR_EINVAL, "scale"),
    (dict(scale=float("inf")), L.HR_EINVAL, "scale"),
    (dict(window=-1), L.HR_EINVAL, "window"),
    (dict(window=4, causal=0), L.HR_EINVAL, "window needs causal"),
    (dict(q=None), L.HR_EINVAL, "q is NULL"),
    (dict(out=OUT + 4), L.HR_EINVAL, "out is not 16-byte"),
    (dict(st=100), L.HR_EINVAL, "q rows"),
    (dict(osh=64), L.HR_EINVAL, "smaller than a row"),
    (dict(ost=136, osh=128), L.HR_EINVAL, "make rows overlap"),
    (dict(pool=None), L.HR_EINVAL, "pool is NULL"),
    (dict(lse=LSE + 2), L.HR_EINVAL, "lse"),
    (dict(n_pages=-1), L.HR_EINVAL, "n_pages"),
    (dict(sq=seqs(cu=None, rows=3)), L.HR_EINVAL, "multiple of rows"),
    (dict(**WHOLE, out=Q + 4096), L.HR_EINVAL, "out overlaps q"),
    (dict(**WHOLE, out=Q, ost=4096 * 2), L.HR_EINVAL, "out overlaps q"),
    (dict(**WHOLE, lse=OUT + 64), L.HR_EINVAL, "out overlaps lse"),
    (dict(**WHOLE, out=POOL), L.HR_EINVAL, "out overlaps pool"),
    (dict(**WHOLE, sq=seqs(lens=OUT)), L.HR_EINVAL, "out overlaps lens"),
])
def test_attention_refusals(kw, status, text):
    refused(attention(**kw), status, text)


def test_empty_calls_are_fine():
    assert append(tokens=0, k=None, v=None, pool=None) == L.HR_OK
    assert attention(tokens=0, q=None, out=None, work=None) == L.HR_OK


def update(pool=POOL, layers=2, n_pages=100, spec=None, table=TAB, lens=LENS, rows=4, max_pages=10, parents=X1, grow=X2,
           new_rows=5, new_table=X3, new_lens=X4, refs=OUT, status=LSE, work=WORK, bytes_=1 << 20):
    return K._cache_lib().hr_cache_update(pool, layers, n_pages, ctypes.byref(spec or cspec()), table, lens, rows, max_pages,
                                          parents, grow, new_rows, new_table, new_lens, refs, status, work, bytes_, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(spec=cspec(g=8)), L.HR_EUNSUPPORTED, "group_size"),
    (dict(layers=0), L.HR_EINVAL, "layers"),
    (dict(n_pages=0), L.HR_EINVAL, "n_pages"),
    (dict(rows=-1), L.HR_EINVAL, "rows"),
    (dict(new_rows=-1), L.HR_EINVAL, "new_rows"),
    (dict(max_pages=-1), L.HR_EINVAL, "max_pages"),
    (dict(pool=None), L.HR_EINVAL, "pool"),
    (dict(refs=None), L.HR_EINVAL, "refs"),
    (dict(status=None), L.HR_EINVAL, "status"),
    (dict(table=None), L.HR_EINVAL, "table"),
    (dict(lens=None), L.HR_EINVAL, "lens"),
    (dict(parents=None), L.HR_EINVAL, "parents"),
    (dict(grow=X2 + 2), L.HR_EINVAL, "grow"),
    (dict(new_table=None), L.HR_EINVAL, "new_table"),
    (dict(new_lens=None), L.HR_EINVAL, "new_lens"),
    (dict(work=None), L.HR_EINVAL, "work"),
    (dict(bytes_=100), L.HR_EINVAL, "work_bytes"),
    (dict(new_table=TAB), L.HR_EINVAL, "overlaps"),
    (dict(new_lens=LENS), L.HR_EINVAL, "overlaps"),
    (dict(refs=X3 + 40), L.HR_EINVAL, "overlaps"),
])
def test_update_refusals(kw, status, text):
    refused(update(**kw), status, text)


def compact(pool=POOL, layers=2, n_pages=100, table=TAB, lens=LENS, rows=4, max_pages=10, into=None, into_pages=0,
            new_table=X3, refs=OUT, status=LSE, work=WORK, bytes_=1 << 20):
    return K._cache_lib().hr_cache_compact(pool, layers, n_pages, ctypes.byref(cspec()), table, lens, rows, max_pages, into,
                                           into_pages, new_table, refs, status, work, bytes_, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(layers=-1), L.HR_EINVAL, "layers"),
    (dict(n_pages=1 << 31), L.HR_EINVAL, "n_pages"),
    (dict(rows=-1), L.HR_EINVAL, "rows"),
    (dict(into=X1, into_pages=0), L.HR_EINVAL, "into_pages"),
    (dict(into=X1 + 8, into_pages=4), L.HR_EINVAL, "into is not"),
    (dict(into=POOL + 4096, into_pages=4), L.HR_EINVAL, "overlaps"),
    (dict(new_table=TAB + 4), L.HR_EINVAL, "overlaps"),
    (dict(table=None), L.HR_EINVAL, "table"),
    (dict(new_table=None), L.HR_EINVAL, "new_table"),
    (dict(refs=None), L.HR_EINVAL, "refs"),
    (dict(status=LSE + 1), L.HR_EINVAL, "status"),
    (dict(work=None), L.HR_EINVAL, "work"),
    (dict(bytes_=0), L.HR_EINVAL, "work_bytes"),
])
def test_compact_refusals(kw, status, text):
    refused(compact(**kw), status, text)


def test_binding_refusals():
    """What the binding checks before the C call: types, shapes, devices."""
    spec = hr.CacheSpec(2, 64, 16, hr.QSpec("int", 4, 64, False, "bf16"))
    pool = hr.cache_pool(spec, 4, device="cpu")
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    bad = [
        lambda: hr.cache_append(pool[:, :-16], spec, k, k, table, lens),
        lambda: hr.cache_append(pool.float(), spec, k, k, table, lens),
        lambda: hr.cache_append(pool, hr.CacheSpec(2, 128, 16), k, k, table, lens),
        lambda: hr.cache_append(pool, spec, k[:, :1], k, table, lens),
        lambda: hr.cache_append(pool, spec, k, k.float(), table, lens),
        lambda: hr.cache_append(pool, spec, k, k[:2], table, lens),
        lambda: hr.cache_append(pool, spec, k.half(), k.half(), table, lens),
        lambda: hr.cache_append(pool, spec, k, k, table.long(), lens),
        lambda: hr.cache_append(pool, spec, k, k, table, torch.zeros(2, dtype=torch.int32)),
        lambda: hr.cache_append(pool, spec, k, k, table, lens, cu_q=lens),
        lambda: hr.cache_append(pool, spec, k.transpose(1, 2).contiguous().transpose(1, 2), k, table, lens),
        lambda: hr.cache_update(pool, spec, table, lens, lens, torch.zeros(2, dtype=torch.int32)),
        lambda: hr.cache_update(pool, spec, table, lens, lens.long(), lens),
        lambda: hr.cache_compact(pool, spec, table, lens, into=pool[None].repeat(2, 1, 1)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError("case %d was accepted" % i)
