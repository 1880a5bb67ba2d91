"""CPU tests of the latent cache's C ABI and binding (no GPU): exports, the page
layout and every refusal, with its status and before anything touches the device.
Pointers are fake, aligned addresses far apart: every case fails validation."""
import ctypes
import os
import re

import pytest
import torch

import hadamard_rotation_preprocessing_amd as hr
from hadamard_rotation_preprocessing_amd import _lib as L
from hadamard_rotation_preprocessing_amd import latent as A
from oracle import latent as O
from test_cache_host import CU, KP, LENS, LSE, OUT, POOL, Q, ROOT, TAB, VP, WORK, X1, X2, X3, X4, refused, seqs

BIG = 1 << 36


def lspec(d=512, rope=64, page=64, fmt=L.HR_Q_INT, bits=4, g=128, sym=0, sd=L.HR_BF16):
    return A.hr_latent_spec(d, rope, page, L.hr_qspec(fmt, bits, g, sym, sd, 0.0))


def test_exports_every_header_symbol():
    text = open(os.path.join(ROOT, "include", "hadarot_latent.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = re.findall(r"^\s*int\s+(\w+)\s*\(", text, flags=re.M)
    assert set(names) == set(A.EXPORTS)
    for n in names:
        assert hasattr(A._latent_lib(), n), n


@pytest.mark.parametrize("kw,status,text", [
    (dict(d=0), L.HR_EINVAL, "latent_dim"),
    (dict(d=128), L.HR_EUNSUPPORTED, "latent_dim"),
    (dict(d=1024), L.HR_EUNSUPPORTED, "latent_dim"),
    (dict(rope=0), L.HR_EINVAL, "rope_dim"),
    (dict(rope=32), L.HR_EUNSUPPORTED, "rope_dim"),
    (dict(page=0), L.HR_EINVAL, "page_size"),
    (dict(page=24), L.HR_EUNSUPPORTED, "page_size"),
    (dict(page=512), L.HR_EUNSUPPORTED, "page_size"),
    (dict(fmt=L.HR_Q_MXFP4, g=32, sd=L.HR_E8M0), L.HR_EUNSUPPORTED, "MXFP4"),
    (dict(fmt=L.HR_Q_NVFP4, g=16, sd=L.HR_E4M3), L.HR_EUNSUPPORTED, "NVFP4"),
    (dict(fmt=9), L.HR_EINVAL, "format"),
    (dict(bits=8), L.HR_EUNSUPPORTED, "bits"),
    (dict(sym=2), L.HR_EINVAL, "sym"),
    (dict(sd=L.HR_E8M0), L.HR_EINVAL, "scales"),
    (dict(g=0), L.HR_EINVAL, "group_size"),
    (dict(g=-128), L.HR_EINVAL, "group_size"),
    (dict(g=48), L.HR_EINVAL, "group_size"),
    (dict(g=1024), L.HR_EINVAL, "group_size"),
    (dict(g=64), L.HR_EUNSUPPORTED, "group_size"),
])
def test_spec_refusals(kw, status, text):
    refused(A._latent_lib().hr_latent_page_layout(ctypes.byref(lspec(**kw)), ctypes.byref(A.hr_latent_page())), status, text)


def test_null_spec_and_out():
    l = A._latent_lib()
    refused(l.hr_latent_page_layout(None, ctypes.byref(A.hr_latent_page())), L.HR_EINVAL, "spec")
    refused(l.hr_latent_page_layout(ctypes.byref(lspec()), None), L.HR_EINVAL, "out")
    refused(l.hr_latent_attention_work(L.HR_BF16, 4, 16, ctypes.byref(lspec()), 4, 0, None), L.HR_EINVAL, "bytes")


@pytest.mark.parametrize("d", [256, 512])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("sym", [False, True])
@pytest.mark.parametrize("sdt", ["bf16", "f32"])
def test_layout_matches_the_definition(d, page, sym, sdt):
    for g in (128, d):
        spec = hr.LatentSpec(d, 64, page, hr.QSpec("int", 4, g, sym, sdt))
        lay, c = spec.layout(), O.LatentDef(d, page, g, sym, sdt)
        off = c.offsets()[0]
        assert spec.page_bytes == lay["page_bytes"] == c.page_bytes and c.page_bytes % 128 == 0
        for name in ("codes", "scales", "zeros", "rope"):
            assert lay[name] == off.get(name, (0, 0))[0]
            assert lay[name] % 16 == 0
        assert hr.cache_pool(spec, 3, 2, "cpu").shape == (2, 3, c.page_bytes)


def append(pool=POOL, n_pages=100, spec=None, sq=None, c=KP, ct=512, rope=VP, rt=64, dt=L.HR_BF16, tokens=8):
    return A._latent_lib().hr_latent_append(pool, n_pages, ctypes.byref(spec or lspec()), ctypes.byref(sq or seqs()), c, ct, rope, rt,
                                            dt, tokens, 1, None)


def read(pool=POOL, n_pages=100, spec=None, sq=None, c=KP, ct=512, rope=VP, rt=64, dt=L.HR_BF16, positions=8):
    return A._latent_lib().hr_latent_read(pool, n_pages, ctypes.byref(spec or lspec()), ctypes.byref(sq or seqs()), c, ct, rope, rt,
                                          dt, positions, 1, None)


PAGES = [
    (dict(spec=lspec(d=96)), L.HR_EUNSUPPORTED, "latent_dim"),
    (dict(dt=7), L.HR_EINVAL, "dtype"),
    (dict(n_pages=0), L.HR_EINVAL, "n_pages"),
    (dict(sq=seqs(rows=-1)), L.HR_EINVAL, "rows"),
    (dict(sq=seqs(rows=0)), L.HR_EINVAL, "no rows"),
    (dict(sq=seqs(max_pages=0)), L.HR_EINVAL, "max_pages"),
    (dict(sq=seqs(table=None)), L.HR_EINVAL, "table is NULL"),
    (dict(sq=seqs(lens=LENS + 2)), L.HR_EINVAL, "lens is not 4-byte"),
    (dict(pool=None), L.HR_EINVAL, "pool is NULL"),
    (dict(pool=POOL + 8), L.HR_EINVAL, "pool is not 16-byte"),
    (dict(c=None), L.HR_EINVAL, "c is NULL"),
    (dict(rope=VP + 4), L.HR_EINVAL, "rope is not 16-byte"),
    (dict(ct=516), L.HR_EINVAL, "c rows"),
    (dict(ct=256), L.HR_EINVAL, "smaller than a row"),
    (dict(rt=0), L.HR_EINVAL, "smaller than a row"),
    (dict(rt=-64), L.HR_EINVAL, "strides"),
    (dict(c=POOL + 4096), L.HR_EINVAL, "overlaps"),
    (dict(rope=POOL), L.HR_EINVAL, "overlaps"),
]


@pytest.mark.parametrize("kw,status,text", PAGES + [
    (dict(tokens=-1), L.HR_EINVAL, "tokens"),
    (dict(sq=seqs(cu=None), tokens=9), L.HR_EINVAL, "multiple of rows"),
    (dict(sq=seqs(table=POOL)), L.HR_EINVAL, "pool overlaps table"),
])
def test_append_refusals(kw, status, text):
    refused(append(**kw), status, text)


@pytest.mark.parametrize("kw,status,text", PAGES + [
    (dict(positions=-1), L.HR_EINVAL, "positions"),
    (dict(positions=(1 << 30) + 1), L.HR_EINVAL, "positions"),
    (dict(rope=KP + 1022), L.HR_EINVAL, "rope is not 16-byte"),
    (dict(rope=KP + 1008), L.HR_EINVAL, "overlaps"),                    # inside the latents' rows
    (dict(rope=KP + 1024, ct=576, rt=64), L.HR_EINVAL, "overlaps"),     # beside the first only
    (dict(rope=KP + 1024, ct=568, rt=568), L.HR_EINVAL, "overlaps"),    # into the next row
    (dict(sq=seqs(cu=KP)), L.HR_EINVAL, "overlaps"),
    (dict(sq=seqs(lens=VP)), L.HR_EINVAL, "overlaps"),
])
def test_read_refusals(kw, status, text):
    refused(read(**kw), status, text)


def attention(q=Q, st=8192, sh=512, r=KP, rst=1024, rsh=64, dt=L.HR_BF16, tokens=8, heads=16, pool=POOL, n_pages=100, spec=None, sq=None,
              scale=0.1, causal=1, out=OUT, ost=8192, osh=512, lse=None, max_q=0, work=WORK, bytes_=BIG):
    return A._latent_lib().hr_latent_attention(q, st, sh, r, rst, rsh, dt, tokens, heads, pool, n_pages, ctypes.byref(spec or lspec()),
                                               ctypes.byref(sq or seqs()), scale, causal, 1, out, ost, osh, lse, max_q, work, bytes_, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(spec=lspec(page=8)), L.HR_EUNSUPPORTED, "page_size"),
    (dict(dt=L.HR_E8M0), L.HR_EINVAL, "dtype"),
    (dict(tokens=-3), L.HR_EINVAL, "tokens"),
    (dict(heads=0), L.HR_EINVAL, "heads"),
    (dict(max_q=-1), L.HR_EINVAL, "max_q"),
    (dict(tokens=1 << 27), L.HR_EINVAL, "2^31"),
    (dict(n_pages=-1), L.HR_EINVAL, "n_pages"),
    (dict(sq=seqs(cu=None, rows=3)), L.HR_EINVAL, "multiple of rows"),
    (dict(sq=seqs(max_pages=(1 << 25) - 1)), L.HR_EUNSUPPORTED, "2^31 - 2^16"),
    (dict(scale=0.0), L.HR_EINVAL, "scale"),
    (dict(scale=-1.0), L.HR_EINVAL, "scale"),
    (dict(scale=float("nan")), L.HR_EINVAL, "scale"),
    (dict(scale=float("inf")), L.HR_EINVAL, "scale"),
    (dict(q=None), L.HR_EINVAL, "q is NULL"),
    (dict(r=None), L.HR_EINVAL, "q_rope is NULL"),
    (dict(out=OUT + 4), L.HR_EINVAL, "out is not 16-byte"),
    (dict(st=100), L.HR_EINVAL, "q rows"),
    (dict(rsh=32), L.HR_EINVAL, "smaller than a row"),
    (dict(osh=256), L.HR_EINVAL, "smaller than a row"),
    (dict(ost=520, osh=512), L.HR_EINVAL, "make rows overlap"),
    (dict(pool=None), L.HR_EINVAL, "pool is NULL"),
    (dict(lse=LSE + 2), L.HR_EINVAL, "lse"),
])
def test_attention_refusals(kw, status, text):
    refused(attention(**kw), status, text)


def prompt(q=Q, st=16 * 200, sh=200, k=KP, kt=4096, kh=256, v=VP, vt=4096, vh=256, rope=X1, rt=64, dt=L.HR_BF16, tokens=200,
           positions=300, heads=16, nope=128, cu_q=CU, cu_k=LENS, rows=4, scale=0.0, causal=1, out=OUT, ost=2048, osh=128, lse=None):
    return A._latent_lib().hr_latent_prompt_attention(q, st, sh, k, kt, kh, v, vt, vh, rope, rt, dt, tokens, positions, heads, nope, cu_q,
                                                      cu_k, rows, scale, causal, out, ost, osh, lse, None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dt=9), L.HR_EINVAL, "dtype"),
    (dict(dt=L.HR_F32), L.HR_EUNSUPPORTED, "HR_BF16 only"),
    (dict(tokens=-1), L.HR_EINVAL, "tokens"),
    (dict(positions=-1), L.HR_EINVAL, "positions"),
    (dict(heads=0), L.HR_EINVAL, "heads"),
    (dict(tokens=1 << 27), L.HR_EINVAL, "2^31"),
    (dict(nope=0), L.HR_EINVAL, "nope"),
    (dict(nope=96), L.HR_EUNSUPPORTED, "nope"),
    (dict(rows=-1), L.HR_EINVAL, "rows"),
    (dict(rows=0), L.HR_EINVAL, "no rows"),
    (dict(scale=-2.0), L.HR_EINVAL, "scale"),
    (dict(scale=float("inf")), L.HR_EINVAL, "scale"),
    (dict(cu_q=None), L.HR_EINVAL, "cu_q is NULL"),
    (dict(cu_k=LENS + 2), L.HR_EINVAL, "cu_k is not"),
    (dict(q=None), L.HR_EINVAL, "q is NULL"),
    (dict(sh=128), L.HR_EINVAL, "smaller than a row"),
    (dict(k=KP + 8), L.HR_EINVAL, "k is not 16-byte"),
    (dict(vh=64), L.HR_EINVAL, "smaller than a row"),
    (dict(rope=None), L.HR_EINVAL, "rope is NULL"),
    (dict(ost=136), L.HR_EINVAL, "make rows overlap"),
    (dict(lse=LSE + 1), L.HR_EINVAL, "lse"),
    (dict(out=Q), L.HR_EINVAL, "out overlaps q"),
    (dict(out=KP + 4096), L.HR_EINVAL, "out overlaps k"),
    (dict(out=X1), L.HR_EINVAL, "out overlaps rope"),
    (dict(lse=CU), L.HR_EINVAL, "lse overlaps cu_q"),
])
def test_prompt_refusals(kw, status, text):
    refused(prompt(**kw), status, text)


def test_empty_calls_are_fine():
    assert append(tokens=0, c=None, rope=None, pool=None) == L.HR_OK
    assert read(positions=0, c=None, rope=None, pool=None) == L.HR_OK
    assert attention(tokens=0, q=None, r=None, out=None, work=None, bytes_=0) == L.HR_OK
    assert prompt(tokens=0, q=None, out=None, cu_q=None) == L.HR_OK


def update(spec=None, new_table=X3, work=WORK, bytes_=1 << 20, layers=2):
    return A._latent_lib().hr_latent_update(POOL, layers, 100, ctypes.byref(spec or lspec()), TAB, LENS, 4, 10, X1, X2, 5, new_table, X4, OUT,
                                            LSE, work, bytes_, None)


def compact(spec=None, into=None, into_pages=0, new_table=X3, bytes_=1 << 20):
    return A._latent_lib().hr_latent_compact(POOL, 2, 100, ctypes.byref(spec or lspec()), TAB, LENS, 4, 10, into, into_pages, new_table, OUT,
                                             LSE, WORK, bytes_, None)


def test_pages_that_move():
    refused(update(spec=lspec(g=64)), L.HR_EUNSUPPORTED, "group_size")
    refused(update(layers=0), L.HR_EINVAL, "layers")
    refused(update(new_table=TAB), L.HR_EINVAL, "overlaps")
    refused(update(bytes_=100), L.HR_EINVAL, "work_bytes")
    refused(compact(spec=lspec(d=64)), L.HR_EUNSUPPORTED, "latent_dim")
    refused(compact(into=X1, into_pages=0), L.HR_EINVAL, "into_pages")
    refused(compact(into=POOL + 4096, into_pages=4), L.HR_EINVAL, "overlaps")
    refused(compact(bytes_=0), L.HR_EINVAL, "work_bytes")


def test_binding_refusals():
    spec = hr.LatentSpec(256, 64, 16, hr.QSpec("int", 4, 128, False, "bf16"))
    pool = hr.cache_pool(spec, 4, device="cpu")
    i32 = dict(dtype=torch.int32)
    table, lens, cu = torch.zeros((1, 2), **i32), torch.zeros(1, **i32), torch.zeros(2, **i32)
    c, rope = torch.zeros((3, 256)), torch.zeros((3, 64))
    q, r = torch.zeros((3, 4, 256)), torch.zeros((3, 4, 64))
    pq, pk = torch.zeros((3, 4, 192)).bfloat16(), torch.zeros((5, 4, 128)).bfloat16()
    prope = torch.zeros((5, 64)).bfloat16()
    bad = [
        lambda: hr.latent_append(pool[:, :-16], spec, c, rope, table, lens),
        lambda: hr.latent_append(pool, spec, c[:, :128], rope, table, lens),
        lambda: hr.latent_append(pool, spec, c, rope[:2], table, lens),
        lambda: hr.latent_append(pool, spec, c, rope.bfloat16(), table, lens),
        lambda: hr.latent_append(pool, spec, c.half(), rope.half(), table, lens),
        lambda: hr.latent_append(pool, spec, torch.zeros((256, 3)).t(), rope, table, lens),
        lambda: hr.latent_append(pool, spec, c.to("meta"), rope, table, lens),
        lambda: hr.latent_append(pool, spec, c, rope, table.long(), lens),
        lambda: hr.latent_read(pool, spec, table, lens, None, 3, out=(c, rope.bfloat16())),
        lambda: hr.latent_read(pool, spec, table, lens, None, 4, out=(c, rope)),
        lambda: hr.latent_read(pool, spec, table, lens, lens, 3),
        lambda: hr.latent_attention(q, r[:, :2], pool, spec, table, lens, 0.1),
        lambda: hr.latent_attention(q, r.bfloat16(), pool, spec, table, lens, 0.1),
        lambda: hr.latent_attention(q, r, pool, spec, table, lens, 0.1, out=q.bfloat16()),
        lambda: hr.latent_attention(q, r, pool, spec, table, lens, 0.1, lse=torch.zeros((4, 3))),
        lambda: hr.latent_attention(q, r, pool, spec, table, lens, 0.1, work=torch.empty(64, dtype=torch.uint8, device="meta")),
        lambda: hr.latent_prompt_attention(pq[..., :128], pk, prope, pk, cu, cu),
        lambda: hr.latent_prompt_attention(pq, pk, prope[:4], pk, cu, cu),
        lambda: hr.latent_prompt_attention(pq, pk, prope, pk[:4], cu, cu),
        lambda: hr.latent_prompt_attention(pq, pk.float(), prope, pk, cu, cu),
        lambda: hr.latent_prompt_attention(pq, pk, prope, pk, cu, lens),
        lambda: hr.latent_prompt_attention(pq, pk, prope, pk, cu.long(), cu),
        lambda: hr.latent_prompt_attention(pq, pk, prope, pk, cu, cu, scale=1e-60),
        lambda: hr.latent_prompt_attention(pq, pk, prope, pk, cu, cu, out=torch.zeros((3, 4, 64)).bfloat16()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError("case %d was accepted" % i)
