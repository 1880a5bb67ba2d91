"""The validation layers of the eviction and of the latent cache under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU): their entry points with
those of the cache, launchers stubbed out, running tests/test_evict_host.py and
tests/test_latent_host.py in a child process, and calls that pass validation and
reach the stubs (HR_EDEVICE)."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.join(HERE, "sanitize"))
OUT = os.path.join(HERE, "sanitize", "_build", "libhadarot_evictsan.so")


def build():
    import build_hostsan as B
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-shared", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
           "-I", os.path.join(B.ROOT, "include")] + B.SAN
    cmd += [os.path.join(B.CSRC, n) for n in ("api.cpp", "paley.cpp", "cache_api.cpp", "evict_api.cpp", "latent_api.cpp")]
    cmd += [os.path.join(B.HERE, n) for n in ("launch_stubs.cpp", "cache_stubs.cpp", "evict_latent_stubs.cpp")] + ["-o", OUT]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return B.asan_runtime()


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not installed")
def test_host_layers_under_asan_ubsan():
    rt = build()
    if not os.path.isabs(rt) or not os.path.exists(rt):
        pytest.skip("g++ has no shared AddressSanitizer runtime")
    env = dict(os.environ)
    env.update(HADAROT_LIBRARY=OUT, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.join(HERE, "test_evict_host.py"),
                        os.path.join(HERE, "test_latent_host.py"), os.path.abspath(__file__) + "::test_valid_calls_reach_the_launchers"],
                       env=env, capture_output=True, text=True, cwd=os.path.dirname(HERE), timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert " passed" in out, out[-2000:]


def test_valid_calls_reach_the_launchers():
    if os.environ.get("HADAROT_LIBRARY") != OUT:
        pytest.skip("runs in the sanitizer build")
    import test_evict_host as E
    import test_latent_host as A
    from hadamard_rotation_preprocessing_amd import _lib as L
    need = ctypes.c_int64()
    for d in (64, 128, 256):
        for dt in (L.HR_BF16, L.HR_F32):
            for page, rows, tokens, max_q in ((16, 1, 1, 0), (64, 4, 8, 2), (256, 1000, 3000, 0), (64, 3, 60, 1 << 40)):
                spec, sq = E.cspec(d=d, g=d, page=page), E.seqs(rows=rows)
                l = E.E._evict_lib()
                assert l.hr_cache_weights_work(dt, tokens, 32, ctypes.byref(spec), rows, max_q, ctypes.byref(need)) == 0
                kw = dict(spec=spec, sq=sq, dt=dt, tokens=tokens, st=32 * d, sh=d, width=10 * page, max_q=max_q)
                assert E.weights(bytes_=need.value, **kw) == L.HR_EDEVICE
                E.refused(E.weights(bytes_=need.value - 1, **kw), L.HR_EINVAL, "work_bytes")
    assert E.weights(sq=E.seqs(max_pages=(1 << 25) - (1 << 10)), width=(1 << 31) - 1) == L.HR_EDEVICE
    assert E.evict() == L.HR_EDEVICE
    assert E.evict(rows=0, table=None, lens=None, w=None, new_table=None, new_lens=None) == L.HR_EDEVICE
    assert E.evict(sinks=0, recent=64) == L.HR_EDEVICE
    assert A.append() == L.HR_EDEVICE and A.read() == L.HR_EDEVICE and A.prompt() == L.HR_EDEVICE
    assert A.read(rope=A.KP + 1024, ct=576, rt=576) == L.HR_EDEVICE      # columns of one matrix
    assert A.read(c=A.KP + 128, rope=A.KP, ct=576, rt=576) == L.HR_EDEVICE
    assert A.prompt(positions=0, k=None, v=None, rope=None) == L.HR_EDEVICE
    assert A.update() == L.HR_EDEVICE and A.compact() == L.HR_EDEVICE and A.compact(into=A.X1, into_pages=7) == L.HR_EDEVICE
    for d in (256, 512):
        for dt in (L.HR_BF16, L.HR_F32):
            for rows, tokens, heads, max_q in ((1, 1, 16, 0), (4, 8, 128, 2), (1000, 3000, 16, 0), (8, 8, 1, 1)):
                spec = A.lspec(d=d)
                l = A.A._latent_lib()
                assert l.hr_latent_attention_work(dt, tokens, heads, ctypes.byref(spec), rows, max_q, ctypes.byref(need)) == 0
                kw = dict(spec=spec, sq=A.seqs(rows=rows), dt=dt, tokens=tokens, heads=heads, st=heads * d, sh=d, rst=heads * 64,
                          ost=heads * d, osh=d, max_q=max_q)
                assert A.attention(bytes_=need.value, **kw) == L.HR_EDEVICE
                assert A.attention(bytes_=need.value, **{**kw, "out": A.Q}) == L.HR_EDEVICE   # in place
                A.refused(A.attention(bytes_=need.value - 1, **kw), L.HR_EINVAL, "work_bytes")
                A.refused(A.attention(bytes_=need.value, **{**kw, "work": None}), L.HR_EINVAL, "work is NULL")
                for other in ("work", "lse"):
                    A.refused(A.attention(bytes_=need.value, **{**kw, other: A.OUT}), L.HR_EINVAL, "overlaps")
                    A.refused(A.attention(bytes_=need.value, **{**kw, other: A.Q}), L.HR_EINVAL, "overlaps")
                A.refused(A.attention(bytes_=need.value, **{**kw, "out": A.POOL}), L.HR_EINVAL, "overlaps")
                A.refused(A.attention(bytes_=need.value, **{**kw, "lse": A.KP}), L.HR_EINVAL, "overlaps")
