"""The paged cache's validation layer under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU): cache_api.cpp with api.cpp and paley.cpp,
launchers stubbed out, running tests/test_cache_host.py in a child process, and
calls that pass validation and reach the stubs (HR_EDEVICE)."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.join(HERE, "sanitize"))
OUT = os.path.join(HERE, "sanitize", "_build", "libhadarot_cachesan.so")


def build():
    import build_hostsan as B
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-shared", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
           "-I", os.path.join(B.ROOT, "include")] + B.SAN
    cmd += [os.path.join(B.CSRC, n) for n in ("api.cpp", "paley.cpp", "cache_api.cpp")]
    cmd += [os.path.join(B.HERE, n) for n in ("launch_stubs.cpp", "cache_stubs.cpp")] + ["-o", OUT]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return B.asan_runtime()


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not installed")
def test_cache_host_under_asan_ubsan():
    rt = build()
    if not os.path.isabs(rt) or not os.path.exists(rt):
        pytest.skip("g++ has no shared AddressSanitizer runtime")
    env = dict(os.environ)
    env.update(HADAROT_LIBRARY=OUT, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.join(HERE, "test_cache_host.py"),
                        os.path.abspath(__file__) + "::test_valid_calls_reach_the_launchers"], env=env,
                       capture_output=True, text=True, cwd=os.path.dirname(HERE), timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert " passed" in out, out[-2000:]


def test_valid_calls_reach_the_launchers():
    if os.environ.get("HADAROT_LIBRARY") != OUT:
        pytest.skip("runs in the sanitizer build")
    import test_cache_host as T
    from hadamard_rotation_preprocessing_amd import _lib as L
    for d in (64, 128, 256):
        for g in (32, d):
            for dt in (L.HR_BF16, L.HR_F32):
                for page, rows, tokens in ((16, 1, 1), (64, 4, 8), (256, 1000, 3000)):
                    spec = T.cspec(d=d, g=g, page=page)
                    sq = T.seqs(rows=rows)
                    assert T.append(spec=spec, sq=sq, dt=dt, tokens=tokens, kst=8 * d, ksh=d, vst=8 * d, vsh=d) == L.HR_EDEVICE
                    for max_q in (0, 1, 5, 4096):
                        need = ctypes.c_int64()
                        l = T.K._cache_lib()
                        assert l.hr_cache_attention_work(dt, tokens, 32, ctypes.byref(spec), rows, max_q, ctypes.byref(need)) == 0
                        kw = dict(spec=spec, sq=sq, dt=dt, tokens=tokens, st=32 * d, sh=d, ost=32 * d, osh=d, max_q=max_q)
                        assert T.attention(bytes_=need.value, **kw) == L.HR_EDEVICE
                        assert T.attention(bytes_=need.value, **{**kw, "out": T.Q}) == L.HR_EDEVICE   # in place
                        if need.value:
                            T.refused(T.attention(bytes_=need.value - 1, **kw), L.HR_EINVAL, "work_bytes")
                            T.refused(T.attention(bytes_=need.value, **{**kw, "work": None}), L.HR_EINVAL, "work is NULL")
                            T.refused(T.attention(bytes_=need.value, **{**kw, "work": T.OUT}), L.HR_EINVAL, "overlaps")
    assert T.update() == L.HR_EDEVICE and T.compact() == L.HR_EDEVICE
    assert T.update(rows=0, table=None, lens=None) == L.HR_EDEVICE
    assert T.update(new_rows=0, parents=None, grow=None, new_table=None, new_lens=None) == L.HR_EDEVICE
    assert T.compact(into=T.X1, into_pages=7) == L.HR_EDEVICE
