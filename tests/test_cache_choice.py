"""Which attention kernel a call takes (CPU): cache_api.cpp with its launchers
replaced by recorders."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest

import test_cache_host as H
from hadamard_rotation_preprocessing_amd import _lib as L
from hadamard_rotation_preprocessing_amd import cache as K

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.join(HERE, "sanitize"))
pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not installed")


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    import build_hostsan as B
    out = str(tmp_path_factory.mktemp("choice") / "libchoice.so")
    cmd = ["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
           "-I", os.path.join(B.ROOT, "include")]
    cmd += [os.path.join(B.CSRC, n) for n in ("api.cpp", "paley.cpp", "cache_api.cpp")]
    cmd += [os.path.join(B.HERE, n) for n in ("launch_stubs.cpp", "choice_stubs.cpp")] + ["-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return ctypes.CDLL(out)


def waves(lib, tokens, rows, cu=True, max_q=0, keys=32768, dt=L.HR_BF16, hq=32):
    spec, sq = H.cspec(), H.seqs(rows=rows, max_pages=keys // 64, cu=H.CU if cu else None)
    need = ctypes.c_int64()
    f = lib.hr_cache_attention_work
    f.argtypes, g = K._cache_lib().hr_cache_attention_work.argtypes, lib.hr_cache_attention
    g.argtypes = K._cache_lib().hr_cache_attention.argtypes
    assert f(dt, tokens, hq, ctypes.byref(spec), rows, max_q, ctypes.byref(need)) == L.HR_OK
    st = g(H.Q, hq * 128, 128, dt, tokens, hq, H.POOL, 100, ctypes.byref(spec), ctypes.byref(sq), 0.0, 1, 0, 1, H.OUT, hq * 128,
           128, None, max_q, H.WORK, need.value, None)
    assert st == L.HR_EDEVICE, lib.hr_last_error   # (the scratch asked for suffices)
    return lib.chosen_waves()


@pytest.mark.parametrize("cu", [False, True])
def test_single_tokens_of_many_sequences(recorder, cu):
    """One new token in each of many sequences has few query rows a sequence,
    whether or not the caller says so."""
    for rows in (1, 16, 64, 1000):
        assert waves(recorder, rows, rows, cu) == 1
        assert waves(recorder, rows, rows, cu, max_q=1) == 1
    assert waves(recorder, 64 * 3, 64, cu) == 1
    assert waves(recorder, 40, 64) == 1            # most of them idle


def test_prompts(recorder):
    assert waves(recorder, 2048, 1) == 8
    assert waves(recorder, 2 * 2048, 2, cu=False) == 8
    assert waves(recorder, 64, 64, max_q=64) == 8  # the caller's bound goes before the mean
    assert waves(recorder, 64 * 64, 64) == 8
    assert waves(recorder, 30, 1, keys=64) == 1    # too few scores for it
