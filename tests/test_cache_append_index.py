"""cache_append's index arithmetic on the CPU (csrc/cache_index.h, the same
source that the kernel compiles): no block reads a token outside its sequence,
idle sequences included, and every new position is taken once."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not installed")
def test_append_blocks_stay_in_their_sequences(tmp_path):
    exe = str(tmp_path / "append_index")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Werror", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=undefined", os.path.join(HERE, "sanitize", "append_index.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and out.endswith("0 errors\n"), out[:3000]
