"""The cap of attention's scores (attn_cap.h), built for the host with g++, against
tanh in 64 bits: within 2^-21 over every cap that a call may have."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_block_scaled_gemv_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_the_cap_is_tanh(tmp_path):
    exe = tmp_path / "cap_check"
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-ffp-contract=off", "-I", CSRC, "-o",
                    str(exe), os.path.join(ROOT, "tests", "cap_check.cpp")],
                   check=True, capture_output=True, timeout=300)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.startswith("ok ") and int(out.stdout.split()[1]) > 10 ** 6, out.stdout
