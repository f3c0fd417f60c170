"""The norm's quotients by a reciprocal and its remainder (divide.h), built for
the host with g++, against the division: no difference in some 2e7 of them."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_block_scaled_gemv_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_quotients_are_the_divisions(tmp_path):
    exe = tmp_path / "divide_check"
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-ffp-contract=off", "-I", CSRC, "-o",
                    str(exe), os.path.join(ROOT, "tests", "divide_check.cpp")],
                   check=True, capture_output=True, timeout=300)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.startswith("ok ") and int(out.stdout.split()[1]) > 10 ** 7
