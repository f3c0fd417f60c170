"""Tiles of 16, 32 and 64 keys (attn_span.h), built for the host with g++ and walked
up to lengths of 2^31 - 1: no fetch, two tiles ahead and past the last one too, leaves
the sequence's table row, and what is looked up once lies in one page."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_block_scaled_gemv_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")
def test_fetches_of_every_tile(tmp_path):
    exe = tmp_path / "attn_tiles_check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-I", CSRC, "-o", str(exe),
                    os.path.join(ROOT, "tests", "attn_tiles_check.cpp")],
                   check=True, capture_output=True, timeout=300)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.startswith("ok "), out.stdout
