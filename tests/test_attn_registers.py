"""The registers of plain attention's kernels, as the compiler reports them: what
they are shared with must not cost them any. Limits: lane registers and spilled
ones of each form as they were before scored attention and the NVFP4 cache came."""
import os
import re
import shutil
import subprocess

import pytest

from nvfp4_block_scaled_gemv_amd import build

# kernel, D, E4M3, row tiles, pages of whole runs: lane registers, spilled
FORMS = {
    ("runs", 64, False, 1, True): (135, 0),
    ("runs", 64, False, 2, True): (182, 0),
    ("runs", 64, True, 1, False): (128, 0),
    ("runs", 64, True, 2, True): (167, 0),
    ("runs", 128, False, 1, True): (191, 0),
    ("runs", 128, True, 1, False): (168, 0),
    ("runs", 128, False, 2, True): (255, 0),
    ("runs", 256, False, 2, True): (256, 45),
    ("whole", 64, False, 2, True): (187, 0),
    ("whole", 128, False, 1, True): (191, 0),
    ("whole", 128, False, 2, True): (256, 15),
    ("whole", 128, False, 2, False): (256, 53),
    ("whole", 128, True, 1, False): (176, 0),
    ("whole", 128, True, 2, False): (256, 4),
}


@pytest.fixture(scope="module")
def usage(tmp_path_factory):
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if shutil.which(hipcc) is None:
        pytest.skip("hipcc not installed")
    out = tmp_path_factory.mktemp("registers") / "attn.o"
    flags = [f for f in build.FLAGS if f != "-shared"]
    r = subprocess.run([hipcc, *flags, f"-I{build.INCLUDE}", f"-I{build.CSRC}",
                        "--cuda-device-only", "-c", "-o", str(out),
                        "-Rpass-analysis=kernel-resource-usage",
                        os.path.join(build.CSRC, "paged_attn.hip")],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    found, name = {}, None
    for line in r.stderr.splitlines():
        m = re.search(r"Function Name: (\S+)", line)
        if m:
            # the wavefront's class: head, E4M3, row tiles, pages, scored, heads side by side
            k = re.search(r"k_attn_(runs|whole)INS0_8AttnWaveILi(\d+)ELb(\d)ELi(\d)ELb(\d)ELb0ELi1E",
                          m[1])
            name = k and (k[1], int(k[2]), k[3] == "1", int(k[4]), k[5] == "1")
        m = re.search(r"remark: +.*?\b(VGPRs|VGPRs Spill): (\d+)", line)
        if m and name:
            found.setdefault(name, {})[m[1]] = int(m[2])
    return found


@pytest.mark.parametrize("form", list(FORMS), ids=lambda f: "-".join(map(str, f)))
def test_plain_attention_keeps_its_registers(usage, form):
    registers, spilled = FORMS[form]
    got = usage[form]
    assert got["VGPRs"] <= registers and got["VGPRs Spill"] <= spilled, got
