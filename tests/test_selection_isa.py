"""The tile kernels with adapters in their epilogue, in this build's own
gfx950 assembly (CPU only): none may spill.  Their accumulators fill the
AGPRs, and with one register too few this compiler has stored part of an
accumulator and reloaded it incompletely (wrong sums, no error)."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w4a8_quantized_gemm_amd", "csrc")
HIPCC = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")


def test_adapter_tile_kernels_do_not_spill(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    out = str(tmp_path / "mfma16.s")
    cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "--offload-device-only", "-S",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(CSRC, "gemm_mfma16.hip"), "-o", out]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    text = open(out).read()
    seen = 0
    for body in re.split(r"\n(?=_Z\S+:)", text):
        name = body.split(":", 1)[0]
        if name.startswith("_Z") and "mfma16_lora_kernel" in name:
            seen += 1
            code = body.split(".Lfunc_end", 1)[0]
            assert "scratch_" not in code, name
    assert seen == 8  # two tile heights, two group sizes, two adapter types
    spills = dict(re.findall(r"\.name:\s+(\S*mfma16_lora_kernel\S*)[\s\S]*?"
                             r"\.vgpr_spill_count:\s+(\d+)", text))
    assert len(spills) == 8 and set(spills.values()) == {"0"}, spills
