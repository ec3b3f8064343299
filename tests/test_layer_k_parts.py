"""The K-tiles whose weights the tile kernels load lie in their row, whatever its
length and the number of parts (CPU only; tests/sanitize/kparts_driver.cpp).

One K-tile in two parts leaves the first part without any: its waves once loaded
the K-tile in front of the row, at a scalar offset that the buffer's range
check does not cover."""
import os
import subprocess

import pytest

from test_sanitizers import ENV, ROCM, ROOT, SAN, _clean, _run


def test_every_k_tile_lies_in_its_row(tmp_path):
    hipcc = os.path.join(ROCM, "bin", "hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    csrc = os.path.join(ROOT, "w4a8_quantized_gemm_amd", "csrc")
    drv = str(tmp_path / "kparts_driver")
    _run([hipcc, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-Xclang", "-target-feature",
          "-Xclang", "-packed-fp32-ops", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host",
          "-fno-sanitize-recover=all", "-I", csrc, "-x", "hip",
          os.path.join(SAN, "kparts_driver.cpp"), "-o", drv])
    env = dict(ENV, HIP_VISIBLE_DEVICES="-1")
    r = subprocess.run([drv], capture_output=True, text=True, env=env, timeout=300)
    _clean(r.stdout + r.stderr)
    assert r.returncode == 0 and "0 failures" in r.stdout, r.stdout + r.stderr
