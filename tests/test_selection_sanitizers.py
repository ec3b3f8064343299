"""Host arithmetic of w4a8_route's launch plans under
UndefinedBehaviorSanitizer (CPU only; tests/sanitize/route_driver.cpp)."""
import os
import subprocess

import pytest

from test_sanitizers import ENV, ROCM, ROOT, SAN, _clean, _run


def test_route_plans_under_sanitizer(tmp_path):
    hipcc = os.path.join(ROCM, "bin", "hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    csrc = os.path.join(ROOT, "w4a8_quantized_gemm_amd", "csrc")
    obj, drv = str(tmp_path / "route.o"), str(tmp_path / "route_driver")
    host_san = ["-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all"]
    flags = [hipcc, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-Xclang",
             "-target-feature", "-Xclang", "-packed-fp32-ops", *host_san,
             "-I", os.path.join(ROOT, "include"), "-I", csrc]
    _run([*flags, "-c", os.path.join(csrc, "route.hip"), "-o", obj])
    _run([*flags, "-x", "hip", os.path.join(SAN, "route_driver.cpp"), "-x", "none", obj,
          "-o", drv])
    r = subprocess.run([drv], capture_output=True, text=True, env=ENV, timeout=300)
    _clean(r.stdout + r.stderr)
    assert r.returncode == 0 and "0 failures" in r.stdout, r.stdout + r.stderr
