"""Host arithmetic of w4a8_norm_quant and w4a8_ffn (argument checks, kernel
plans, workspace sizes) under UndefinedBehaviorSanitizer (CPU only;
tests/sanitize/layer_driver.cpp)."""
import os
import subprocess

import pytest

from test_sanitizers import ENV, ROCM, ROOT, SAN, _clean, _run


def test_layer_plans_under_sanitizer(tmp_path):
    hipcc = os.path.join(ROCM, "bin", "hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    csrc = os.path.join(ROOT, "w4a8_quantized_gemm_amd", "csrc")
    host_san = ["-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all"]
    flags = [hipcc, "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-Xclang",
             "-target-feature", "-Xclang", "-packed-fp32-ops", *host_san,
             "-I", os.path.join(ROOT, "include"), "-I", csrc]
    objs = []
    for src in ("api.hip", "gemm_mfma.hip"):
        objs.append(str(tmp_path / (src + ".o")))
        _run([*flags, "-c", os.path.join(csrc, src), "-o", objs[-1]])
    drv = str(tmp_path / "layer_driver")
    # the other launchers are not linked: no call gets that far without a GPU
    _run([*flags, "-x", "hip", os.path.join(SAN, "layer_driver.cpp"), "-x", "none", *objs,
          "-Wl,--unresolved-symbols=ignore-all", "-o", drv])
    env = dict(ENV, HIP_VISIBLE_DEVICES="-1")
    r = subprocess.run([drv], capture_output=True, text=True, env=env, timeout=300)
    _clean(r.stdout + r.stderr)
    assert r.returncode == 0 and "0 failures" in r.stdout, r.stdout + r.stderr
