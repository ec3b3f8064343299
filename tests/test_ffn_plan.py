"""The kernels w4a8_ffn takes, through w4a8_ffn_plan (host logic, no GPU): real
blocks, and every form that a plan can choose against the sizes of the GPU
tests, so that a change of the rules cannot leave a kernel without a test."""
import ast
import ctypes
import os
import re

import pytest

import w4a8_quantized_gemm_amd as w4
from ffn_cases import CASES

HERE = os.path.dirname(os.path.abspath(__file__))


def form(p):
    return (p["kernel"], p["tile_rows"], p["tile_channels"], p["splits"], p["k_parts"])


def forms(M, H, F):
    p = w4.ffn_plan(M, H, F)
    return form(p["up"]), form(p["down"])


PLANS = {  # (M, H, F): gate and up, down
    (1, 4096, 11008): (("stream", 16, 16, 1, 8), ("rows", 16, 16, 1, 8)),
    (1, 8192, 28672): (("stream", 16, 16, 1, 8), ("rows", 16, 32, 1, 8)),
    (16, 8192, 28672): (("stream", 16, 32, 1, 8), ("stream", 16, 32, 1, 8)),
    (47, 4096, 11008): (("tile16", 64, 64, 1, 2), ("stream", 32, 32, 1, 8)),
    (64, 8192, 28672): (("tile16", 64, 64, 1, 2), ("tile16", 64, 128, 8, 2)),
    (133, 2048, 1408): (("stream", 32, 16, 1, 4), ("stream", 32, 32, 1, 4)),
    (2048, 4096, 11008): (("tile16", 128, 128, 1, 1), ("tile32", 128, 256, 1, 1)),
    (4096, 5120, 13824): (("tile16", 128, 128, 1, 1), ("tile16", 256, 256, 1, 1)),
    (8192, 7168, 18944): (("tile16", 128, 128, 1, 1), ("tile16", 256, 256, 1, 1)),
    (4096, 8192, 28672): (("tile16", 256, 128, 1, 1), ("tile16", 256, 256, 1, 1)),
}


@pytest.mark.parametrize("shape", PLANS, ids=lambda s: "x".join(map(str, s)))
def test_plan(shape):
    assert forms(*shape) == PLANS[shape]


def kinds(M, H, F):
    """Forms without the number of splits beyond "more than one"."""
    return {(n, f[:3], f[3] > 1, f[4]) for n, f in zip(("up", "down"), forms(M, H, F))}


def test_every_form_has_a_gpu_test():
    tree = ast.parse(open(os.path.join(HERE, "test_gpu_layer.py")).read())
    lists = [ast.literal_eval(n.value) for n in tree.body
             if isinstance(n, ast.Assign) and n.targets[0].id == "FFN"]
    tested = set().union(*(kinds(*c[:3]) for c in lists[0] + CASES))
    rows = [1, 2, 3, 4, 8, 16, 17, 24, 32, 33, 48, 63, 64, 65, 80, 96, 97, 128, 129, 160, 200, 256,
            257, 300, 400, 512, 513, 640, 1000, 1500, 2048, 4096, 5000, 8192, 16384]
    widths = [128 * i for i in (1, 2, 3, 4, 5, 6, 8, 9, 11, 12, 13, 16, 18, 20, 25, 28, 30, 32, 40,
                                44, 48, 52, 56, 64, 65, 80, 86, 100, 128, 160, 200, 224, 256, 300,
                                400, 512, 1024)]
    for H in widths:
        for F in widths:
            if 2 * H * F >= 1 << 32:
                continue
            for M in rows:
                if M * max(H, F) >= 1 << 31:
                    continue
                missing = kinds(M, H, F) - tested
                assert not missing, ((M, H, F), missing)


def test_plan_errors():
    out = [ctypes.c_int(0) for _ in range(5)]
    ptrs = [ctypes.addressof(v) for v in out]
    plan = w4.lib.w4a8_ffn_plan
    assert plan(0, 256, 384, 0, *ptrs) == 0 and plan(0, 256, 384, 1, *ptrs) == 0
    for i in range(5):
        assert plan(4, 256, 384, 0, *ptrs[:i], None, *ptrs[i + 1:]) == 1
    assert plan(-1, 256, 384, 0, *ptrs) == 2 and plan(4, 200, 384, 0, *ptrs) == 2
    assert plan(4, 256, 64, 1, *ptrs) == 2 and plan(1 << 23, 256, 384, 1, *ptrs) == 2
    assert plan(4, 256, 384, 2, *ptrs) == 5 and plan(4, 256, 384, -1, *ptrs) == 5


def test_no_streamed_kernel_without_a_plan():
    """Compiled forms (tiles, row blocks) against those that plans choose: gate and
    up with two or four tiles and one or two row blocks, bfloat16 results (of the
    down product alone) with one, two or four tiles and one or two."""
    from test_isa_hazards import HIPCC, OUT, _asm
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    os.makedirs(OUT, exist_ok=True)

    def compiled(src, pattern):
        return {tuple(map(int, m)) for m in re.findall(pattern, _asm(src))}
    glu = compiled("gemm_stream_glu.hip",
                   r"w4a8_stream_glu_kernelILi(\d)ELi\dELi\d+ELb\dELi(\d)ELi\dEE")
    assert glu == {(4, 1), (4, 2), (2, 1), (2, 2)}
    bf16 = compiled("gemm_stream.hip",  # <tiles, stages, 2, group, parameters in LDS, W4A8, blocks>
                    r"w4a8_stream_kernelILi(\d)ELi\dELi2ELi\d+ELb\dELi0ELi(\d)EE")
    assert bf16 == {(4, 1), (4, 2), (2, 1), (2, 2), (1, 1), (1, 2)}
