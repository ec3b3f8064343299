"""The feed-forward block's and the norm's kernels in this build's own gfx950
assembly (CPU only).

The tile kernels accumulate in AGPRs by hand-issued matrix-core instructions:
the wait states in front of every other access are checked as for the GEMMs'
(test_isa_hazards), and none may spill (a register too few has lost part of an
accumulator with this compiler).  The norm defines every float32 operation as
rounded by itself: outside the correctly rounded quotients its kernels hold no
fused multiply-add of float32."""
import os
import re

import pytest

from test_isa_hazards import HIPCC, OUT, _asm, _check, _functions


@pytest.fixture(scope="module")
def tile_asm():
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    os.makedirs(OUT, exist_ok=True)
    return _asm("gemm_mfma16_ffn.hip")


def test_accumulator_reads_follow_the_drain(tile_asm):
    funcs = _functions(tile_asm)
    hand = {n: items for n, items in funcs.items()
            if any(mn and mn.startswith("v_mfma") and h for mn, _, h, _ in items)}
    # four tile shapes, two group sizes, two activations; the down product's
    # two output types and its partial sums for two group sizes
    assert sum("w4a8_ffn_up_kernel" in n for n in hand) == 16
    assert sum("w4a8_ffn_down_kernel" in n for n in hand) == 6
    for name, items in hand.items():
        _, bad = _check(items)
        assert not bad, (name, bad[:4])


def test_tile_kernels_do_not_spill(tile_asm):
    spills = dict(re.findall(r"\.name:\s+(\S*w4a8_ffn_\S*)[\s\S]*?\.vgpr_spill_count:\s+(\d+)",
                             tile_asm))
    assert len(spills) == 22 and set(spills.values()) == {"0"}, spills


def test_norm_has_no_fused_float32_multiply_add():
    """The kernels that quantise hold the fused operations of their quotients
    (v_div_* sequences); in the part of a kernel in front of the first quotient
    there is none.  (float64 sums of exact squares are fused on purpose.)"""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    os.makedirs(OUT, exist_ok=True)
    seen = 0
    for name, items in _functions(_asm("norm.hip")).items():
        if "norm_kernel" not in name:
            continue
        seen += 1
        for mn, _, _, _ in items:
            if not mn:
                continue
            if mn.startswith("v_div_scale_f32"):
                break
            assert not re.match(r"v_(pk_)?(fma|fmac|mad|mac)(ak|mk)?_(mix_?)?f32", mn), (name, mn)
    assert seen >= 48
