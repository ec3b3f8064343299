"""The norm's and the streamed feed-forward kernels in this build's own gfx950
assembly (CPU only): rows held in registers stay there, and no float32
operation of the norm's definition is fused, in any pass of any kernel."""
import os
import re

import pytest

from test_isa_hazards import HIPCC, OUT, _asm

FUSED = re.compile(r"\n\s+v_(?:pk_)?(?:fma|fmac|mad|mac)(?:ak|mk)?_(?:mix_?)?f32\S*")


@pytest.fixture(scope="module")
def asm():
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    os.makedirs(OUT, exist_ok=True)
    return {src: _asm(src) for src in ("norm.hip", "gemm_stream_glu.hip", "ffn.hip")}


@pytest.mark.parametrize("src,kernels", [("norm.hip", 96), ("gemm_stream_glu.hip", 64),
                                         ("ffn.hip", 1)])
def test_no_spills(asm, src, kernels):
    spills = dict(re.findall(r"\.name:\s+(\S+)\n(?:(?!\.name:)[\s\S])*?\.vgpr_spill_count:\s+(\d+)",
                             asm[src]))
    assert len(spills) >= kernels, len(spills)
    assert set(spills.values()) == {"0"}, {k: v for k, v in spills.items() if v != "0"}


def test_norm_fuses_only_quotients_and_code_rounding(asm):
    """Five fused operations in each correctly rounded quotient; two in each INT8
    code's fast form (v inv plus 1.5 2^23, and the distance from it), which falls
    back to the quotient next to a half.  None is left for the definition."""
    bodies = re.findall(r"\n(_ZN4w4a8\S*norm_\S*kernel\S*):[^\n]*\n([\s\S]*?)\n\.Lfunc_end",
                        asm["norm.hip"])
    assert len(bodies) >= 96 and sum("norm_long_kernel" in n for n, _ in bodies) == 12
    for name, body in bodies:
        fused = len(FUSED.findall(body))
        quotients = body.count("v_div_fixup_f32")
        chunks = re.search(r"norm_kernelILi\dELi\w+?ELi(\d)ELi\d+EE", name)
        codes = 8 * int(chunks.group(1) if chunks else 1)  # of a thread, in its code
        assert quotients >= 2 * codes, (name, quotients)   # e4m3's, INT8's slow form
        assert fused == 5 * quotients + 2 * codes, (name, fused, quotients, codes)
