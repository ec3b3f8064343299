"""LDS use of the expert layer's and the adapters' kernels (CPU only), mostly
checked in this build's own gfx950 assembly.

moe_product_kernel keeps the X tiles of its waves and, behind them in time,
the partial sums of all waves in the same LDS bytes, and walks the rows of an
expert in a loop.  A wave that starts the next rows while another still adds
up sums gives wrong results on the GPU only now and then, so the order is
checked here: on every path from a read of the sums (4-byte LDS reads) to a
write of an X tile (16-byte LDS writes) there is a barrier.
"""
import os
import re
import subprocess

import pytest

from test_isa_hazards import CSRC, HIPCC, ROOT, _asm, _blocks, _functions


@pytest.fixture(scope="module")
def kernels():
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    os.makedirs(os.path.join(os.path.dirname(__file__), "sanitize", "_build"), exist_ok=True)
    return {n: items for n, items in _functions(_asm("moe.hip")).items()
            if "moe_product_kernel" in n}


def unordered(items):
    """X-tile writes that a read of the sums reaches without a barrier."""
    blocks, succ = _blocks(items)
    open_read = [False] * len(blocks)  # a read of the sums may be open at entry

    def walk(i):
        state, bad = open_read[i], 0
        for mn, _, _ in blocks[i]:
            if mn == "s_barrier":
                state = False
            elif re.fullmatch(r"ds_read(2|2st64)?_b32", mn):
                state = True
            elif mn.startswith("ds_write") and mn.endswith("b128") and state:
                bad += 1
        return state, bad

    work = list(range(len(blocks)))
    while work:
        i = work.pop()
        if walk(i)[0]:
            for j in succ[i]:
                if not open_read[j]:
                    open_read[j] = True
                    work.append(j)
    return sum(walk(i)[1] for i in range(len(blocks)))


def test_sums_are_read_before_the_next_rows_tiles(kernels):
    assert len(kernels) == 12  # two products, three row-block counts, two group sizes
    for name, items in kernels.items():
        mnemonics = [mn for mn, _, _, _ in items if mn]
        assert any(m.endswith("b128") and m.startswith("ds_write") for m in mnemonics), name
        assert any(re.fullmatch(r"ds_read(2|2st64)?_b32", m) for m in mnemonics), name
        assert unordered(items) == 0, name


def test_adapter_epilogue_lds_is_aligned(tmp_path):
    """The tile kernels' epilogue with adapters reads and writes LDS in pieces
    of 16 bytes: its object, and the arrays in it, are declared so."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    src = tmp_path / "aligned.hip"
    src.write_text('#include "gemm_mfma16.hip"\n#include <cstddef>\n' + "".join(
        f"using L{mt}_{t} = w4a8::LoraLds<{mt}, {t}>;\n"
        f"static_assert(alignof(L{mt}_{t}) % 16 == 0, \"object\");\n"
        f"static_assert(offsetof(L{mt}_{t}, v) % 16 == 0, \"operands\");\n"
        f"static_assert(offsetof(L{mt}_{t}, sw) % 16 == 0, \"scales\");\n"
        for mt in (128, 256) for t in (1, 2)))
    res = subprocess.run(
        [HIPCC, "--offload-arch=gfx950", "-std=c++17", "--offload-device-only", "-fsyntax-only",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src)],
        capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
