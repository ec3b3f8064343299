"""Size limits of w4a8_route, w4a8_moe and w4a8_gemm_lora (no GPU: every call
below is refused before any HIP call).  A call whose sizes are accepted is
told by the next check it fails, a missing pointer."""
import pytest

from test_selection_abi import NULL, SHAPE, WS, lib, lora, moe, route

w4 = pytest.importorskip("w4a8_quantized_gemm_amd")

# the longest row whose int32 sum of INT8 products is exact for any codes
LONGEST = w4.EXACT_MAX_K


def test_longest_exact_row():
    assert LONGEST % 128 == 0 and 127 * 128 * LONGEST < 1 << 31


@pytest.mark.parametrize("over", [128, 4096, LONGEST])
def test_rows_whose_sums_could_wrap_are_refused(over):
    for bad in (dict(H=LONGEST + over, F=128), dict(H=128, F=LONGEST + over)):
        assert moe(**bad) == SHAPE, bad
        assert lib.w4a8_moe_workspace_size(4, 8, 2, bad["H"], bad["F"]) == 0
    assert lora(K=LONGEST + over) == SHAPE
    assert lib.w4a8_gemm_lora_workspace_size(16, 64, LONGEST + over, 16) == 0


def test_the_longest_rows_are_accepted():
    assert moe(H=LONGEST, F=128, X=None) == NULL
    assert moe(H=128, F=LONGEST, X=None) == NULL
    assert lib.w4a8_moe_workspace_size(4, 8, 2, 128, LONGEST) > 0
    assert lora(K=LONGEST, X=None) == NULL
    assert lib.w4a8_gemm_lora_workspace_size(16, 64, LONGEST, 16) > 0


def test_route_plans_of_the_largest_batches():
    """T * E next to 2^31: the workspace stays within 512 blocks' counts and
    the call is accepted."""
    size = lib.w4a8_route_workspace_size
    most = (1 << 31) - 1
    for E, T in ((1, most), (1, most - (1 << 22)), (2, most // 2), (3, most // 3),
                 (16, most // 16), (512, most // 512)):
        for k in {1, min(E, 16)}:
            assert 0 < size(T, E, k) <= 512 * E * 4, (T, E, k)
            assert route(T=T, E=E, k=k, ws=None) == NULL, (T, E, k)
            assert route(T=T, E=E, k=k, wsb=size(T, E, k) - 1) == WS, (T, E, k)
