"""Values, sizes and kernels at the borders of the norm with quantisation and of
the gated feed-forward block, on the GPU (references: layer_refs.py)."""
import numpy as np
import pytest

import layer_refs as ref
import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a8_quantized_gemm_amd as w4  # noqa: E402
from test_gpu_layer import same_bits  # noqa: E402
from test_gpu_selection import DEV, say  # noqa: E402


def subnormal_rows(K):
    """Rows of subnormal float32 values: the largest is m smallest subnormals, so
    the scale is a whole number of them and max / scale is not the codes' top
    (667 / 1 against 448, 190 / 1 against 127)."""
    tops = [1, 3, 63, 64, 190, 191, 224, 225, 465, 600, 667, 671, 672, 928, 929, 1000, 1119, 1121,
            2500, 5000, 100003, 8000009]
    rng = np.random.default_rng(K)
    x = np.zeros((len(tops), K), np.int32)
    for i, m in enumerate(tops):
        x[i] = rng.integers(-m, m + 1, K)
        x[i, rng.integers(K)] = m * (-1) ** i
    return np.copysign(np.abs(x).view(np.float32), x.astype(np.float32))


@pytest.mark.parametrize("K", [48, 5008, 33024])
def test_subnormal_rows(K):
    """Quotients past the codes' range saturate: no code of a finite row is NaN."""
    x = subnormal_rows(K)
    dx = torch.from_numpy(x).to(DEV)
    for many in (False, True):
        reps = 20 if many else 1
        d, r = dx.repeat(reps, 1), np.tile(x, (reps, 1))
        for out, quant in (("int8", w4.quant_act), ("e4m3", w4.quant_act_fp8)):
            say(f"subnormal rows K={K} {out} x{reps}")
            q, s = ref.codes(r, out)
            got = w4.norm_quant(d, out_type=getattr(w4, "NORM_OUT_" + out.upper()))
            same_bits(got["sx"], s)
            same_bits(got["out"], q)
            codes, scales = quant(d)
            same_bits(scales, s)
            same_bits(codes, q)
            if out == "e4m3":
                assert np.abs(oracle.e4m3_decode(q)).max() == 448.0
