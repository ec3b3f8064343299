// The activation of a gated feed-forward block.
#pragma once
#include "act_common.h"

namespace w4a8 {

// act(g) u, ACT 0: SiLU, g / (1 + exp(-g)); 1: GELU in its tanh form, which is
// g / (1 + exp(-z)) with z = g 2 sqrt(2 / pi) (1 + 0.044715 g^2).
// The power and the reciprocal are the hardware's (one unit in the last place
// each); the rounded product z log2(e) moves the power by |z| 2^-24, less than
// the three roundings of g itself do.  A power that overflows gives the
// reciprocal 0, as the quotient would.
template <int ACT>
__device__ __forceinline__ float gated(float g, float u) {
    float z = g;
    if constexpr (ACT == 1) z = g * 1.5957691216057308f * (1.0f + 0.044715f * g * g);
    const float p = __builtin_amdgcn_exp2f(z * -1.4426950408889634f);
    return g * __builtin_amdgcn_rcpf(1.0f + p) * u;
}

// Where the gate and up kernels put h and, per row, the largest |h| of every
// 16 (streamed) or 32 (tile) channels as the bits of a float: the row's
// maximum is known without reading h again, and no workgroup waits for
// another's atomic.
struct FfnRows {
    float* h;         // [M][F]
    unsigned* tops;   // [M][ntops]
    int ntops;        // F / 16 or F / 32
};

}  // namespace w4a8
