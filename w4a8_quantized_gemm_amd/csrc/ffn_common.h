// The activation of a gated feed-forward block.
#pragma once
#include "act_common.h"

namespace w4a8 {

// act(g) u, ACT 0: SiLU, g / (1 + exp(-g)); 1: GELU in its tanh form, which is
// g / (1 + exp(-z)) with z = g 2 sqrt(2 / pi) (1 + 0.044715 g^2).  The exponential
// is good to one unit in the last place whatever z is, and the quotient is
// rounded once, as in the expert layer (the hardware's power of the rounded
// product z log2(e) is off by up to |z| 2^-24 of itself).
template <int ACT>
__device__ __forceinline__ float gated(float g, float u) {
    float z = g;
    if constexpr (ACT == 1) z = g * 1.5957691216057308f * (1.0f + 0.044715f * g * g);
    return g / (1.0f + expf(-z)) * u;
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
