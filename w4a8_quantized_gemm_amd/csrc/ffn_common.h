// The activation of a gated feed-forward block.
#pragma once
#include <hip/hip_runtime.h>

namespace w4a8 {

// act(g) u, ACT 0: SiLU, g / (1 + exp(-g)); 1: GELU in its tanh form, which is
// g / (1 + exp(-z)) with z = g 2 sqrt(2 / pi) (1 + 0.044715 g^2).
template <int ACT>
__device__ __forceinline__ float gated(float g, float u) {
    float z = g;
    if constexpr (ACT == 1) z = g * 1.5957691216057308f * (1.0f + 0.044715f * g * g);
    return g / (1.0f + expf(-z)) * u;
}

}  // namespace w4a8
