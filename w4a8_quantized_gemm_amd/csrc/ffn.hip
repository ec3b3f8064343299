// Gated feed-forward block on W4A8 weights, between its two products:
//   g, u = the two halves of (Xq . W13^T) sx sw13
//   h    = act(g) u          (float32)
//   hq, sh = per-row INT8 of h
#include "act_common.h"
#include "ffn_common.h"
#include "launch.h"
#include "wave_common.h"

namespace w4a8 {

// One workgroup per row; a thread forms four h at a time, twice: for the row's
// maximum and for the codes.
template <int ACT>
__global__ __launch_bounds__(1024) void ffn_join_kernel(const int* __restrict__ acc, int splits,
                                                        const float* __restrict__ sx,
                                                        const float* __restrict__ sw, int M, int F,
                                                        int8_t* __restrict__ hq,
                                                        float* __restrict__ sh) {
    const size_t m = blockIdx.x, part = (size_t)M * 2 * F;
    const int* row = acc + m * 2 * F;
    const float x = sx[m];
    auto form = [&](int f, float (&h)[4]) {
        v4i g = v4i{0, 0, 0, 0}, u = g;
        for (int s = 0; s < splits; ++s) {
            g += *reinterpret_cast<const v4i*>(row + s * part + f);
            u += *reinterpret_cast<const v4i*>(row + s * part + F + f);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            h[j] = gated<ACT>(((float)g[j] * x) * sw[f + j], ((float)u[j] * x) * sw[F + f + j]);
    };
    unsigned top = 0;
    for (int f = 4 * threadIdx.x; f < F; f += 4 * blockDim.x) {
        float h[4];
        form(f, h);
#pragma unroll
        for (int j = 0; j < 4; ++j) top = MaxU32{}(top, abs_bits(h[j]));
    }
    const float s = row_scale_bits(block_max_bits(top)), inv = __fdiv_rn(1.0f, s);
    if (threadIdx.x == 0) sh[m] = s;
    for (int f = 4 * threadIdx.x; f < F; f += 4 * blockDim.x) {
        float h[4];
        form(f, h);
        *reinterpret_cast<unsigned*>(hq + m * F + f) = quant4_fast(h[0], h[1], h[2], h[3], s, inv);
    }
}

hipError_t launch_ffn_join(const int* acc, int splits, const float* sx, const float* sw13, int M,
                           int F, int act, int8_t* hq, float* sh, hipStream_t st) {
    const dim3 block(F / 4 < 1024 ? (F / 4 + 63) / 64 * 64 : 1024);
    if (act == 1)
        hipLaunchKernelGGL(ffn_join_kernel<1>, dim3(M), block, 0, st, acc, splits, sx, sw13, M, F,
                           hq, sh);
    else
        hipLaunchKernelGGL(ffn_join_kernel<0>, dim3(M), block, 0, st, acc, splits, sx, sw13, M, F,
                           hq, sh);
    return hipGetLastError();
}

}  // namespace w4a8
