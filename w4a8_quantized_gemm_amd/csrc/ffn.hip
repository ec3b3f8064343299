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

// INT8 of h.  A row's maximum is that of its `ntops` parts; blockIdx.y: part of
// the row (few rows: more workgroups than rows).
__global__ __launch_bounds__(256) void ffn_quant_kernel(const float* __restrict__ h,
                                                        const unsigned* __restrict__ tops,
                                                        int ntops, int F, int8_t* __restrict__ hq,
                                                        float* __restrict__ sh) {
    const size_t m = blockIdx.x;
    unsigned top = 0;
    for (int i = threadIdx.x; i < ntops; i += 256) top = MaxU32{}(top, tops[m * ntops + i]);
    const float s = row_scale_bits(block_max_bits(top)), inv = __fdiv_rn(1.0f, s);
    if (threadIdx.x == 0 && blockIdx.y == 0) sh[m] = s;
    const v4f* row = reinterpret_cast<const v4f*>(h + m * F);
    unsigned* out = reinterpret_cast<unsigned*>(hq + m * F);
    for (int i = blockIdx.y * 256 + threadIdx.x; i < F / 4; i += 256 * gridDim.y) {
        const v4f v = row[i];
        out[i] = quant4_fast(v[0], v[1], v[2], v[3], s, inv);
    }
}

hipError_t launch_ffn_quant(const float* h, const unsigned* tops, int ntops, int M, int F,
                            int8_t* hq, float* sh, hipStream_t st) {
    // about four workgroups per CU, each with four elements a thread at least
    const int most = (F / 4 + 255) / 256;
    int parts = (1024 + M - 1) / M;
    if (parts > most) parts = most;
    hipLaunchKernelGGL(ffn_quant_kernel, dim3(M, parts), dim3(256), 0, st, h, tops, ntops, F, hq,
                       sh);
    return hipGetLastError();
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
