// Gated feed-forward block on W4A8 weights, between its two products: the
// per-row INT8 of h = act(gate) up.
#include "act_common.h"
#include "launch.h"

namespace w4a8 {

// INT8 of h.  A row's maximum is that of its `ntops` parts, so h is read once;
// blockIdx.y: part of the row (few rows: more workgroups than rows).  Bound by
// memory: 4096 x 28672 float32 in 116 us, 5.1 TB/s, a copy's rate.  h stays in
// float32: rounded to 16 bits first, one code in a few hundred would fall on the
// other side of a half.
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

}  // namespace w4a8
