// The 16 x 16 x 64 tile kernel (mfma16_body.h) for a gated feed-forward block:
// its gate and up products with the activation in the epilogue, and 64-row
// tiles for the few rows between the streamed kernel's and the GEMM's own.
//
// A wave holds the gate and the up sums of the same 32 channels, so act(gate) up
// is formed in registers: 4096 x 57344 x 8192 takes 1454 us (2.65 POP/s, matrix
// cores busy 57 %), 50 of them for the exponential and the quotient of the
// activation; int32 sums written instead took 1486, and a second kernel 320 to
// join them.  64-row tiles are bound by the pace of one workgroup's K-steps (64 x
// 57344 x 8192: 57 us for 242 MB of weights): loads four steps ahead instead of
// two, or eight waves on four K parts, gained 5 %.
#include "mfma16_body.h"

namespace w4a8 {

template <int MT, int GROUP, int KIN, int GLU>
__global__ __launch_bounds__(256, MT <= 128 ? 2 : 1) void w4a8_ffn_up_kernel(
    const int8_t* __restrict__ X, const float* __restrict__ sx, const uint8_t* __restrict__ wq,
    const uint8_t* __restrict__ s_u8, const uint8_t* __restrict__ a_u8,
    const float* __restrict__ sw, FfnRows ffn, int M, int N, int K, int tiles_n, int tiles_m) {
    mfma16_body<MT, 0, GROUP, false, false, KIN, 0, GLU>(X, sx, wq, s_u8, a_u8, sw, nullptr,
                                                         nullptr, M, N, K, tiles_n, tiles_m, 1,
                                                         nullptr, LoraArgs{}, ffn);
}

// 64-row tiles, two K parts; PARTIAL: int32 sums of `splits` parts of K.
template <int OUT, int GROUP, bool PARTIAL>
__global__ __launch_bounds__(256, 2) void w4a8_ffn_down_kernel(
    const int8_t* __restrict__ X, const float* __restrict__ sx, const uint8_t* __restrict__ wq,
    const uint8_t* __restrict__ s_u8, const uint8_t* __restrict__ a_u8,
    const float* __restrict__ sw, void* __restrict__ Y, int* __restrict__ part, int M, int N,
    int K, int tiles_n, int tiles_m, int splits) {
    mfma16_body<64, OUT, GROUP, PARTIAL, false, 2, 0>(X, sx, wq, s_u8, a_u8, sw, Y, part, M, N, K,
                                                      tiles_n, tiles_m, splits, nullptr,
                                                      LoraArgs{});
}

namespace {

template <int MT, int KIN>
void launch_up(const int8_t* X, const float* sx, const uint8_t* wq, const uint8_t* s_u8,
               const uint8_t* a_u8, const float* sw, int act, const FfnRows& out, int M, int F,
               int K, int group, hipStream_t st) {
    const int tiles_n = F / (kNT / 2 / KIN), tiles_m = (M + MT - 1) / MT;
#define UP(G_, A_)                                                                          \
    hipLaunchKernelGGL((w4a8_ffn_up_kernel<MT, G_, KIN, A_>), dim3(tiles_n * tiles_m),      \
                       dim3(256), 0, st, X, sx, wq, s_u8, a_u8, sw, out, M, 2 * F, K, tiles_n, \
                       tiles_m)
    if (group == 64) {
        if (act == 1) UP(64, 2);
        else UP(64, 1);
    } else {
        if (act == 1) UP(128, 2);
        else UP(128, 1);
    }
#undef UP
}

template <int OUT, bool PARTIAL>
void launch_down(const int8_t* X, const float* sx, const uint8_t* wq, const uint8_t* s_u8,
                 const uint8_t* a_u8, const float* sw, void* Y, int* part, int M, int N, int K,
                 int group, int splits, hipStream_t st) {
    const int tiles_n = N / (kNT / 2), tiles_m = (M + 63) / 64;
    const dim3 grid(tiles_n * tiles_m * splits);
    if (group == 64)
        hipLaunchKernelGGL((w4a8_ffn_down_kernel<OUT, 64, PARTIAL>), grid, dim3(256), 0, st, X, sx,
                           wq, s_u8, a_u8, sw, Y, part, M, N, K, tiles_n, tiles_m, splits);
    else
        hipLaunchKernelGGL((w4a8_ffn_down_kernel<OUT, 128, PARTIAL>), grid, dim3(256), 0, st, X, sx,
                           wq, s_u8, a_u8, sw, Y, part, M, N, K, tiles_n, tiles_m, splits);
}

}  // namespace

hipError_t launch_w4a8_ffn_up(const int8_t* X, const float* sx, const uint8_t* wq,
                              const uint8_t* s_u8, const uint8_t* a_u8, const float* sw, int act,
                              float* h, unsigned* tops, int M, int F, int K, int group, int mt,
                              int kin, hipStream_t st) {
    const FfnRows out{h, tops, F / 32};
    if (mt == 256) launch_up<256, 1>(X, sx, wq, s_u8, a_u8, sw, act, out, M, F, K, group, st);
    else if (mt == 128) launch_up<128, 1>(X, sx, wq, s_u8, a_u8, sw, act, out, M, F, K, group, st);
    else if (kin == 1) launch_up<64, 1>(X, sx, wq, s_u8, a_u8, sw, act, out, M, F, K, group, st);
    else launch_up<64, 2>(X, sx, wq, s_u8, a_u8, sw, act, out, M, F, K, group, st);
    return hipGetLastError();
}

hipError_t launch_w4a8_ffn_down64(const int8_t* X, const float* sx, const uint8_t* wq,
                                  const uint8_t* s_u8, const uint8_t* a_u8, const float* sw,
                                  void* Y, int out_type, int M, int N, int K, int group, int splits,
                                  int* part, hipStream_t st) {
    if (splits > 1) {
        launch_down<1, true>(X, sx, wq, s_u8, a_u8, sw, Y, part, M, N, K, group, splits, st);
        return launch_splitk_reduce(part, splits, M, N, sx, sw, Y, out_type, st);
    }
    if (out_type == 2)
        launch_down<2, false>(X, sx, wq, s_u8, a_u8, sw, Y, part, M, N, K, group, 1, st);
    else
        launch_down<0, false>(X, sx, wq, s_u8, a_u8, sw, Y, part, M, N, K, group, 1, st);
    return hipGetLastError();
}

}  // namespace w4a8
