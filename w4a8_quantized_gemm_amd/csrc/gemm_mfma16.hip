// Large-M W4A8 and W8A8 GEMM kernels for gfx950 on v_mfma_i32_16x16x64_i8, and
// the W4A8 ones with low-rank adapters in their epilogue (mfma16_body.h).
#include "mfma16_body.h"

namespace w4a8 {

template <int MT, int OUT, int GROUP, bool PARTIAL, bool W8, int KIN>
__global__ __launch_bounds__(256, (MT == 128 && KIN == 1) ? 2 : 1) void w4a8_mfma16_kernel(
    const int8_t* __restrict__ X, const float* __restrict__ sx, const uint8_t* __restrict__ wq,
    const uint8_t* __restrict__ s_u8, const uint8_t* __restrict__ a_u8,
    const float* __restrict__ sw, void* __restrict__ Y, int* __restrict__ part, int M, int N,
    int K, int tiles_n, int tiles_m, int splits, const int* __restrict__ offsets) {
    mfma16_body<MT, OUT, GROUP, PARTIAL, W8, KIN, 0>(X, sx, wq, s_u8, a_u8, sw, Y, part, M, N, K,
                                                     tiles_n, tiles_m, splits, offsets,
                                                     LoraArgs{});
}

// The unsplit fp16 kernel with the adapters in its epilogue.
template <int MT, int GROUP, int LORA>
__global__ __launch_bounds__(256, MT == 128 ? 2 : 1) void w4a8_mfma16_lora_kernel(
    const int8_t* __restrict__ X, const float* __restrict__ sx, const uint8_t* __restrict__ wq,
    const uint8_t* __restrict__ s_u8, const uint8_t* __restrict__ a_u8,
    const float* __restrict__ sw, LoraArgs lora, void* __restrict__ Y, int M, int N, int K,
    int tiles_n, int tiles_m) {
    mfma16_body<MT, 0, GROUP, false, false, 1, LORA>(X, sx, wq, s_u8, a_u8, sw, Y, nullptr, M, N,
                                                     K, tiles_n, tiles_m, 1, nullptr, lora);
}

template <int MT, int OUT, bool PARTIAL, bool W8, int KIN = 1>
static void launch_tile16(const int8_t* X, const float* sx, const uint8_t* wq,
                          const uint8_t* s_u8, const uint8_t* a_u8, const float* sw, void* Y,
                          int* part, int M, int N, int K, int group, int splits, hipStream_t st,
                          const int* offsets, int E, int max_rows) {
    const int tiles_n = N / (kNT / KIN);
    const int tiles_m = ((offsets ? max_rows : M) + MT - 1) / MT;
    dim3 grid(tiles_n * tiles_m * splits, offsets ? E : 1), block(256);
    if (group == 64 && !W8)
        hipLaunchKernelGGL((w4a8_mfma16_kernel<MT, OUT, 64, PARTIAL, W8, KIN>), grid, block, 0,
                           st, X, sx, wq, s_u8, a_u8, sw, Y, part, M, N, K, tiles_n, tiles_m,
                           splits, offsets);
    else
        hipLaunchKernelGGL((w4a8_mfma16_kernel<MT, OUT, 128, PARTIAL, W8, KIN>), grid, block, 0,
                           st, X, sx, wq, s_u8, a_u8, sw, Y, part, M, N, K, tiles_n, tiles_m,
                           splits, offsets);
}

template <bool W8>
static hipError_t run_mfma16(const int8_t* X, const float* sx, const uint8_t* wq,
                             const uint8_t* s_u8, const uint8_t* a_u8, const float* sw, void* Y,
                             int out_type, int M, int N, int K, int group, const MfmaPlan& plan,
                             void* workspace, hipStream_t st, const int* offsets, int E,
                             int max_rows) {
    int* part = reinterpret_cast<int*>(workspace);
    if (plan.kin == 2) {  // 128-row tiles, no grouped problems
        if (plan.splits == 1) {
            if (out_type == 1)
                launch_tile16<128, 1, false, W8, 2>(X, sx, wq, s_u8, a_u8, sw, Y, part, M, N, K,
                                                    group, 1, st, nullptr, 1, 0);
            else if (!W8 && out_type == 2)
                launch_tile16<128, 2, false, false, 2>(X, sx, wq, s_u8, a_u8, sw, Y, part, M, N, K,
                                                       group, 1, st, nullptr, 1, 0);
            else
                launch_tile16<128, 0, false, W8, 2>(X, sx, wq, s_u8, a_u8, sw, Y, part, M, N, K,
                                                    group, 1, st, nullptr, 1, 0);
            return hipGetLastError();
        }
        launch_tile16<128, 1, true, W8, 2>(X, sx, wq, s_u8, a_u8, sw, Y, part, M, N, K, group,
                                           plan.splits, st, nullptr, 1, 0);
        return launch_splitk_reduce(part, plan.splits, M, N, sx, sw, Y, out_type, st);
    }
    if (plan.splits == 1) {
#define T16(MT_, O_, W_) \
    launch_tile16<MT_, O_, false, W_>(X, sx, wq, s_u8, a_u8, sw, Y, part, M, N, K, group, 1, st, \
                                      offsets, E, max_rows)
        if (plan.mt == 256) {
            if (out_type == 1) T16(256, 1, W8);
            else if (!W8 && out_type == 2) T16(256, 2, false);
            else T16(256, 0, W8);
        } else {
            if (out_type == 1) T16(128, 1, W8);
            else if (!W8 && out_type == 2) T16(128, 2, false);
            else T16(128, 0, W8);
        }
#undef T16
        return hipGetLastError();
    }
    if (plan.mt == 256)
        launch_tile16<256, 1, true, W8>(X, sx, wq, s_u8, a_u8, sw, Y, part, M, N, K, group,
                                        plan.splits, st, nullptr, 1, 0);
    else
        launch_tile16<128, 1, true, W8>(X, sx, wq, s_u8, a_u8, sw, Y, part, M, N, K, group,
                                        plan.splits, st, nullptr, 1, 0);
    return launch_splitk_reduce(part, plan.splits, M, N, sx, sw, Y, out_type, st);
}

hipError_t launch_w4a8_mfma16(const int8_t* X, const float* sx, const uint8_t* wq,
                              const uint8_t* s_u8, const uint8_t* a_u8, const float* sw, void* Y,
                              int out_type, int M, int N, int K, int group, const MfmaPlan& plan,
                              void* workspace, hipStream_t st, const int* offsets, int E,
                              int max_rows) {
    return run_mfma16<false>(X, sx, wq, s_u8, a_u8, sw, Y, out_type, M, N, K, group, plan,
                             workspace, st, offsets, E, max_rows);
}

hipError_t launch_w4a8_mfma16_partial(const int8_t* X, const uint8_t* wq, const uint8_t* s_u8,
                                      const uint8_t* a_u8, int M, int N, int K, int group,
                                      const MfmaPlan& plan, int* part, hipStream_t st) {
    if (plan.mt == 256)
        launch_tile16<256, 1, true, false>(X, nullptr, wq, s_u8, a_u8, nullptr, nullptr, part, M,
                                           N, K, group, plan.splits, st, nullptr, 1, 0);
    else
        launch_tile16<128, 1, true, false>(X, nullptr, wq, s_u8, a_u8, nullptr, nullptr, part, M,
                                           N, K, group, plan.splits, st, nullptr, 1, 0);
    return hipGetLastError();
}

namespace {

template <int MT, int GROUP, int LORA>
void launch_tile16_lora(const int8_t* X, const float* sx, const uint8_t* wq, const uint8_t* s_u8,
                        const uint8_t* a_u8, const float* sw, const LoraArgs& lora, void* Y, int M,
                        int N, int K, hipStream_t st) {
    const int tiles_n = N / kNT, tiles_m = (M + MT - 1) / MT;
    hipLaunchKernelGGL((w4a8_mfma16_lora_kernel<MT, GROUP, LORA>), dim3(tiles_n * tiles_m),
                       dim3(256), 0, st, X, sx, wq, s_u8, a_u8, sw, lora, Y, M, N, K, tiles_n,
                       tiles_m);
}

}  // namespace

hipError_t launch_w4a8_mfma16_lora(const int8_t* X, const float* sx, const uint8_t* wq,
                                   const uint8_t* s_u8, const uint8_t* a_u8, const float* sw,
                                   int in_type, const LoraArgs& lora, void* Y, int M, int N, int K,
                                   int group, int mt, hipStream_t st) {
#define T16_LORA(MT_, G_, L_) \
    launch_tile16_lora<MT_, G_, L_>(X, sx, wq, s_u8, a_u8, sw, lora, Y, M, N, K, st)
#define T16_LORA_TYPE(MT_, G_)             \
    do {                                   \
        if (in_type == 1) T16_LORA(MT_, G_, 1); \
        else T16_LORA(MT_, G_, 2);         \
    } while (0)
    if (mt == 256) {
        if (group == 64) T16_LORA_TYPE(256, 64);
        else T16_LORA_TYPE(256, 128);
    } else {
        if (group == 64) T16_LORA_TYPE(128, 64);
        else T16_LORA_TYPE(128, 128);
    }
#undef T16_LORA_TYPE
#undef T16_LORA
    return hipGetLastError();
}

hipError_t launch_w8a8_mfma16(const int8_t* X, const float* sx, const int8_t* wq8,
                              const float* sw, void* Y, int out_type, int M, int N, int K,
                              const MfmaPlan& plan, void* workspace, hipStream_t st) {
    return run_mfma16<true>(X, sx, reinterpret_cast<const uint8_t*>(wq8), nullptr, nullptr, sw,
                            Y, out_type, M, N, K, 128, plan, workspace, st, nullptr, 1, 0);
}

}  // namespace w4a8
