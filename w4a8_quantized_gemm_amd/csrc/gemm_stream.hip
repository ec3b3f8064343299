// Streamed-tile W4A8 and W4FP8 GEMM kernels for gfx950 (small M; the
// weight-bandwidth-bound decode path).
//
// Each wave streams packed weight tiles (16 rows x 128 K = 1 KiB, one
// 16-byte load per lane) straight from HBM into registers, dequantises them
// in registers and feeds the matrix cores:
//   W4A8:  (q*s + a) XOR 0x80 per byte, two 16-bit-lane multiply-adds and
//          one XOR per 8 weights after the nibble split (LiquidGEMM, Pith
//          review of arXiv 2509.01229, "What carries the argument" and
//          minor comment 1: paper Eq. 12 and Sec. 5.3), then two
//          v_mfma_i32_16x16x64_i8 per tile;
//   W4FP8: sign-magnitude INT4 -> e4m3 by a byte-table v_perm_b32, then one
//          v_mfma_scale_f32_16x16x128_f8f6f4 per tile with unit scales
//          (FireQ, arXiv 2505.20839, abstract: INT4 weights x FP8
//          activations).
// The activation rows (16 per workgroup, rows >= M read as zero) come from
// L2.  `ks` waves of a workgroup split the K range of the same output tile;
// their partial sums are reduced in LDS in wave order (exact for int32), and
// the per-token x per-channel scale epilogue is fused into the store.
#include "stream_body.h"

namespace w4a8 {

template <int NTW, int D, int OUT, int GROUP, bool LDSP, int WK = kWkLQQ, int RB = 1>
__global__ __launch_bounds__(NTW == 1 && RB == 1 ? 1024 : 512) void w4a8_stream_kernel(
    const int8_t* __restrict__ X, const float* __restrict__ sx, const uint8_t* __restrict__ wq,
    const uint8_t* __restrict__ s_u8, const uint8_t* __restrict__ a_u8,
    const float* __restrict__ sw, void* __restrict__ Y, int M, int N, int K, int ks,
    const int* __restrict__ offsets, const float* __restrict__ fsc = nullptr,
    const float* __restrict__ tsc = nullptr) {
    stream_body<NTW, D, OUT, GROUP, LDSP, WK, RB, 0>(X, sx, wq, s_u8, a_u8, sw, Y, M, N, K, ks,
                                                     offsets, fsc, tsc, LoraArgs{});
}

// ----------------------------------------------------------- launchers ----
template <int NTW, int D, int RB = 1>
static hipError_t w4a8_stream_ntw(const int8_t* X, const float* sx, const uint8_t* wq,
                                  const uint8_t* s_u8, const uint8_t* a_u8, const float* sw,
                                  void* Y, int out_type, int M, int N, int K, int group, int ks,
                                  const int* offsets, int E, int max_rows, hipStream_t st) {
    dim3 grid(N / (kTileN * NTW), (max_rows + 16 * RB - 1) / (16 * RB), E);
    dim3 block(64 * ks);
    const int groups = K / group;
    const size_t pbytes = (size_t)2 * stream_param_span<NTW>() * groups * 64;
    const size_t xbytes = (size_t)ks * 2048 * RB;  // X slots
    const size_t rbytes = (size_t)ks * RB * NTW * 256 * sizeof(int);
    const bool ldsp = pbytes + xbytes <= 128 * 1024;
    const size_t used = (ldsp ? pbytes : 0) + xbytes;
    const size_t lds = used > rbytes ? used : rbytes;
    if (lds > kMaxLdsBytes) return hipErrorInvalidConfiguration;
#define W4A8_LS(O, G, P)                                                                    \
    hipLaunchKernelGGL((w4a8_stream_kernel<NTW, D, O, G, P, kWkLQQ, RB>), grid, block, lds, \
                       st, X, sx, wq, s_u8, a_u8, sw, Y, M, N, K, ks, offsets)
#define W4A8_LS_GROUP(O, P)                                             \
    do {                                                                \
        if (group == 64) W4A8_LS(O, 64, P); else W4A8_LS(O, 128, P);    \
    } while (0)
    if (out_type == 2) {
        // (the feed-forward block's down product, which takes no wider forms)
        if constexpr (NTW <= 4 && RB <= 2) {
            if (ldsp) W4A8_LS_GROUP(2, true); else W4A8_LS_GROUP(2, false);
        } else {
            return hipErrorInvalidValue;
        }
    } else if (ldsp) {
        if (out_type == 1) W4A8_LS_GROUP(1, true); else W4A8_LS_GROUP(0, true);
    } else {
        if (out_type == 1) W4A8_LS_GROUP(1, false); else W4A8_LS_GROUP(0, false);
    }
#undef W4A8_LS_GROUP
#undef W4A8_LS
    return hipGetLastError();
}

hipError_t launch_w4a8_stream(const int8_t* X, const float* sx, const uint8_t* wq,
                              const uint8_t* s_u8, const uint8_t* a_u8, const float* sw,
                              void* Y, int out_type, int M, int N, int K, int group,
                              StreamCfg cfg, hipStream_t st, const int* offsets, int E,
                              int max_rows) {
    if (!offsets) {
        E = 1;
        max_rows = M;
    }
#define W4A8_NTW(W, D, R)                                                                    \
    return w4a8_stream_ntw<W, D, R>(X, sx, wq, s_u8, a_u8, sw, Y, out_type, M, N, K, group, \
                                    cfg.ks, offsets, E, max_rows, st)
    // several 16-row blocks per workgroup share each decoded weight (ring
    // of two K-tiles: the X operands of every block are held per stage;
    // four blocks of four tiles would not fit the registers)
    switch (cfg.nt_per_wave * 8 + cfg.rb) {
        case 7 * 8 + 1: W4A8_NTW(7, 2, 1);
        case 4 * 8 + 1: W4A8_NTW(4, 2, 1);
        case 4 * 8 + 2: W4A8_NTW(4, 2, 2);
        case 2 * 8 + 1: W4A8_NTW(2, 4, 1);
        case 2 * 8 + 2: W4A8_NTW(2, 2, 2);
        case 2 * 8 + 4: W4A8_NTW(2, 2, 4);
        case 1 * 8 + 1: W4A8_NTW(1, 3, 1);
        case 1 * 8 + 2: W4A8_NTW(1, 2, 2);
        default: return hipErrorInvalidValue;
    }
#undef W4A8_NTW
}

template <int NTW, int D>
static hipError_t w8a8_stream_ntw(const int8_t* X, const float* sx, const int8_t* wq8,
                                  const float* sw, void* Y, int out_type, int M, int N, int K,
                                  int ks, hipStream_t st) {
    dim3 grid(N / (kTileN * NTW), (M + 15) / 16, 1);
    dim3 block(64 * ks);
    const size_t xbytes = (size_t)ks * 2048;
    const size_t rbytes = (size_t)ks * NTW * 256 * sizeof(int);
    const size_t lds = xbytes > rbytes ? xbytes : rbytes;
    const uint8_t* w = reinterpret_cast<const uint8_t*>(wq8);
    if (out_type == 1)
        hipLaunchKernelGGL((w4a8_stream_kernel<NTW, D, 1, 128, false, kWkW8>), grid, block, lds, st,
                           X, sx, w, nullptr, nullptr, sw, Y, M, N, K, ks, nullptr);
    else
        hipLaunchKernelGGL((w4a8_stream_kernel<NTW, D, 0, 128, false, kWkW8>), grid, block, lds, st,
                           X, sx, w, nullptr, nullptr, sw, Y, M, N, K, ks, nullptr);
    return hipGetLastError();
}

hipError_t launch_w8a8_stream(const int8_t* X, const float* sx, const int8_t* wq8,
                              const float* sw, void* Y, int out_type, int M, int N, int K,
                              StreamCfg cfg, hipStream_t st) {
    switch (cfg.nt_per_wave) {
        case 7: return w8a8_stream_ntw<7, 2>(X, sx, wq8, sw, Y, out_type, M, N, K, cfg.ks, st);
        case 4: return w8a8_stream_ntw<4, 3>(X, sx, wq8, sw, Y, out_type, M, N, K, cfg.ks, st);
        case 2: return w8a8_stream_ntw<2, 4>(X, sx, wq8, sw, Y, out_type, M, N, K, cfg.ks, st);
        default: return w8a8_stream_ntw<1, 3>(X, sx, wq8, sw, Y, out_type, M, N, K, cfg.ks, st);
    }
}

template <int NTW, int D, int WK, int GROUP, int RB = 1>
static hipError_t w4fp8_stream_ntw(const uint8_t* X, const float* sx, const uint8_t* wq,
                                   const float* sw, const float* fsc, const float* tsc, void* Y,
                                   int out_type, int M, int N, int K, int ks, hipStream_t st) {
    dim3 grid(N / (kTileN * NTW), (M + 16 * RB - 1) / (16 * RB), 1);
    dim3 block(64 * ks);
    const size_t xbytes = (size_t)ks * 2048 * RB;
    const size_t rbytes = (size_t)ks * RB * NTW * 256 * sizeof(float);
    const size_t lds = xbytes > rbytes ? xbytes : rbytes;
    if (lds > kMaxLdsBytes) return hipErrorInvalidConfiguration;
    const int8_t* Xb = reinterpret_cast<const int8_t*>(X);
    if (out_type == 1)
        hipLaunchKernelGGL((w4a8_stream_kernel<NTW, D, 1, GROUP, false, WK, RB>), grid, block, lds,
                           st, Xb, sx, wq, nullptr, nullptr, sw, Y, M, N, K, ks, nullptr, fsc, tsc);
    else
        hipLaunchKernelGGL((w4a8_stream_kernel<NTW, D, 0, GROUP, false, WK, RB>), grid, block, lds,
                           st, Xb, sx, wq, nullptr, nullptr, sw, Y, M, N, K, ks, nullptr, fsc, tsc);
    return hipGetLastError();
}

template <int WK, int GROUP>
static hipError_t w4fp8_stream_run(const uint8_t* X, const float* sx, const uint8_t* wq,
                                   const float* sw, const float* fsc, const float* tsc, void* Y,
                                   int out_type, int M, int N, int K, StreamCfg cfg,
                                   hipStream_t st) {
#define F8_NTW(W, D, R)                                                                          \
    return w4fp8_stream_ntw<W, D, WK, GROUP, R>(X, sx, wq, sw, fsc, tsc, Y, out_type, M, N, K, \
                                                cfg.ks, st)
    switch (cfg.nt_per_wave * 8 + cfg.rb) {
        case 7 * 8 + 1: F8_NTW(7, 2, 1);
        case 4 * 8 + 1: F8_NTW(4, 2, 1);
        case 4 * 8 + 2: F8_NTW(4, 2, 2);
        case 2 * 8 + 1: F8_NTW(2, 4, 1);
        case 2 * 8 + 2: F8_NTW(2, 2, 2);
        case 2 * 8 + 4: F8_NTW(2, 2, 4);
        case 1 * 8 + 1: F8_NTW(1, 3, 1);
        case 1 * 8 + 2: F8_NTW(1, 2, 2);
        default: return hipErrorInvalidValue;
    }
#undef F8_NTW
}

hipError_t launch_w4fp8_stream(const uint8_t* X, const float* sx, const uint8_t* wq,
                               const float* sw, void* Y, int out_type, int M, int N, int K,
                               StreamCfg cfg, hipStream_t st) {
    return w4fp8_stream_run<kWkF8, 128>(X, sx, wq, sw, nullptr, nullptr, Y, out_type, M, N, K,
                                        cfg, st);
}

hipError_t launch_w4fp8g_stream(const uint8_t* X, const float* sx, const uint8_t* wq,
                                const float* fsc, const float* tsc, void* Y, int out_type, int M,
                                int N, int K, int group, StreamCfg cfg, hipStream_t st) {
    if (group == 64)
        return w4fp8_stream_run<kWkF8G, 64>(X, sx, wq, nullptr, fsc, tsc, Y, out_type, M, N, K,
                                            cfg, st);
    return w4fp8_stream_run<kWkF8G, 128>(X, sx, wq, nullptr, fsc, tsc, Y, out_type, M, N, K, cfg,
                                         st);
}

}  // namespace w4a8
