// The streamed-tile W4A8 kernel (stream_body.h) for a gated feed-forward block:
// its gate and up products with the activation in the epilogue, and the down
// product of a few rows that its workgroups quantise themselves.
//
// Bound by the weights' stream: gate and up of 16 rows, 57344 x 8192, 42 us (5.75
// TB/s), of one row of 22016 x 4096 12.5 us (3.9 TB/s: start, end and a wave's four
// K-tiles between them).  Quantising one row inside the down product costs it
// nothing (11008 x 4096: 8.4 us either way) and saves a launch of 3-4 us; with
// four rows it took 12.7 us against 9.8 and the launch.
#include "stream_body.h"

namespace w4a8 {

template <int NTW, int D, int GROUP, bool LDSP, int RB, int GLU>
__global__ __launch_bounds__(512) void w4a8_stream_glu_kernel(
    const int8_t* __restrict__ X, const float* __restrict__ sx, const uint8_t* __restrict__ wq,
    const uint8_t* __restrict__ s_u8, const uint8_t* __restrict__ a_u8,
    const float* __restrict__ sw, FfnRows ffn, int M, int N, int K, int ks) {
    stream_body<NTW, D, 0, GROUP, LDSP, kWkLQQ, RB, 0, GLU>(X, sx, wq, s_u8, a_u8, sw, nullptr, M, N,
                                                            K, ks, nullptr, nullptr, nullptr,
                                                            LoraArgs{}, ffn);
}

template <int NTW, int D, int OUT, int GROUP, bool LDSP, int ROWS>
__global__ __launch_bounds__(512) void w4a8_stream_rows_kernel(
    FfnRows ffn, const uint8_t* __restrict__ wq, const uint8_t* __restrict__ s_u8,
    const uint8_t* __restrict__ a_u8, const float* __restrict__ sw, void* __restrict__ Y, int N,
    int K, int ks) {
    stream_body<NTW, D, OUT, GROUP, LDSP, kWkLQQ, 1, 0, 0, ROWS>(
        nullptr, nullptr, wq, s_u8, a_u8, sw, Y, ROWS, N, K, ks, nullptr, nullptr, nullptr, LoraArgs{},
        ffn);
}

namespace {

template <int NTW, int D, int R>
hipError_t stream_rows(const FfnRows& ffn, const uint8_t* wq, const uint8_t* s_u8,
                       const uint8_t* a_u8, const float* sw, void* Y, int out_type, int N, int K,
                       int group, int ks, hipStream_t st) {
    const dim3 grid(N / (kTileN * NTW)), block(64 * ks);
    const size_t pbytes = (size_t)2 * stream_param_span<NTW>() * (K / group) * 64;
    const size_t xbytes = (size_t)ks * 2048;  // X slots
    const size_t rbytes = (size_t)ks * NTW * 256 * sizeof(int);
    const bool ldsp = pbytes + xbytes <= 128 * 1024;
    const size_t used = (ldsp ? pbytes : 0) + xbytes;
    const size_t lds = used > rbytes ? used : rbytes;
#define ROWS(O, G, P)                                                                        \
    hipLaunchKernelGGL((w4a8_stream_rows_kernel<NTW, D, O, G, P, R>), grid, block, lds, st, \
                       ffn, wq, s_u8, a_u8, sw, Y, N, K, ks)
#define ROWS_GROUP(O, P)                \
    do {                                \
        if (group == 64) ROWS(O, 64, P); \
        else ROWS(O, 128, P);           \
    } while (0)
    if (ldsp) {
        if (out_type == 2) ROWS_GROUP(2, true);
        else ROWS_GROUP(0, true);
    } else {
        if (out_type == 2) ROWS_GROUP(2, false);
        else ROWS_GROUP(0, false);
    }
#undef ROWS_GROUP
#undef ROWS
    return hipGetLastError();
}

template <int NTW, int D, int RB>
hipError_t stream_glu(const int8_t* X, const float* sx, const uint8_t* wq, const uint8_t* s_u8,
                      const uint8_t* a_u8, const float* sw, int act, const FfnRows& ffn, int M,
                      int F, int K, int group, int ks, hipStream_t st) {
    const dim3 grid(F / (kTileN * NTW / 2), (M + 16 * RB - 1) / (16 * RB)), block(64 * ks);
    const size_t pbytes = (size_t)4 * stream_param_span<NTW / 2>() * (K / group) * 64;
    const size_t xbytes = (size_t)ks * 2048 * RB;  // X slots
    const size_t rbytes = (size_t)ks * RB * NTW * 256 * sizeof(int);
    const bool ldsp = pbytes + xbytes <= 128 * 1024;
    const size_t used = (ldsp ? pbytes : 0) + xbytes;
    const size_t lds = used > rbytes ? used : rbytes;
    if (lds > kMaxLdsBytes) return hipErrorInvalidConfiguration;
#define GLU_LS(G, P, A)                                                                         \
    hipLaunchKernelGGL((w4a8_stream_glu_kernel<NTW, D, G, P, RB, A>), grid, block, lds, st, X, \
                       sx, wq, s_u8, a_u8, sw, ffn, M, 2 * F, K, ks)
#define GLU_GROUP(P, A)                     \
    do {                                    \
        if (group == 64) GLU_LS(64, P, A);  \
        else GLU_LS(128, P, A);             \
    } while (0)
    if (ldsp) {
        if (act == 1) GLU_GROUP(true, 2);
        else GLU_GROUP(true, 1);
    } else {
        if (act == 1) GLU_GROUP(false, 2);
        else GLU_GROUP(false, 1);
    }
#undef GLU_GROUP
#undef GLU_LS
    return hipGetLastError();
}

}  // namespace

hipError_t launch_w4a8_stream_rows(const float* h, const unsigned* tops, int ntops,
                                   const uint8_t* wq, const uint8_t* s_u8, const uint8_t* a_u8,
                                   const float* sw, void* Y, int out_type, int M, int N, int K,
                                   int group, StreamCfg cfg, hipStream_t st) {
    const FfnRows ffn{const_cast<float*>(h), const_cast<unsigned*>(tops), ntops};
#define ROWS_NTW(W, D, R) \
    return stream_rows<W, D, R>(ffn, wq, s_u8, a_u8, sw, Y, out_type, N, K, group, cfg.ks, st)
    if (cfg.nt_per_wave == 2) {
        if (M == 1) ROWS_NTW(2, 2, 1);
        ROWS_NTW(2, 2, 2);
    }
    if (M == 1) ROWS_NTW(1, 3, 1);
    ROWS_NTW(1, 3, 2);
#undef ROWS_NTW
}

hipError_t launch_w4a8_stream_glu(const int8_t* X, const float* sx, const uint8_t* wq,
                                  const uint8_t* s_u8, const uint8_t* a_u8, const float* sw,
                                  int act, float* h, unsigned* tops, int M, int F, int K,
                                  int group, StreamCfg cfg, hipStream_t st) {
    const FfnRows ffn{h, tops, F / 16};
#define GLU_NTW(W, D, R)                                                                       \
    return stream_glu<W, D, R>(X, sx, wq, s_u8, a_u8, sw, act, ffn, M, F, K, group, cfg.ks, st)
    switch (cfg.nt_per_wave * 8 + cfg.rb) {
        case 4 * 8 + 1: GLU_NTW(4, 2, 1);
        case 4 * 8 + 2: GLU_NTW(4, 2, 2);
        case 2 * 8 + 1: GLU_NTW(2, 2, 1);
        case 2 * 8 + 2: GLU_NTW(2, 2, 2);
        default: return hipErrorInvalidValue;
    }
#undef GLU_NTW
}

}  // namespace w4a8
