// Streamed-tile W4A8 GEMM with low-rank adapters in its epilogue (small M):
// the shared projection's sums leave the workgroup once, with the adapters
// added, instead of passing through memory as int32 to a second launch.
#include "stream_body.h"

namespace w4a8 {

template <int NTW, int D, int GROUP, int RB, int LORA>
__global__ __launch_bounds__(512) void w4a8_stream_lora_kernel(
    const int8_t* __restrict__ X, const float* __restrict__ sx, const uint8_t* __restrict__ wq,
    const uint8_t* __restrict__ s_u8, const uint8_t* __restrict__ a_u8,
    const float* __restrict__ sw, LoraArgs lora, void* __restrict__ Y, int M, int N, int K,
    int ks) {
    stream_body<NTW, D, 0, GROUP, true, kWkLQQ, RB, LORA>(X, sx, wq, s_u8, a_u8, sw, Y, M, N, K, ks,
                                                          nullptr, nullptr, nullptr, lora);
}

namespace {

constexpr size_t kMaxLdsParams = 128 * 1024;  // as the plain kernel's limit

struct Call {
    const int8_t* X;
    const float* sx;
    const uint8_t *wq, *s_u8, *a_u8;
    const float* sw;
    int in_type;
    LoraArgs lora;
    void* Y;
    int M, N, K, group, ks;
    hipStream_t st;
};

template <int NTW, int D, int RB>
hipError_t run(const Call& c) {
    const dim3 grid(c.N / (kTileN * NTW), (c.M + 16 * RB - 1) / (16 * RB)), block(64 * c.ks);
    const size_t pbytes = (size_t)2 * stream_param_span<NTW>() * (c.K / c.group) * 64;
    const size_t used = pbytes + (size_t)c.ks * 2048 * RB;
    const size_t rbytes = (size_t)c.ks * RB * NTW * 256 * sizeof(int);
    if (used > kMaxLdsParams) return hipErrorInvalidConfiguration;
    const size_t lds = used > rbytes ? used : rbytes;
#define STREAM_LORA(G, L)                                                                        \
    hipLaunchKernelGGL((w4a8_stream_lora_kernel<NTW, D, G, RB, L>), grid, block, lds, c.st, c.X, \
                       c.sx, c.wq, c.s_u8, c.a_u8, c.sw, c.lora, c.Y, c.M, c.N, c.K, c.ks)
    if (c.group == 64) {
        if (c.in_type == 1) STREAM_LORA(64, 1); else STREAM_LORA(64, 2);
    } else {
        if (c.in_type == 1) STREAM_LORA(128, 1); else STREAM_LORA(128, 2);
    }
#undef STREAM_LORA
    return hipGetLastError();
}

}  // namespace

bool stream_lora_fits(StreamCfg cfg, int K, int group) {
    const size_t span = (cfg.nt_per_wave + 3) / 4 + 1;
    return 2 * span * (K / group) * 64 + (size_t)cfg.ks * 2048 * cfg.rb <= kMaxLdsParams;
}

hipError_t launch_w4a8_stream_lora(const int8_t* X, const float* sx, const uint8_t* wq,
                                   const uint8_t* s_u8, const uint8_t* a_u8, const float* sw,
                                   int in_type, const LoraArgs& lora, void* Y, int M, int N, int K,
                                   int group, StreamCfg cfg, hipStream_t st) {
    const Call c{X, sx, wq, s_u8, a_u8, sw, in_type, lora, Y, M, N, K, group, cfg.ks, st};
    switch (cfg.nt_per_wave * 8 + cfg.rb) {  // the plain kernel's tiles and ring depths
        case 7 * 8 + 1: return run<7, 2, 1>(c);
        case 4 * 8 + 1: return run<4, 2, 1>(c);
        case 4 * 8 + 2: return run<4, 2, 2>(c);
        case 2 * 8 + 1: return run<2, 4, 1>(c);
        case 2 * 8 + 2: return run<2, 2, 2>(c);
        case 2 * 8 + 4: return run<2, 2, 4>(c);
        case 1 * 8 + 1: return run<1, 3, 1>(c);
        case 1 * 8 + 2: return run<1, 2, 2>(c);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace w4a8
