// Host code of w4a8_norm_quant and w4a8_ffn over sizes up to their limits, with
// UndefinedBehaviorSanitizer on api.hip and the tile plans of gemm_mfma.hip.
// Valid calls stop at the HIP runtime, which finds no GPU; the launchers are
// not linked.  Test infrastructure: only tests/test_layer_sanitizers.py builds
// and runs it.
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "w4a8.h"

int main() {
    int fails = 0;
    auto* p = reinterpret_cast<void*>(uintptr_t(0x10000));
    auto* b = reinterpret_cast<uint8_t*>(p);
    auto* f = reinterpret_cast<float*>(p);
    const long long limit = (1LL << 31) - 1;
    auto stopped = [&](w4a8_status_t s) { return s == W4A8_ERR_HIP || s == W4A8_ERR_UNSUPPORTED; };
    for (int H : {128, 256, 384, 2048, 4096, 8192, 131072})
        for (int F : {128, 640, 1408, 11008, 28672, 131072})
            for (long long M : {1LL, 2LL, 3LL, 16LL, 17LL, 32LL, 33LL, 64LL, 65LL, 128LL, 129LL,
                                300LL, 4096LL, 65536LL, limit / (H > F ? H : F)}) {
                if (M > limit / H || M > limit / F) continue;
                const bool valid = 2LL * H * F < (1LL << 32);
                const size_t ws = w4a8_ffn_workspace_size((int)M, H, F);
                // h, its codes and scales at least; partial sums for at most 512
                // workgroups of 64 x 128
                const size_t least = (size_t)M * F * 5 + 4 * (size_t)M;
                const size_t most = least + (size_t)M * (F / 16) * 4 + (64u << 20) + 4096;
                if (valid ? (ws < least || ws > most) : ws != 0) {
                    std::fprintf(stderr, "M %lld H %d F %d: workspace %zu\n", M, H, F, ws);
                    ++fails;
                }
                for (int act : {W4A8_ACT_SILU, W4A8_ACT_GELU}) {
                    const w4a8_status_t s =
                        w4a8_ffn(reinterpret_cast<int8_t*>(p), f, b, b, b, f, b, b, b, f, act, p,
                                 W4A8_IN_BF16, (int)M, H, F, 64, p, ws, nullptr);
                    if (valid ? !stopped(s) : s != W4A8_ERR_SHAPE) {
                        std::fprintf(stderr, "M %lld H %d F %d: status %d\n", M, H, F, (int)s);
                        ++fails;
                    }
                }
            }
    for (int K : {16, 4096, 1 << 20, (1 << 30) + 16})
        for (int M : {1, 256, 257, (1 << 22) - 1})
            for (int out = W4A8_NORM_OUT_F32; out <= W4A8_NORM_OUT_E4M3; ++out) {
                const w4a8_status_t s =
                    w4a8_norm_quant(p, W4A8_IN_BF16, p, W4A8_IN_F16, f, f, p, 1,
                                    reinterpret_cast<int32_t*>(p), 1.0f, -0.5f, f, f,
                                    W4A8_NORM_LAYER, 1e-5f, p, p, out, f, M, K, nullptr);
                if (!stopped(s)) {
                    std::fprintf(stderr, "norm M %d K %d: status %d\n", M, K, (int)s);
                    ++fails;
                }
            }
    std::printf("layer plans: %d failures\n", fails);
    return fails != 0;
}
