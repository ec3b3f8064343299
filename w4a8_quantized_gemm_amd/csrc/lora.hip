// Low-rank adapters of many requests beside a shared W4A8 projection.
//
//   Y[m] = fp16( (acc[m] sx[m]) sw + scale[a] (X[m] . A[a]^T) . B[a]^T ),  a = adapter[m]
//
// acc is the exact int32 product of w4a8_gemm on the INT8 rows of X, the
// adapter's two products are float32 sums over X, A and B as stored, and the
// sum is rounded once.  Rows whose adapter lies outside [0, n) get the
// shared projection alone.
#include "act_common.h"
#include "launch.h"
#include "wave_common.h"

namespace w4a8 {

// V[m][r] = scale[a] sum_k X[m][k] A[a][r][k]: one wave per row and eight
// ranks.
template <int IN>
__global__ __launch_bounds__(256) void lora_shrink_kernel(
    const void* __restrict__ X, const void* __restrict__ A, const int* __restrict__ adapter,
    const float* __restrict__ scale, int n_adapters, int M, int K, int R,
    float* __restrict__ V) {
    const int lane = threadIdx.x & 63;
    const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int chunks = R / 8;
    const int m = (int)(unit / chunks), r0 = (int)(unit % chunks) * 8;
    if (m >= M) return;
    const int a = adapter[m];
    if (a < 0 || a >= n_adapters) return;
    const uint8_t* x = reinterpret_cast<const uint8_t*>(X) + (size_t)m * K * 2;
    const uint8_t* w = reinterpret_cast<const uint8_t*>(A) + ((size_t)a * R + r0) * K * 2;
    float sum[8] = {};
    for (int i = lane; i < K / 8; i += 64) {
        const Row8<IN> xv = load_row8<IN>(x, i);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const Row8<IN> wv = load_row8<IN>(w + (size_t)r * K * 2, i);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[r] = fmaf(xv.v[j], wv.v[j], sum[r]);
        }
    }
    const float s = scale[a];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const float v = wave_sum(sum[r]) * s;
        if (lane == r) V[(size_t)m * R + r0 + r] = v;
    }
}

// The epilogue over int32 sums in memory: one thread per output element.
template <int IN>
__global__ __launch_bounds__(256) void lora_expand_kernel(
    const int* __restrict__ acc, const float* __restrict__ sx, const float* __restrict__ sw,
    const float* __restrict__ V, const void* __restrict__ B, const int* __restrict__ adapter,
    int n_adapters, int N, int R, unsigned short* __restrict__ Y) {
    const int nb = (N + 255) / 256;
    const size_t m = blockIdx.x / nb;
    const int n = (int)(blockIdx.x % nb) * 256 + threadIdx.x;
    if (n >= N) return;
    float y = ((float)acc[m * N + n] * sx[m]) * sw[n];
    const int a = adapter[m];
    if (a >= 0 && a < n_adapters) {
        const uint8_t* b = reinterpret_cast<const uint8_t*>(B) + ((size_t)a * N + n) * R * 2;
        const float* v = V + m * R;
        float d = 0.0f;
        for (int i = 0; i < R / 8; ++i) {
            const Row8<IN> bv = load_row8<IN>(b, i);
#pragma unroll
            for (int j = 0; j < 8; ++j) d = fmaf(v[8 * i + j], bv.v[j], d);
        }
        y += d;
    }
    Y[m * N + n] = f32_to_f16_bits(y);
}

hipError_t launch_lora_shrink(const void* X, int in_type, const void* A, const int* adapter,
                              const float* scale, int n_adapters, int M, int K, int R, float* V,
                              hipStream_t st) {
    const long long units = (long long)M * (R / 8);
    const dim3 grid((unsigned)((units + 3) / 4));
    if (in_type == 1)
        hipLaunchKernelGGL(lora_shrink_kernel<1>, grid, dim3(256), 0, st, X, A, adapter, scale,
                           n_adapters, M, K, R, V);
    else
        hipLaunchKernelGGL(lora_shrink_kernel<2>, grid, dim3(256), 0, st, X, A, adapter, scale,
                           n_adapters, M, K, R, V);
    return hipGetLastError();
}

hipError_t launch_lora_expand(const int* acc, const float* sx, const float* sw, const float* V,
                              int in_type, const void* B, const int* adapter, int n_adapters,
                              int M, int N, int R, void* Y, hipStream_t st) {
    const dim3 grid((unsigned)((size_t)((N + 255) / 256) * M));
    unsigned short* y = reinterpret_cast<unsigned short*>(Y);
    if (in_type == 1)
        hipLaunchKernelGGL(lora_expand_kernel<1>, grid, dim3(256), 0, st, acc, sx, sw, V, B,
                           adapter, n_adapters, N, R, y);
    else
        hipLaunchKernelGGL(lora_expand_kernel<2>, grid, dim3(256), 0, st, acc, sx, sw, V, B,
                           adapter, n_adapters, N, R, y);
    return hipGetLastError();
}

}  // namespace w4a8
