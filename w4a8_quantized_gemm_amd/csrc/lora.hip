// Low-rank adapters of many requests beside a shared W4A8 projection.
//
//   Y[m] = fp16( (acc[m] sx[m]) sw + scale[a] (X[m] . A[a]^T) . B[a]^T ),  a = adapter[m]
//
// acc is the exact int32 product of w4a8_gemm on the INT8 rows of X, the
// adapter's two products are float32 sums over A, B and X as stored, and the
// sum is rounded once.  Rows whose adapter lies outside [0, n) get the
// shared projection alone.
//
// This file: the inner product V = scale (X . A^T), with the quantisation of
// X in the same launch for small calls, and the epilogue of projections
// whose int32 sums (one or several K parts) lie in memory.
#include "act_common.h"
#include "launch.h"
#include "lora_common.h"
#include "wave_common.h"

namespace w4a8 {

namespace {
constexpr int kRanksPerGroup = 4;  // ranks of one workgroup of the small kernel
}

// Inner product of one row and four ranks by a workgroup of 16 waves: wave w
// takes rank w % 4 and the (w / 4)-th quarter of K, so a short row's loads
// are all in flight at once; the quarters are added in order.
template <int IN>
__device__ __forceinline__ void shrink_row(const void* X, const void* A, int m, int a, float scale,
                                           int K, int R, int r0, float* V) {
    __shared__ float part[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint8_t* x = reinterpret_cast<const uint8_t*>(X) + (size_t)m * K * 2;
    const uint8_t* w =
        reinterpret_cast<const uint8_t*>(A) + ((size_t)a * R + r0 + (wave & 3)) * K * 2;
    float sum = 0.0f;
    const int n8 = K / 8;
    // two partial sums per lane keep the chain short
    float sum1 = 0.0f;
    for (int i = (wave >> 2) * 64 + lane; i < n8; i += 256) {
        const Row8<IN> xv = load_row8<IN>(x, i), wv = load_row8<IN>(w, i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sum = fmaf(xv.v[j], wv.v[j], sum);
            sum1 = fmaf(xv.v[4 + j], wv.v[4 + j], sum1);
        }
    }
    const float v = wave_sum(sum + sum1);
    if (lane == 0) part[wave] = v;
    __syncthreads();
    if (threadIdx.x < kRanksPerGroup) {
        const int r = threadIdx.x;
        V[(size_t)m * R + r0 + r] = (part[r] + part[4 + r] + (part[8 + r] + part[12 + r])) * scale;
    }
}

// Workgroups b < M quantise row b (CH > 0: the row in registers), the others
// take a row and four ranks each.
template <int IN, int CH>
__global__ __launch_bounds__(1024) void lora_inputs_kernel(
    const void* __restrict__ X, const void* __restrict__ A, const int* __restrict__ adapter,
    const float* __restrict__ scale, int n_adapters, int M, int K, int R,
    uint8_t* __restrict__ Xq, float* __restrict__ sx, float* __restrict__ V) {
    int b = blockIdx.x;
    if constexpr (CH > 0) {
        if (b < M) {
            quant_row_regs<IN, 0, CH, 1024>(reinterpret_cast<const uint8_t*>(X) + (size_t)b * K * 2,
                                            K, Xq + (size_t)b * K, sx + b);
            return;
        }
        b -= M;
    }
    const int per_row = R / kRanksPerGroup;
    const int m = b / per_row, r0 = (b % per_row) * kRanksPerGroup;
    const int a = adapter[m];
    if (a < 0 || a >= n_adapters) return;
    shrink_row<IN>(X, A, m, a, scale[a], K, R, r0, V);
}

// Epilogue over int32 sums in memory (`splits` parts of M x N, added in
// order): a wave takes 16 rows and 64 channels.
template <int IN>
__global__ __launch_bounds__(256) void lora_join_kernel(const int* __restrict__ acc, int splits,
                                                        const float* __restrict__ sx,
                                                        const float* __restrict__ sw, LoraArgs L,
                                                        int M, int N,
                                                        unsigned short* __restrict__ Y) {
    const int lane = threadIdx.x & 63, r = lane & 15, G = lane >> 4;
    const int panels = N / 64;
    const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int m = (int)(unit / panels) * 16 + r, n0 = (int)(unit % panels) * 64;
    if ((int)(unit / panels) * 16 >= M) return;
    const bool live = m < M;
    const int id = lora_id(L, m, live);
    v4i sum[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) sum[c] = v4i{0, 0, 0, 0};
    if (live)
        for (int p = 0; p < splits; ++p)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                sum[c] += load16(acc + ((size_t)p * M + m) * N + n0 + 16 * c + 4 * G);
    const float s = live ? sx[m] : 0.0f;
    v4f delta[4];
    lora_block<IN, 4>(L, m, id, N, n0, delta);
    if (!live) return;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int n = n0 + 16 * c + 4 * G;
        unsigned short h[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const float y = ((float)sum[c][v] * s) * sw[n + v];
            h[v] = f32_to_f16_bits(id >= 0 ? y + delta[c][v] : y);
        }
        *reinterpret_cast<uint2*>(Y + (size_t)m * N + n) =
            uint2{h[0] | ((unsigned)h[1] << 16), h[2] | ((unsigned)h[3] << 16)};
    }
}

namespace {

template <int IN>
hipError_t inputs_run(const void* X, const void* A, const int* adapter, const float* scale,
                      int n_adapters, int M, int K, int R, int8_t* Xq, float* sx, float* V,
                      hipStream_t st) {
    const int shrink = n_adapters > 0 ? M * (R / kRanksPerGroup) : 0;
    uint8_t* q = reinterpret_cast<uint8_t*>(Xq);
#define INPUTS(CH, G)                                                                        \
    hipLaunchKernelGGL((lora_inputs_kernel<IN, CH>), dim3(G), dim3(1024), 0, st, X, A, adapter, \
                       scale, n_adapters, M, K, R, q, sx, V)
    const int ch = (K / 8 + 1023) / 1024;
    if (M < 256 && ch <= 4) {  // as w4a8_quant_act's choice of 1024 threads a row
        if (ch <= 1) INPUTS(1, M + shrink);
        else if (ch <= 2) INPUTS(2, M + shrink);
        else INPUTS(4, M + shrink);
        return hipGetLastError();
    }
    hipError_t e = launch_act_int8(X, IN, M, K, Xq, sx, st);
    if (e != hipSuccess || shrink == 0) return e;
    INPUTS(0, shrink);
#undef INPUTS
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_inputs(const void* X, int in_type, const void* A, const int* adapter,
                              const float* scale, int n_adapters, int M, int K, int R,
                              int8_t* Xq, float* sx, float* V, hipStream_t st) {
    if (in_type == 1)
        return inputs_run<1>(X, A, adapter, scale, n_adapters, M, K, R, Xq, sx, V, st);
    return inputs_run<2>(X, A, adapter, scale, n_adapters, M, K, R, Xq, sx, V, st);
}

hipError_t launch_lora_join(const int* acc, int splits, const float* sx, const float* sw,
                            int in_type, const LoraArgs& lora, int M, int N, void* Y,
                            hipStream_t st) {
    const long long units = (long long)((M + 15) / 16) * (N / 64);
    const dim3 grid((unsigned)((units + 3) / 4));
    unsigned short* y = reinterpret_cast<unsigned short*>(Y);
    if (in_type == 1)
        hipLaunchKernelGGL(lora_join_kernel<1>, grid, dim3(256), 0, st, acc, splits, sx, sw, lora,
                           M, N, y);
    else
        hipLaunchKernelGGL(lora_join_kernel<2>, grid, dim3(256), 0, st, acc, splits, sx, sw, lora,
                           M, N, y);
    return hipGetLastError();
}

}  // namespace w4a8
