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
            quant_row_regs<IN, 0, CH, 1024, true>(reinterpret_cast<const uint8_t*>(X) + (size_t)b * K * 2,
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

// INT8 of one row by one wave, the row in registers (K <= 512 CH): no barrier.
template <int IN, int CH>
__device__ __forceinline__ void quant_row_wave(const void* row, int K, uint8_t* xq, float* sx) {
    const int lane = threadIdx.x & 63, n8 = K / 8;
    Raw8<IN> c[CH];
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int i = lane + 64 * j;
        c[j] = i < n8 ? load_raw8<IN>(row, i) : Raw8<IN>{};
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const Row8<IN> v = widen8<IN>(c[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v.v[e]));
        // a new definition, or the widened elements stay alive for the codes
        asm volatile("" : "+v"(c[j].w[0]));
    }
    m = __builtin_bit_cast(float, wave_reduce(__builtin_bit_cast(unsigned, m), MaxU32{}));
    const float s = scale_of(m, 127.0f), inv = __fdiv_rn(1.0f, s);
    if (lane == 0) *sx = s;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int i = lane + 64 * j;
        if (i >= n8) continue;
        const Row8<IN> v = widen8<IN>(c[j]);
        reinterpret_cast<uint2*>(xq)[i] =
            uint2{quant4_fast(v.v[0], v.v[1], v.v[2], v.v[3], s, inv),
                  quant4_fast(v.v[4], v.v[5], v.v[6], v.v[7], s, inv)};
    }
}

// Large calls, workgroups of eight waves: the first ceil(M / 16) take the
// inner product of 16 rows, the others quantise a row per wave (CH > 0); the
// two read X within a few microseconds of each other, so once from HBM.
// Inner product: wave w takes the 128-wide K-tiles w, w + 8, ...  Matrix
// instructions 16 x 16 x 32 take A as the first and X as the
// second operand (lane (r, G): rank / row r, columns 8 G .. + 7 of a 32-wide
// step).  Rows of different adapters run one pass per adapter that occurs
// among them, each row keeping its own (a select).  RT blocks of 16 ranks
// share a pass.
template <int IN, int CH, int RT>
__global__ __launch_bounds__(512, 4) void lora_rows_kernel(
    const void* __restrict__ X, const void* __restrict__ A, const int* __restrict__ adapter,
    const float* __restrict__ scale, int n_adapters, int M, int K, int R,
    uint8_t* __restrict__ Xq, float* __restrict__ sx, float* __restrict__ V) {
    const int blocks = (M + 15) / 16;
    if constexpr (CH > 0) {
        if ((int)blockIdx.x >= blocks) {
            const size_t b = (size_t)(blockIdx.x - blocks) * 8 + (threadIdx.x >> 6);
            if (b < (size_t)M)
                quant_row_wave<IN, CH>(reinterpret_cast<const uint8_t*>(X) + b * K * 2, K,
                                       Xq + b * K, sx + b);
            return;
        }
    }
    __shared__ __attribute__((aligned(16))) float red[8 * RT * 256];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, G = lane >> 4, KT = K / 128;
    const int m = blockIdx.x * 16 + r;
    const bool live = m < M;
    const int id = live ? adapter[m] : -1;
    const uint8_t* x = reinterpret_cast<const uint8_t*>(X) + ((size_t)(live ? m : 0) * K + 8 * G) * 2;
    unsigned rest = (unsigned)__ballot(id >= 0 && id < n_adapters) & 0xFFFFu;
    struct Tile {
        v4i x[4], a[RT][4];
    };
    while (rest) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(rest));
        const unsigned mine = (unsigned)__ballot(id == a) & 0xFFFFu;
        rest &= ~mine;
        const float sc = scale[a];
        for (int r0 = 0; r0 < R; r0 += 16 * RT) {
            v4f acc[RT];
            const uint8_t* ap[RT];
            bool on[RT];
#pragma unroll
            for (int q = 0; q < RT; ++q) {
                acc[q] = v4f{0, 0, 0, 0};
                const int rr = r0 + 16 * q + r;
                on[q] = rr < R;
                ap[q] = reinterpret_cast<const uint8_t*>(A) +
                        (((size_t)a * R + (on[q] ? rr : 0)) * K + 8 * G) * 2;
            }
            auto load = [&](int kt, Tile& t) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const size_t o = ((size_t)kt * 128 + 32 * i) * 2;
                    t.x[i] = load16(x + o);  // a row past the end repeats row 0: not kept
#pragma unroll
                    for (int q = 0; q < RT; ++q) t.a[q][i] = load16(ap[q] + o);
                }
            };
            auto use = [&](const Tile& t) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int q = 0; q < RT; ++q) acc[q] = lora_mfma<IN>(t.a[q][i], t.x[i], acc[q]);
            };
            if constexpr (RT == 1) {  // two tiles in flight
                Tile t0, t1;
                int kt = wave;
                if (kt < KT) load(kt, t0);
                for (; kt + 8 < KT; kt += 16) {
                    load(kt + 8, t1);
                    use(t0);
                    if (kt + 16 < KT) load(kt + 16, t0);
                    use(t1);
                }
                if (kt < KT) use(t0);
            } else {  // (two would not fit 128 registers: four waves per SIMD hide the rest)
                for (int kt = wave; kt < KT; kt += 8) {
                    Tile t;
                    load(kt, t);
                    use(t);
                }
            }
            __syncthreads();  // the previous pass's sums have been read
#pragma unroll
            for (int q = 0; q < RT; ++q)
                *reinterpret_cast<v4f*>(&red[((wave * RT + q) * 64 + lane) * 4]) = acc[q];
            __syncthreads();
            // element e of a rank block: lane e / 4 (row lane % 16), rank 4 (lane / 16) + e % 4
            for (int e = tid; e < RT * 256; e += 512) {
                float s = 0.0f;
#pragma unroll
                for (int w = 0; w < 8; ++w) s += red[w * RT * 256 + e];
                const int l = (e & 255) >> 2, row = l & 15;
                const int rank = r0 + 16 * (e >> 8) + 4 * (l >> 4) + (e & 3);
                if (rank < R && ((mine >> row) & 1))
                    V[((size_t)blockIdx.x * 16 + row) * R + rank] = s * sc;
            }
        }
    }
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
    v4f y[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v) y[c][v] = ((float)sum[c][v] * s) * sw[n0 + 16 * c + 4 * G + v];
    lora_add<IN, false>(
        L, id, N, n0,
        [&](int p) {
            float v[8];
            lora_load_v(L, m, id >= 0, p, v);
            return lora_split<IN>(v);
        },
        y);
    if (!live) return;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        unsigned short h[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) h[v] = f32_to_f16_bits(y[c][v]);
        *reinterpret_cast<uint2*>(Y + (size_t)m * N + n0 + 16 * c + 4 * G) =
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
    if (M >= 512) {
        // without adapters only the rows are quantised
        const int blocks = (M + 15) / 16;
        if (K > 8192 || n_adapters == 0) {
            hipError_t e = launch_act_int8(X, IN, M, K, Xq, sx, st);
            if (e != hipSuccess || n_adapters == 0) return e;
        }
#define ROWS(CH, RT)                                                                         \
    hipLaunchKernelGGL((lora_rows_kernel<IN, CH, RT>), dim3(blocks + (CH > 0 ? (M + 7) / 8 : 0)), dim3(512), \
                       0, st, X, A, adapter, scale, n_adapters, M, K, R, q, sx, V)
#define ROWS_RT(CH)                \
    do {                           \
        if (R <= 16) ROWS(CH, 1);  \
        else ROWS(CH, 2);          \
    } while (0)
        if (K <= 4096) ROWS_RT(8);
        else if (K <= 8192) ROWS_RT(16);
        else ROWS_RT(0);
#undef ROWS_RT
#undef ROWS
        return hipGetLastError();
    }
    if (M < 512 && ch <= 4) {
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
