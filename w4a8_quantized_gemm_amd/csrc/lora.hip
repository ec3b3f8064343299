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
// X in the same launch (except for rows longer than its kernels hold in
// registers: K above 32768, 16384 from 512 rows on), and the epilogue of
// projections whose int32 sums (one or several K parts) lie in memory.
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

// INT8 of the rows of one workgroup of 16 waves: WPR waves a row, its elements
// in registers (K <= 512 CH WPR), maxima joined through LDS.
template <int IN, int WPR, int CH>
__device__ __forceinline__ void quant_rows16(const void* X, long long row0, int M, int K,
                                             uint8_t* Xq, float* sx) {
    __shared__ float part[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long m = row0 + wave / WPR;
    const int first = (wave % WPR) * 64 * CH + lane, n8 = K / 8;
    const uint8_t* row = reinterpret_cast<const uint8_t*>(X) + m * K * 2;
    Raw8<IN> c[CH];
    float mx = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int i = first + 64 * j;
        c[j] = m < M && i < n8 ? load_raw8<IN>(row, i) : Raw8<IN>{};
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const Row8<IN> v = widen8<IN>(c[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v.v[e]));
        // a new definition, or the widened elements stay alive for the codes
        asm volatile("" : "+v"(c[j].w[0]));
    }
    mx = __builtin_bit_cast(float, wave_reduce(__builtin_bit_cast(unsigned, mx), MaxU32{}));
    if constexpr (WPR > 1) {
        if (lane == 0) part[wave] = mx;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WPR; ++w) mx = fmaxf(mx, part[wave / WPR * WPR + w]);
    }
    if (m >= M) return;
    const float s = scale_of(mx, 127.0f), inv = __fdiv_rn(1.0f, s);
    if (first == 0) sx[m] = s;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int i = first + 64 * j;
        if (i >= n8) continue;
        const Row8<IN> v = widen8<IN>(c[j]);
        reinterpret_cast<uint2*>(Xq + m * K)[i] =
            uint2{quant4_fast(v.v[0], v.v[1], v.v[2], v.v[3], s, inv),
                  quant4_fast(v.v[4], v.v[5], v.v[6], v.v[7], s, inv)};
    }
}

// Large calls, workgroups of 16 waves: the first ceil(M / 16) take the inner
// product of 16 rows, the others quantise 16 / WPR rows each (WPR > 0); the
// two read X within a few microseconds of each other, so once from HBM.
// Inner product: wave w takes the 64-wide K-tiles w, w + 16, ...  Matrix
// instructions 16 x 16 x 32 take A as the first and X as the second operand
// (lane (r, G): rank / row r, columns 8 G .. + 7 of a 32-wide step).  Loads
// have four neighbouring lanes on one row (64 bytes) and a lane permutation
// through the LDS network brings them to that layout: loaded in it, every
// lane was a cache access of its own and the cache the bound (2048 x 4096,
// rank 32, two adapters in every block: 27 us; 18 now; 12 without adapters
// or with one, whose pass hides behind the quantisation).  The work of a
// block of rows is a list of jobs, one per adapter that occurs among the rows
// and 16 of its ranks; a pass over K takes two jobs, and every row keeps its
// own adapter's (a select).
template <int IN, int WPR, int CH>
__global__ __launch_bounds__(1024, 8) void lora_rows_kernel(
    const void* __restrict__ X, const void* __restrict__ A, const int* __restrict__ adapter,
    const float* __restrict__ scale, int n_adapters, int M, int K, int R,
    uint8_t* __restrict__ Xq, float* __restrict__ sx, float* __restrict__ V) {
    const int blocks = (M + 15) / 16;
    if constexpr (WPR > 0) {
        if ((int)blockIdx.x >= blocks) {
            quant_rows16<IN, WPR, CH>(X, (long long)(blockIdx.x - blocks) * (16 / WPR), M, K, Xq, sx);
            return;
        }
    }
    __shared__ __attribute__((aligned(16))) float red[16 * 2 * 256];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, G = lane >> 4, KT = K / 64;
    const int m = blockIdx.x * 16 + r;
    const bool live = m < M;
    const int id = live ? adapter[m] : -1;
    const int lr = lane >> 2, lc = 8 * (lane & 3);  // row and column this lane loads
    const int from = 4 * (4 * r + G);               // and the lane whose load it uses
    auto arrange = [&](v4i v) {
        v4i o;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = __builtin_amdgcn_ds_bpermute(from, v[q]);
        return o;
    };
    // (a row past the end repeats the first: not kept)
    const int mx = (int)blockIdx.x * 16 + lr < M ? (int)blockIdx.x * 16 + lr : 0;
    const uint8_t* x = reinterpret_cast<const uint8_t*>(X) + ((size_t)mx * K + lc) * 2;
    unsigned rest = (unsigned)__ballot(id >= 0 && id < n_adapters) & 0xFFFFu;
    struct Job {
        int a, r0;
        unsigned rows;  // 0: no job
    };
    Job at{-1, R, 0};
    auto next = [&]() {
        at.r0 += 16;
        if (at.r0 >= R) {
            at.rows = 0;
            if (rest) {
                at.a = __builtin_amdgcn_readlane(id, __builtin_ctz(rest));
                at.rows = (unsigned)__ballot(id == at.a) & 0xFFFFu;
                at.r0 = 0;
                rest &= ~at.rows;
            }
        }
        return at;
    };
    for (;;) {
        Job job[2];
        job[0] = next();
        if (job[0].rows == 0) return;
        job[1] = next();
        const bool both = job[1].rows != 0;
        v4f acc[2] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
        const uint8_t* ap[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // ranks past R repeat the last: not kept
            const int rr = min(job[q].r0 + lr, R - 1);
            ap[q] = reinterpret_cast<const uint8_t*>(A) +
                    (((size_t)job[both ? q : 0].a * R + (both || q == 0 ? rr : 0)) * K + lc) * 2;
        }
        for (int kt = wave; kt < KT; kt += 16) {
            v4i xv[2], av[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const size_t o = ((size_t)kt * 64 + 32 * i) * 2;
                xv[i] = load16(x + o);
                av[0][i] = load16(ap[0] + o);
                if (both) av[1][i] = load16(ap[1] + o);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const v4i xo = arrange(xv[i]);
                acc[0] = lora_mfma<IN>(arrange(av[0][i]), xo, acc[0]);
                if (both) acc[1] = lora_mfma<IN>(arrange(av[1][i]), xo, acc[1]);
            }
        }
        __syncthreads();  // the previous pass's sums have been read
#pragma unroll
        for (int q = 0; q < 2; ++q)
            *reinterpret_cast<v4f*>(&red[((wave * 2 + q) * 64 + lane) * 4]) = acc[q];
        __syncthreads();
        // element e of a job: lane e / 4 (row lane % 16), rank 4 (lane / 16) + e % 4
        if (tid < 512) {
            const Job j = tid < 256 ? job[0] : job[1];
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < 16; ++w) s += red[w * 512 + tid];
            const int l = (tid & 255) >> 2, row = l & 15;
            const int rank = j.r0 + 4 * (l >> 4) + (tid & 3);
            if (((j.rows >> row) & 1) && rank < R)
                V[((size_t)blockIdx.x * 16 + row) * R + rank] = s * scale[j.a];
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
    auto scaled = [&](int c) {
        v4f o;
#pragma unroll
        for (int v = 0; v < 4; ++v) o[v] = ((float)sum[c][v] * s) * sw[n0 + 16 * c + 4 * G + v];
        return o;
    };
    v4f y[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = scaled(c);
    lora_add<IN, false>(
        L, id, N, n0,
        [&](int p) {
            float v[8];
            lora_load_v(L, m, id >= 0, p, v);
            return lora_split<IN>(v);
        },
        y);
    lora_redo<IN>(L, id, m, N, n0, scaled, y);
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
        if (K > 16384 || n_adapters == 0) {
            hipError_t e = launch_act_int8(X, IN, M, K, Xq, sx, st);
            if (e != hipSuccess || n_adapters == 0) return e;
        }
        // waves per row: more for long rows, and until the rows fill 256 workgroups
        int wpr = 1, ch = 2;
        while (wpr < 4 && ((long long)M * wpr < 4096 || K > 4096 * wpr)) wpr *= 2;
        while (512 * ch * wpr < K) ch *= 2;
#define ROWS(WPR, CH)                                                                            \
    hipLaunchKernelGGL((lora_rows_kernel<IN, WPR, CH>),                                          \
                       dim3(blocks + (WPR ? (M * (long long)WPR + 15) / 16 : 0)), dim3(1024), 0, st, \
                       X, A, adapter, scale, n_adapters, M, K, R, q, sx, V)
#define ROWS_CH(WPR)               \
    do {                           \
        if (ch == 2) ROWS(WPR, 2); \
        else if (ch == 4) ROWS(WPR, 4); \
        else ROWS(WPR, 8);         \
    } while (0)
        if (K > 16384) ROWS(0, 2);
        else if (wpr == 1) ROWS_CH(1);
        else if (wpr == 2) ROWS_CH(2);
        else ROWS_CH(4);
#undef ROWS_CH
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
