// What lies between two projections of a layer, in one pass over a row:
//
//   b  = Y[m]; post norm, gate; x' = x_scale X[m] + y_scale b   (residual sum)
//   n  = pre norm of x'                                         (float32)
//   out = n in a floating type, or its INT8 / e4m3 codes and the row's scale
//
// norm(v) = (v r) w + bias with r = 1 / sqrt(mean(v^2) + eps) (RMS), or of
// d = v - mean(v) (layer norm).  Every float32 operation is rounded by itself
// (no fused multiply-add), and the sums behind mean() are taken in float64 of
// exact float32 terms, in an order that K alone fixes (launch_norm_types): a row's
// codes are a function of its own inputs, whatever the batch.  Another order
// would show where a signed sum cancels, and once in some 2^29 sums of squares,
// which lie 29 bits below the float32 they are rounded to.  A float64 addition
// costs this chip what a float32 one does.
//
// One workgroup per row, the row in registers between the reductions: X, Y
// and the gate are read once and each output is written once.  Many rows are
// bound by memory (8192 x 8192, 16-bit X and Y to INT8: 470 MB in 84-88 us, 5.3
// to 5.6 TB/s; float32 X and Y: 872 MB in 156 us; the float64 sums cost nothing
// measurable there: 88 us with float32 ones against 89).  A layer norm's second
// reduction makes that 100 us, e4m3's rounded quotients 94.  Fewer rows than a few
// per CU are bound by one chain of loads, two or three reductions and stores (2048
// x 4096 gated: 75 MB in 21 us; 16 x 8192: 5 us).
#include "act_common.h"
#include "launch.h"
#include "wave_common.h"

#pragma clang fp contract(off)

namespace w4a8 {

namespace {

// pairs, for the conversions that round two floats at once (nearest even)
typedef float v2f __attribute__((ext_vector_type(2)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

template <int CTRL>
__device__ __forceinline__ double dpp_step(double v) {
    const uint2 u = __builtin_bit_cast(uint2, v);
    const uint2 o{(unsigned)__builtin_amdgcn_mov_dpp((int)u.x, CTRL, 0xF, 0xF, true),
                  (unsigned)__builtin_amdgcn_mov_dpp((int)u.y, CTRL, 0xF, 0xF, true)};
    return v + __builtin_bit_cast(double, o);
}
__device__ __forceinline__ double lane64(double v, int l) {
    const uint2 u = __builtin_bit_cast(uint2, v);
    return __builtin_bit_cast(double, uint2{(unsigned)__builtin_amdgcn_readlane((int)u.x, l),
                                            (unsigned)__builtin_amdgcn_readlane((int)u.y, l)});
}
// Sum over a wave (the steps of row16_reduce, then the four rows).
__device__ __forceinline__ double wave_sum64(double v) {
    v = dpp_step<0xB1>(v);
    v = dpp_step<0x4E>(v);
    v = dpp_step<0x141>(v);
    v = dpp_step<0x140>(v);
    return (lane64(v, 0) + lane64(v, 16)) + (lane64(v, 32) + lane64(v, 48));
}
// Sum over a workgroup, the same bits in every thread.  `part` holds a value
// per wave; no barrier stands behind the reads, so two reductions in a row
// take two arrays.
template <int TPB>
__device__ __forceinline__ double block_sum64(double v, double* part) {
    v = wave_sum64(v);
    if constexpr (TPB == 64) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < TPB / 64; ++w) v += part[w];
    return v;
}
template <int TPB>
__device__ __forceinline__ unsigned block_max_u32(unsigned v, unsigned* part) {
    v = wave_reduce(v, MaxU32{});
    if constexpr (TPB == 64) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < TPB / 64; ++w) v = MaxU32{}(v, part[w]);
    return v;
}

struct F8v {
    float v[8];
};
__device__ __forceinline__ F8v load_f8(const float* p, int i) {  // (4-byte aligned only)
    F8v r;
#pragma unroll
    for (int j = 0; j < 8; ++j) r.v[j] = p[8 * i + j];
    return r;
}

template <int IN>
__device__ __forceinline__ const void* row_at(const void* X, size_t m, int K) {
    return reinterpret_cast<const uint8_t*>(X) + m * K * (IN == 0 ? 4 : 2);
}

// Eight consecutive elements of a row as type T (W4A8_IN_*), rounded once.
__device__ __forceinline__ void store_row8(void* X, int type, size_t m, int K, int i,
                                           const float (&v)[8]) {
    if (type == 0) {
        v4f* p = reinterpret_cast<v4f*>(reinterpret_cast<float*>(X) + m * K) + 2 * i;
        p[0] = v4f{v[0], v[1], v[2], v[3]};
        p[1] = v4f{v[4], v[5], v[6], v[7]};
        return;
    }
    v4i w;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a = v[2 * j], b = v[2 * j + 1];
        asm("" : "+v"(a), "+v"(b));  // rounded to float32 before they are converted
        if (type == 1)
            w[j] = __builtin_bit_cast(int, __builtin_convertvector((v2f{a, b}), v2h));
        else
            w[j] = __builtin_bit_cast(int, __builtin_convertvector((v2f{a, b}), v2b));
    }
    reinterpret_cast<v4i*>(reinterpret_cast<unsigned short*>(X) + m * K)[i] = w;
}

// Gate row of row m: its own, the batch's, or the one it names (-1: none).
__device__ __forceinline__ int gate_row(const NormArgs& a, int m) {
    if (!a.gate) return -1;
    if (a.gate_ids) {
        const int g = a.gate_ids[m];
        return g >= 0 && g < a.gate_rows ? g : -1;
    }
    return a.gate_rows == 1 ? 0 : m;
}

// sum / K, correctly rounded: inv_k is the rounded 1 / K, the product's remainder is
// exact in a fused operation, and the corrected quotient rounds as the true one.
__device__ __forceinline__ double over_k(double sum, const NormArgs& a) {
    const double q = sum * a.inv_k;
    return __builtin_fma(__builtin_fma(-q, (double)a.K, sum), a.inv_k, q);
}

// float32(1 / sqrt(sum / K + eps)).  The hardware's estimate and two Newton steps
// leave about 2^-51; where a middle between two float32 numbers lies within 2^-47 (one
// row in 2^21), or the result is subnormal, the rounded square root and its rounded
// reciprocal decide.  (Taken for every row they made 8192 x 8192 84.9 -> 86.5 us.)  A
// row whose squares add up to infinity gets 0.
__device__ __forceinline__ float inverse_rms(double sum, const NormArgs& a) {
    const double v = over_k(sum, a) + (double)a.eps;
    double y = __builtin_amdgcn_rsq(v);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const double e = __builtin_fma(-v * y, y, 1.0);
        y = __builtin_fma(0.5 * y, e, y);
    }
    const unsigned low = (unsigned)__builtin_bit_cast(uint64_t, y) & 0x1FFFFFFFu;
    if (low - (0x10000000u - 64u) <= 128u || y < 0x1p-126) {
        // the first step leaves one unit at most, the second an exact remainder: the
        // rounded quotient (fewer registers than a general division)
        const double s = sqrt(v);
        y = __builtin_fma(y, __builtin_fma(-s, y, 1.0), y);
        y = __builtin_fma(y, __builtin_fma(-s, y, 1.0), y);
    }
    return sum == __builtin_inf() ? 0.0f : (float)y;
}

// Codes of eight elements (finite) with scale s.
__device__ __forceinline__ uint2 int8_codes(const float (&n)[8], float s, float inv) {
    return uint2{quant4_fast(n[0], n[1], n[2], n[3], s, inv),
                 quant4_fast(n[4], n[5], n[6], n[7], s, inv)};
}
__device__ __forceinline__ uint2 e4m3_codes(const float (&n)[8], float s) {
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = __fdiv_rn(n[j], s);
    return e4m3_codes8(t);
}

}  // namespace

// XT, YT: element types of the residual stream and of the block's output
// (YT = -1: no block).  A row of at most 8 TPB CH elements by TPB threads; rows
// of one wave (TPB = 64) lie four to a workgroup and meet no barrier.
template <int XT, int YT, int CH, int TPB>
__global__ __launch_bounds__(TPB == 64 ? 256 : TPB) void norm_kernel(NormArgs a) {
    constexpr bool HASY = YT >= 0;
    constexpr int YL = HASY ? YT : 0;
    constexpr int W = TPB / 64;
    __shared__ double sums[4][W];
    __shared__ unsigned maxs[W];
    const int K = a.K, n8 = K / 8;
    const size_t m = TPB == 64 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    const int tid = TPB == 64 ? threadIdx.x & 63 : threadIdx.x;
    if (TPB == 64 && (int)m >= a.M) return;

    // The gate is requested with the other rows, except where x, y and gate of
    // float32 would take 96 of the 128 registers that 1024 threads have each (nine
    // more went to scratch): there behind the norm of y (257 x 32768, layer norms:
    // 71 -> 62 us).
    constexpr bool kLateGate = XT == 0 && YT == 0 && CH * TPB == 4096;
    Raw8<XT> xr[CH];
    Raw8<YL> yr[HASY ? CH : 1], gr[HASY ? CH : 1];
    const void* xrow = row_at<XT>(a.x, m, K);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int i = tid + TPB * j;
        xr[j] = i < n8 ? load_raw8<XT>(xrow, i) : Raw8<XT>{};
    }
    int g = -1;
    if constexpr (HASY) {
        const void* yrow = row_at<YL>(a.y, m, K);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int i = tid + TPB * j;
            yr[j] = i < n8 ? load_raw8<YL>(yrow, i) : Raw8<YL>{};
        }
        g = gate_row(a, (int)m);
    }
    auto load_gate = [&] {
        const void* grow = row_at<YL>(a.gate, (size_t)g, K);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int i = tid + TPB * j;
            gr[j] = i < n8 ? load_raw8<YL>(grow, i) : Raw8<YL>{};
        }
    };
    if constexpr (HASY && !kLateGate)
        if (g >= 0) load_gate();

    // v = norm(v); elements past the row end stay zero
    auto normed = [&](float (&v)[CH][8], const float* w, const float* bias, int at) {
        double s = 0.0;
        if (a.layer) {
#pragma unroll
            for (int j = 0; j < CH; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) s += (double)v[j][e];
            const float mean = (float)over_k(block_sum64<TPB>(s, sums[at]), a);
            s = 0.0;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                if (tid + TPB * j >= n8) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] - mean;
            }
        }
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double d = (double)v[j][e];
                s = __builtin_fma(d, d, s);
            }
        const float r = inverse_rms(block_sum64<TPB>(s, sums[at + 1]), a);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int i = tid + TPB * j;
            if (i >= n8) continue;
            const F8v wv = load_f8(w, i);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = (v[j][e] * r) * wv.v[e];
            if (bias) {
                const F8v bv = load_f8(bias, i);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] + bv.v[e];
            }
        }
    };
    const bool scaled = a.x_scale != 1.0f || a.y_scale != 1.0f;

    float v[CH][8];
    if constexpr (HASY) {
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const Row8<YL> y = widen8<YL>(yr[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = y.v[e];
        }
        if (a.y_weight) normed(v, a.y_weight, a.y_bias, 0);
        if (g >= 0) {
            if constexpr (kLateGate) load_gate();
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const Row8<YL> gv = widen8<YL>(gr[j]);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] * gv.v[e];
            }
        }
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int i = tid + TPB * j;
            const Row8<XT> x = widen8<XT>(xr[j]);
            if (scaled) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] = x.v[e] * a.x_scale + v[j][e] * a.y_scale;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] = x.v[e] + v[j][e];
            }
            if (i < n8) store_row8(a.xout, XT, m, K, i, v[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const Row8<XT> x = widen8<XT>(xr[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = x.v[e] * a.x_scale;
        }
    }
    if (a.weight) normed(v, a.weight, a.bias, 2);

    if (a.out_type < 3) {
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int i = tid + TPB * j;
            if (i < n8) store_row8(a.out, a.out_type, m, K, i, v[j]);
        }
        return;
    }
    unsigned top = 0;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = MaxU32{}(top, abs_bits(v[j][e]));
    top = block_max_u32<TPB>(top, maxs);
    const float s = row_scale_bits(top, a.out_type == 3 ? 127.0f : 448.0f);
    const float inv = __fdiv_rn(1.0f, s);
    if (tid == 0) a.sx[m] = s;
    uint2* q = reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(a.out) + m * K);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int i = tid + TPB * j;
        if (i >= n8) continue;
        q[i] = s != s ? uint2{0, 0}
               : a.out_type == 3 ? int8_codes(v[j], s, inv)
                                 : e4m3_codes(v[j], s);
    }
}

// Rows too long for the registers: the same values, formed again from memory
// in every pass.
template <int XT, int YT>
__global__ __launch_bounds__(1024) void norm_long_kernel(NormArgs a) {
    constexpr bool HASY = YT >= 0;
    constexpr int YL = HASY ? YT : 0;
    constexpr int TPB = 1024;
    __shared__ double sums[4][TPB / 64];
    __shared__ unsigned maxs[TPB / 64];
    const int K = a.K, n8 = K / 8, tid = threadIdx.x;
    const size_t m = blockIdx.x;
    const void* xrow = row_at<XT>(a.x, m, K);
    const void* yrow = HASY ? row_at<YL>(a.y, m, K) : nullptr;
    const int g = HASY ? gate_row(a, (int)m) : -1;
    const void* grow = g >= 0 ? row_at<YL>(a.gate, (size_t)g, K) : nullptr;

    float y_mean = 0.0f, y_r = 1.0f, mean = 0.0f, r = 1.0f;
    auto norm8 = [&](float (&v)[8], int i, float mu, float inv, const float* w, const float* b) {
        const F8v wv = load_f8(w, i);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = ((v[e] - mu) * inv) * wv.v[e];
        if (b) {
            const F8v bv = load_f8(b, i);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] + bv.v[e];
        }
    };
    auto block_out = [&](int i, float (&v)[8]) {  // elements of Y
        const Row8<YL> y = load_row8<YL>(yrow, i);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = y.v[e];
    };
    auto stream = [&](int i, float (&v)[8]) {  // elements of x'
        const Row8<XT> x = load_row8<XT>(xrow, i);
        if constexpr (HASY) {
            block_out(i, v);
            if (a.y_weight) norm8(v, i, y_mean, y_r, a.y_weight, a.y_bias);
            if (grow) {
                const Row8<YL> gv = load_row8<YL>(grow, i);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = v[e] * gv.v[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = x.v[e] * a.x_scale + v[e] * a.y_scale;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = x.v[e] * a.x_scale;
        }
    };
    auto statistics = [&](auto get, float& mu, float& inv, int at) {
        if (a.layer) {
            double s = 0.0;
            for (int i = tid; i < n8; i += TPB) {
                float v[8];
                get(i, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) s += (double)v[e];
            }
            mu = (float)over_k(block_sum64<TPB>(s, sums[at]), a);
        }
        double s = 0.0;
        for (int i = tid; i < n8; i += TPB) {
            float v[8];
            get(i, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double d = (double)(v[e] - mu);
                s = __builtin_fma(d, d, s);
            }
        }
        inv = inverse_rms(block_sum64<TPB>(s, sums[at + 1]), a);
    };
    if constexpr (HASY)
        if (a.y_weight) statistics(block_out, y_mean, y_r, 0);
    if (a.weight) statistics(stream, mean, r, 2);
    const bool quantised = a.out_type >= 3;
    float s = 1.0f, inv = 1.0f;
    if (quantised) {
        unsigned top = 0;
        for (int i = tid; i < n8; i += TPB) {
            float v[8];
            stream(i, v);
            if (a.weight) norm8(v, i, mean, r, a.weight, a.bias);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = MaxU32{}(top, abs_bits(v[e]));
        }
        s = row_scale_bits(block_max_u32<TPB>(top, maxs), a.out_type == 3 ? 127.0f : 448.0f);
        inv = __fdiv_rn(1.0f, s);
        if (tid == 0) a.sx[m] = s;
    }
    uint2* q = reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(a.out) + m * K);
    for (int i = tid; i < n8; i += TPB) {
        float v[8];
        stream(i, v);
        // Xout may be X: a thread writes what it alone reads, after reading it
        if constexpr (HASY) store_row8(a.xout, XT, m, K, i, v);
        if (a.weight) norm8(v, i, mean, r, a.weight, a.bias);
        if (!quantised)
            store_row8(a.out, a.out_type, m, K, i, v);
        else
            q[i] = s != s ? uint2{0, 0}
                   : a.out_type == 3 ? int8_codes(v, s, inv)
                                     : e4m3_codes(v, s);
    }
}

namespace {

// Threads and chunks of eight elements a thread for a row, by its width alone: they
// fix the order of the float64 sums, so a row gets the same bits in every batch.
// Two chunks a thread where that is possible.  us, threads x chunks (16-bit x and y
// to INT8, residual sum and norm):
//   8192 x 8192: 512 x 2 84, 256 x 4 89, 1024 x 1 112     16 x 8192: 512 x 2 4.4,
//   8192 x 4096: 256 x 2 44.4, 512 x 1 50.4                 1024 x 1 5.5, 256 x 4 5.4
//   2048 x 16384: 512 x 4 51.1, 1024 x 2 54.5             1 x 4096: 256 x 2 3.1,
//   8192 x 2048: 128 x 2 25.5, 256 x 1 28.0, 64 x 4 28.2    1024 x 1 3.3, 64 x 8 6.4
//   8192 x 1024: 64 x 2 15.6, 256 x 1 20.1
// Few rows alone would take more threads there (16 x 2048: 256 x 2 3.6, 128 x 2 4.1;
// 256 x 1024: 3.9 against 4.2), and 256 x 3 saves many rows of 4112 .. 6144 little
// (1000 x 5120, two norms: 14.1 against 14.5) but costs few a lot (16 x 5120: 4.8
// against 4.1).
template <int XT, int YT>
void launch_norm_types(const NormArgs& a, hipStream_t st) {
    const int n8 = a.K / 8;
#define NORM(CH, TPB)                                                                    \
    if (n8 <= TPB * CH) {                                                                \
        const int rows = TPB == 64 ? 4 : 1;                                              \
        hipLaunchKernelGGL((norm_kernel<XT, YT, CH, TPB>), dim3((a.M + rows - 1) / rows), \
                           dim3(rows * TPB), 0, st, a);                                  \
        return;                                                                          \
    }
    NORM(2, 64)
    NORM(2, 128)
    NORM(2, 256)
    NORM(2, 512)
    NORM(3, 512)
    NORM(4, 512)
    NORM(4, 1024)
#undef NORM
    hipLaunchKernelGGL((norm_long_kernel<XT, YT>), dim3(a.M), dim3(1024), 0, st, a);
}

template <int XT>
void launch_norm_x(const NormArgs& a, int y_type, hipStream_t st) {
    if (!a.y) launch_norm_types<XT, -1>(a, st);
    else if (y_type == 1) launch_norm_types<XT, 1>(a, st);
    else if (y_type == 2) launch_norm_types<XT, 2>(a, st);
    else launch_norm_types<XT, 0>(a, st);
}

}  // namespace

hipError_t launch_norm_quant(const NormArgs& a, int x_type, int y_type, hipStream_t st) {
    if (x_type == 1) launch_norm_x<1>(a, y_type, st);
    else if (x_type == 2) launch_norm_x<2>(a, y_type, st);
    else launch_norm_x<0>(a, y_type, st);
    return hipGetLastError();
}

}  // namespace w4a8
