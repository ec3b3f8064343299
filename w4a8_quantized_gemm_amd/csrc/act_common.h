// Device helpers of the kernels that quantise rows: symmetric scales and
// codes, loads of float32 / fp16 / bf16 elements widened to float32, and the
// largest value of a workgroup.
#pragma once
#include "device_common.h"
#include "wave_common.h"

namespace w4a8 {

__device__ __forceinline__ float scale_of(float amax, float qmax) {
    float s = __fdiv_rn(amax, qmax);
    return (s > 0.0f) ? s : 1.0f;
}

__device__ __forceinline__ int quant_sym(float x, float s, float qmax) {
    float v = __builtin_rintf(__fdiv_rn(x, s));
    v = fminf(fmaxf(v, -qmax), qmax);
    return (int)v;
}

// Absolute maximum as the bits of a non-negative float: an integer maximum,
// so a NaN (whose bits lie above infinity's) is not lost.
__device__ __forceinline__ unsigned abs_bits(float v) {
    return __builtin_bit_cast(unsigned, v) & 0x7FFFFFFFu;
}
__device__ __forceinline__ unsigned block_max_bits(unsigned m) {
    __shared__ unsigned part[16];
    m = wave_reduce(m, MaxU32{});
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) m = MaxU32{}(m, part[w]);
    __syncthreads();
    return m;
}
// Scale of a row: max / qmax, 1 for an all-zero row, and NaN for a row with
// an element that is not finite (all of the row's results are NaN then).
__device__ __forceinline__ float row_scale_bits(unsigned m, float qmax = 127.0f) {
    if (m >= 0x7F800000u) return __builtin_nanf("");
    return scale_of(__builtin_bit_cast(float, m), qmax);
}

// Four quant_sym(v, s, 127) codes as the bytes of a dword, in fewer
// instructions: inv = 1 / s; v inv is within two units in the last place of
// the correctly rounded quotient, so both round to the same integer unless
// the product lies next to a half (or is not finite), where the quotient
// decides.  The integer comes out of an addition of 1.5 2^23, which rounds
// to nearest even at its unit digit and leaves the code in the low byte
// (|v| <= 127 s (1 + 2^-23), so |v inv| rounds to at most 127).
__device__ __forceinline__ unsigned quant4_fast(float a, float b, float c, float d, float s,
                                                float inv) {
    constexpr float kMagic = 12582912.0f;
    const float v[4] = {a, b, c, d};
    float t[4];
    bool sure = true;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float q = v[j] * inv;
        t[j] = q + kMagic;
        sure = sure && fabsf(q - (t[j] - kMagic)) <= 0.49996f;
    }
    unsigned w = __builtin_amdgcn_perm(__builtin_bit_cast(unsigned, t[1]),
                                       __builtin_bit_cast(unsigned, t[0]), 0x0C0C0400u) |
                 __builtin_amdgcn_perm(__builtin_bit_cast(unsigned, t[3]),
                                       __builtin_bit_cast(unsigned, t[2]), 0x04000C0Cu);
    if (!sure) {
        w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) w |= (unsigned)(quant_sym(v[j], s, 127.0f) & 0xFF) << (8 * j);
    }
    return w;
}

// OCP e4m3 codes of eight quotients of a row's elements and its scale: nearest even,
// saturating at 448.  While the scale is a normal float32 they stay below
// 448 (1 + 2^-23); a subnormal one is a whole number of 2^-149, and a quotient may
// reach 671, of which the conversion alone makes the NaN code.
__device__ __forceinline__ uint2 e4m3_codes8(const float (&t)[8]) {
    float c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = __builtin_amdgcn_fmed3f(t[e], -448.0f, 448.0f);
    unsigned w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int l = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * h], c[4 * h + 1], 0, false);
        w[h] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * h + 2], c[4 * h + 3], l, true);
    }
    return uint2{w[0], w[1]};
}

// Elements of float32, fp16 or bf16 rows (IN = 0, 1, 2).
template <int IN>
struct Row8 {  // eight consecutive elements of a row, widened to float32
    float v[8];
};

template <int IN>
struct Raw8 {  // the same eight elements as stored (32 bytes float32, 16 otherwise)
    v4i w[IN == 0 ? 2 : 1];
};

template <int IN>
__device__ __forceinline__ Raw8<IN> load_raw8(const void* row, int i) {  // elements 8i..8i+7
    Raw8<IN> r;
    const v4i* p = reinterpret_cast<const v4i*>(row) + (IN == 0 ? 2 * i : i);
    r.w[0] = p[0];
    if constexpr (IN == 0) r.w[1] = p[1];
    return r;
}

template <int IN>
__device__ __forceinline__ Row8<IN> widen8(const Raw8<IN>& w) {
    Row8<IN> r;
    if constexpr (IN == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // through a scalar: a bit cast of the vector element itself
            // reads lane 0 of the vector with this compiler
            const int x = w.w[j >> 2][j & 3];
            r.v[j] = __builtin_bit_cast(float, x);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const unsigned h = ((unsigned)w.w[0][j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
            if constexpr (IN == 1)
                r.v[j] = (float)__builtin_bit_cast(_Float16, (unsigned short)h);
            else
                r.v[j] = __builtin_bit_cast(float, h << 16);
        }
    }
    return r;
}

template <int IN>
__device__ __forceinline__ Row8<IN> load_row8(const void* row, int i) {
    return widen8<IN>(load_raw8<IN>(row, i));
}

// Largest of the TPB threads' values.
template <int TPB = 256>
__device__ __forceinline__ float block_max(float m) {
    for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    __shared__ float part[TPB / 64];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    m = part[0];
#pragma unroll
    for (int w = 1; w < TPB / 64; ++w) m = fmaxf(m, part[w]);
    __syncthreads();
    return m;
}

// Per-token quantisation of one row by a workgroup of TPB threads, the row
// held in registers between the absolute maximum and the quantisation (rows
// of at most 8 TPB CH elements), so it is read from memory once.  Q: 0 =
// INT8 (qmax 127), 1 = e4m3.  FAST: the same INT8 codes by quant4_fast.
template <int IN, int Q, int CH, int TPB, bool FAST = false>
__device__ __forceinline__ void quant_row_regs(const void* row, int K, uint8_t* Xq_row,
                                               float* sx_row) {
    const int n8 = K / 8;
    Raw8<IN> c[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int i = threadIdx.x + TPB * j;
        c[j] = i < n8 ? load_raw8<IN>(row, i) : Raw8<IN>{};
    }
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const Row8<IN> r = widen8<IN>(c[j]);  // zeros past the row end
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(r.v[e]));
    }
    const float s = scale_of(block_max<TPB>(m), Q == 0 ? 127.0f : 448.0f);
    if (threadIdx.x == 0) *sx_row = s;
    [[maybe_unused]] const float inv = __fdiv_rn(1.0f, s);
    uint2* out = reinterpret_cast<uint2*>(Xq_row);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int i = threadIdx.x + TPB * j;
        if (i >= n8) continue;
        const Row8<IN> r = widen8<IN>(c[j]);
        if constexpr (Q == 0 && FAST) {
            out[i] = uint2{quant4_fast(r.v[0], r.v[1], r.v[2], r.v[3], s, inv),
                           quant4_fast(r.v[4], r.v[5], r.v[6], r.v[7], s, inv)};
        } else if constexpr (Q == 0) {
            unsigned b[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = (unsigned)(quant_sym(r.v[e], s, 127.0f) & 0xFF);
            out[i] = uint2{b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24),
                           b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24)};
        } else {
            // a NaN quotient (NaN input) gets 0x7F whatever its sign
            float t[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = __fdiv_rn(r.v[e], s);
            const uint2 codes = e4m3_codes8(t);
            unsigned w[2] = {codes.x, codes.y};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (t[e] != t[e])
                    w[e / 4] = (w[e / 4] & ~(0xFFu << (8 * (e % 4)))) | (0x7Fu << (8 * (e % 4)));
            out[i] = uint2{w[0], w[1]};
        }
    }
}

}  // namespace w4a8
