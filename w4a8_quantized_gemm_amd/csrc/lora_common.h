// The outer product of low-rank adapters, as the epilogues of the shared
// projection's kernels add it: delta[m][n] = sum_r V[m][r] B[a(m)][n][r].
//
// A 16 x 16 block (16 channels, 16 rows of X) takes one 16 x 16 x 32 matrix
// instruction per 32 ranks and operand part.  B is used as stored (fp16 or
// bfloat16, 16 bytes per lane straight from memory); V is float32 and is
// split into two operands of B's type, V = hi + lo, each rounded to nearest:
//   bfloat16: hi + lo keeps 16 significant bits of each element;
//   fp16: the 32 ranks of a row are first scaled by a power of two that
//     brings their largest to [2^14, 2^15) (its range would lose V
//     otherwise), hi + lo then keeps 21 bits, or 2^-38 of the largest for
//     elements far below it.
// Sums are float32.  Rows of a block may select different adapters: the
// block is multiplied by each adapter that occurs in it and every row keeps
// its own product (a select, so another row's infinities do not reach it).
#pragma once
#include "device_common.h"
#include "launch.h"

namespace w4a8 {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <int IN>
__device__ __forceinline__ v4f lora_mfma(v4i a, v4i b, v4f c) {
    if constexpr (IN == 1)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Operand parts of 8 ranks of one row, and the factor of their products.
struct LoraV {
    v4i hi, lo;
    float back;
};

// v: ranks 32 s + 8 G .. + 7 of row (lane % 16), G = lane / 16.
template <int IN>
__device__ __forceinline__ LoraV lora_split(const float (&v)[8]) {
    LoraV o;
    unsigned h[8], l[8];
    if constexpr (IN == 1) {
        unsigned m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const unsigned b = __builtin_bit_cast(unsigned, v[j]) & 0x7FFFFFFFu;
            m = b > m ? b : m;
        }
        const unsigned m1 = __shfl_xor(m, 16, 64);
        m = m1 > m ? m1 : m;
        const unsigned m2 = __shfl_xor(m, 32, 64);
        m = m2 > m ? m2 : m;
        // exponent field of the largest; far below float32's normal range
        // the elements may vanish (their products are below 2^-90)
        const unsigned e = m >> 23 > 20 ? m >> 23 : 20;
        const float to = __builtin_bit_cast(float, (e < 254 ? 268 - e : 14u) << 23);
        o.back = __builtin_bit_cast(float, (e < 254 ? e - 14 : 240u) << 23);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = v[j] * to;
            const _Float16 a = (_Float16)x;
            const float d = x - (float)a;
            const _Float16 b = (_Float16)(d == d ? d : 0.0f);
            h[j] = __builtin_bit_cast(unsigned short, a);
            l[j] = __builtin_bit_cast(unsigned short, b);
        }
    } else {
        o.back = 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            h[j] = f32_to_bf16_bits(v[j]);
            const float d = v[j] - __builtin_bit_cast(float, h[j] << 16);
            l[j] = f32_to_bf16_bits(d == d ? d : 0.0f);  // hi infinite: lo 0
        }
    }
    o.hi = v4i{(int)(h[0] | h[1] << 16), (int)(h[2] | h[3] << 16), (int)(h[4] | h[5] << 16),
               (int)(h[6] | h[7] << 16)};
    o.lo = v4i{(int)(l[0] | l[1] << 16), (int)(l[2] | l[3] << 16), (int)(l[4] | l[5] << 16),
               (int)(l[6] | l[7] << 16)};
    return o;
}

// Ranks 32 s + 8 G .. + 7 of row m of V (zeros past R and for rows that have
// no adapter, whose V is never written).
__device__ __forceinline__ void lora_load_v(const LoraArgs& L, int m, bool live, int s,
                                            float (&v)[8]) {
    const int k0 = 32 * s + 8 * ((threadIdx.x & 63) >> 4);
    v4f a = v4f{0, 0, 0, 0}, b = a;
    if (live && k0 < L.R) {
        const v4f* p = reinterpret_cast<const v4f*>(L.V + (size_t)m * L.R + k0);
        a = p[0];
        b = p[1];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = a[j];
        v[4 + j] = b[j];
    }
}

// B operand of adapter a, ranks 32 s .. + 31, channels n0 .. n0 + 15.
__device__ __forceinline__ v4i lora_load_b(const LoraArgs& L, int a, int N, int n0, int s) {
    const int lane = threadIdx.x & 63, k0 = 32 * s + 8 * (lane >> 4);
    if (k0 >= L.R) return v4i{0, 0, 0, 0};
    const size_t row = (size_t)a * N + n0 + (lane & 15);
    return load16(reinterpret_cast<const uint8_t*>(L.B) + (row * L.R + k0) * 2);
}

// The adapter of row m (or -1).
__device__ __forceinline__ int lora_id(const LoraArgs& L, int m, bool live) {
    const int a = live ? L.adapter[m] : -1;
    return a >= 0 && a < L.n_adapters ? a : -1;
}

// delta[c][v] for row (lane % 16), channel n0 + 16 c + 4 (lane / 16) + v, of
// the 16 rows whose adapters are `id` (equal for the four lanes of a row).
// Adapters are taken four at a time, so their operands are in flight
// together; every 32 ranks are one pass.
template <int IN, int NC>
__device__ __forceinline__ void lora_block(const LoraArgs& L, int m, int id, int N, int n0,
                                           v4f (&delta)[NC]) {
    constexpr int BATCH = NC == 1 ? 4 : 1;
#pragma unroll
    for (int c = 0; c < NC; ++c) delta[c] = v4f{0, 0, 0, 0};
    const unsigned any = (unsigned)__ballot(id >= 0) & 0xFFFFu;
    if (any == 0) return;
    for (int s = 0; 32 * s < L.R; ++s) {
        float v[8];
        lora_load_v(L, m, id >= 0, s, v);
        LoraV V;
        bool split = false;
        unsigned rest = any;
        while (rest) {
            int a[BATCH];
            v4i b[BATCH][NC];
            unsigned left = rest;
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                a[i] = -1;
                if (left) {
                    a[i] = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
                    left &= ~(unsigned)__ballot(id == a[i]);
#pragma unroll
                    for (int c = 0; c < NC; ++c) b[i][c] = lora_load_b(L, a[i], N, n0 + 16 * c, s);
                }
            }
            rest = left;
            if (!split) {
                V = lora_split<IN>(v);
                split = true;
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if (a[i] < 0) continue;
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    v4f t = lora_mfma<IN>(b[i][c], V.lo, v4f{0, 0, 0, 0});
                    t = lora_mfma<IN>(b[i][c], V.hi, t);
                    if (id == a[i])
#pragma unroll
                        for (int q = 0; q < 4; ++q) delta[c][q] = fmaf(t[q], V.back, delta[c][q]);
                }
            }
        }
    }
}

}  // namespace w4a8
