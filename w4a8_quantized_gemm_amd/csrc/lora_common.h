// The outer product of low-rank adapters, as the epilogues of the shared
// projection's kernels add it: delta[m][n] = sum_r V[m][r] B[a(m)][n][r].
//
// A 16 x 16 block (16 channels, 16 rows of X) takes one 16 x 16 x 32 matrix
// instruction per 32 ranks and operand part.  B is used as stored (fp16 or
// bfloat16, 16 bytes per lane straight from memory); V is float32 and is
// split into operands of B's type, each rounded to nearest:
//   bfloat16: three parts of 8 bits, V exactly from 2^-100 on (two, 16 bits,
//     took 754 us against 760 at 4096 x 28672 x 8192, rank 16, and 22.9
//     against 23.4 at 47 x 11008 x 4096, rank 64);
//   fp16: the 32 ranks of a row are first scaled by a power of two that
//     brings their largest to [2^14, 2^15) (V's range is not fp16's), then
//     split into two parts, the second times 2^11 so that it keeps its bits
//     where the first is subnormal.  V is met within 2^-23, one unit in its
//     last place, or 2^-50 of the largest of the 32 ranks.
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

// Operand parts of 8 ranks of one row, the smallest first, and the factor of
// their products.
template <int IN>
struct LoraV {
    static constexpr int PARTS = IN == 1 ? 2 : 3;
    v4i part[PARTS];
    float back;
};
// fp16: the second part's factor, taken back in the sums.
constexpr float kLoraLow = 2048.0f;

// v: 8 of a row's 32 ranks; the lanes that hold the other 24 are this lane's
// number with the bits X1 and X2 flipped.
template <int IN, int X1 = 16, int X2 = 32>
__device__ __forceinline__ LoraV<IN> lora_split(const float (&v)[8]) {
    LoraV<IN> o;
    constexpr int P = LoraV<IN>::PARTS;
    unsigned h[P][8];
    if constexpr (IN == 1) {
        unsigned m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const unsigned b = __builtin_bit_cast(unsigned, v[j]) & 0x7FFFFFFFu;
            m = b > m ? b : m;
        }
        const unsigned m1 = __shfl_xor(m, X1, 64);
        m = m1 > m ? m1 : m;
        const unsigned m2 = __shfl_xor(m, X2, 64);
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
            const float d = x - (float)a;  // NaN where a is infinite: no low part then
            const _Float16 b = (_Float16)(d == d ? d * kLoraLow : 0.0f);
            h[1][j] = __builtin_bit_cast(unsigned short, a);
            h[0][j] = __builtin_bit_cast(unsigned short, b);
        }
    } else {
        o.back = 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float d = v[j];
#pragma unroll
            for (int p = P - 1; p >= 0; --p) {
                h[p][j] = __builtin_bit_cast(unsigned short, (__bf16)d);  // to nearest even
                d -= __builtin_bit_cast(float, h[p][j] << 16);
                d = d == d ? d : 0.0f;
            }
        }
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
        o.part[p] = v4i{(int)(h[p][0] | h[p][1] << 16), (int)(h[p][2] | h[p][3] << 16),
                        (int)(h[p][4] | h[p][5] << 16), (int)(h[p][6] | h[p][7] << 16)};
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

// t[c] += the products of four channel blocks and one operand part (fp16) or
// all three (bfloat16), inside a tile kernel, whose accumulators fill the
// AGPRs.  There the compiler would give these instructions AGPR operands too
// and move accumulators out of their way (and, where it runs out of
// registers, has stored an accumulator incompletely), so they are issued in
// assembly on VGPRs: five wait states for the operands, the dependent
// instructions four apart, and 20 wait states (see mfma_loop_exit_wait)
// before anything reads the results or overwrites the operands.
#define LORA_MFMA4(OP, V)                                                                        \
    OP " %0, %4, " V ", %0\n\t" OP " %1, %5, " V ", %1\n\t" OP " %2, %6, " V ", %2\n\t" OP        \
       " %3, %7, " V ", %3\n\t"
#define LORA_MFMA4_WAIT "s_nop 7\n\ts_nop 7\n\ts_nop 3"
__device__ __forceinline__ void lora_mfma4_f16(const v4i (&b)[4], v4i v, v4f (&t)[4]) {
    asm volatile("s_nop 4\n\t" LORA_MFMA4("v_mfma_f32_16x16x32_f16", "%8") LORA_MFMA4_WAIT
                 : "+&v"(t[0]), "+&v"(t[1]), "+&v"(t[2]), "+&v"(t[3])
                 : "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]), "v"(v));
}
__device__ __forceinline__ void lora_mfma4_bf16(const v4i (&b)[4], const v4i (&v)[3],
                                                v4f (&t)[4]) {
    asm volatile("s_nop 4\n\t" LORA_MFMA4("v_mfma_f32_16x16x32_bf16", "%8")
                     LORA_MFMA4("v_mfma_f32_16x16x32_bf16", "%9")
                         LORA_MFMA4("v_mfma_f32_16x16x32_bf16", "%10") LORA_MFMA4_WAIT
                 : "+&v"(t[0]), "+&v"(t[1]), "+&v"(t[2]), "+&v"(t[3])
                 : "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]), "v"(v[0]), "v"(v[1]), "v"(v[2]));
}
#undef LORA_MFMA4_WAIT
#undef LORA_MFMA4

// y[c] += the product of NC channel blocks for one adapter: bfloat16
// accumulates onto y in the matrix core, fp16 is scaled back and added.
// TILE: inside a tile kernel.
template <int IN, bool TILE, int NC>
__device__ __forceinline__ void lora_mac(const v4i (&b)[NC], const LoraV<IN>& V, v4f (&y)[NC]) {
    static_assert(!TILE || NC == 4, "four channel blocks");
    v4f t[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) t[c] = IN == 2 ? y[c] : v4f{0, 0, 0, 0};
    if constexpr (IN == 2 && TILE) {
        lora_mfma4_bf16(b, V.part, t);
    } else {
#pragma unroll
        for (int p = 0; p < LoraV<IN>::PARTS; ++p) {
            if constexpr (TILE) {
                lora_mfma4_f16(b, V.part[p], t);
            } else {
#pragma unroll
                for (int c = 0; c < NC; ++c) t[c] = lora_mfma<IN>(b[c], V.part[p], t[c]);
            }
            if (IN == 1 && p == 0)
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int q = 0; q < 4; ++q) t[c][q] *= 1.0f / kLoraLow;
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) y[c][q] = IN == 2 ? t[c][q] : fmaf(t[c][q], V.back, y[c][q]);
}

// y[c][v] += the adapter's product for row (lane % 16), channel
// n0 + 16 c + 4 (lane / 16) + v, of the 16 rows whose adapters are `id`
// (equal for the four lanes of a row); get_v(s) gives the row's operands of
// the s-th 32 ranks.  Adapters are taken four at a time (one with several
// channel blocks), so their operands are in flight together; every 32 ranks
// are one pass.
template <int IN, bool TILE, int NC, typename GetV>
__device__ __forceinline__ void lora_add(const LoraArgs& L, int id, int N, int n0, GetV get_v,
                                         v4f (&y)[NC]) {
    constexpr int BATCH = NC == 1 ? 4 : 1;
    const unsigned any = (unsigned)__ballot(id >= 0) & 0xFFFFu;
    if (any == 0) return;
    for (int s = 0; 32 * s < L.R; ++s) {
        const LoraV<IN> V = get_v(s);
        unsigned rest = any;
        while (rest) {
            int a[BATCH];
            v4i b[BATCH][NC];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                a[i] = -1;
                if (rest) {
                    a[i] = __builtin_amdgcn_readlane(id, __builtin_ctz(rest));
                    rest &= ~(unsigned)__ballot(id == a[i]);
#pragma unroll
                    for (int c = 0; c < NC; ++c) b[i][c] = lora_load_b(L, a[i], N, n0 + 16 * c, s);
                }
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if (a[i] < 0) continue;
                v4f t[NC];
#pragma unroll
                for (int c = 0; c < NC; ++c) t[c] = y[c];
                lora_mac<IN, TILE>(b[i], V, t);
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int q = 0; q < 4; ++q) y[c][q] = id == a[i] ? t[c][q] : y[c][q];
            }
        }
    }
}

// B operands of one adapter held in registers over consecutive row blocks,
// for adapters of at most 32 NS ranks: 128 of them in the 256-row tile kernel,
// 32 in the 128-row one, which spills 21 registers with 64.  Held against
// loaded again for every block, us: 4096 x 28672 x 8192 (256 rows) rank 16
// 800 / 815, 64 894 / 952, 128 1122 / 1257; 2048 x 4096 x 4096 (128 rows)
// rank 16 51.1 / 51.5, 32 56.5 / 56.9, and beyond 32 ranks, where both load,
// 40 69 / 68, 128 125 / 124.
template <int NS>
struct LoraHeld {
    v4i b[NS][4];
    int a = -1;
};

// lora_add for the tile kernels, which walk many row blocks of the same
// channels: a block whose rows all select one adapter (prompts: almost every
// block) uses the held operands and needs no select.
template <int IN, int NS, typename GetV>
__device__ __forceinline__ void lora_add_held(const LoraArgs& L, int id, int N, int n0, GetV get_v,
                                              LoraHeld<NS>& held, v4f (&y)[4]) {
    const int a = __builtin_amdgcn_readfirstlane(id);
    if (a < 0 || L.R > 32 * NS || __ballot(id == a) != ~0ull) {
        lora_add<IN, true>(L, id, N, n0, get_v, y);
        return;
    }
    if (held.a != a) {
        held.a = a;
#pragma unroll
        for (int s = 0; s < NS; ++s)
            if (32 * s < L.R)
#pragma unroll
                for (int c = 0; c < 4; ++c) held.b[s][c] = lora_load_b(L, a, N, n0 + 16 * c, s);
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        if (32 * s >= L.R) continue;
        lora_mac<IN, true>(held.b[s], get_v(s), y);
    }
}

// Whether the results of a row that has an adapter hold a NaN (per lane).
template <int NC>
__device__ __forceinline__ bool lora_nan(int id, const v4f (&y)[NC]) {
    bool nan = false;
#pragma unroll
    for (int c = 0; c < NC; ++c)
        nan |= __builtin_isunordered(y[c][0], y[c][1]) || __builtin_isunordered(y[c][2], y[c][3]);
    return nan && id >= 0;
}

// Results that came out as NaN are formed again, y = base + V . B in plain
// float32: an infinite element of B meets parts of V of both signs or of
// zero, and V may lie beyond its first part's range, where the definition
// gives an infinity or a number.  Called once behind the adapters' products of
// a block (y, id, m, n0 as in lora_add); base(c) gives its scaled sums.  The
// branch is not taken for finite operands, and rows whose V holds a NaN, whose
// results are NaN, are left (2048 x 11008 x 4096, rank 32: 108 us, 203 where
// every 16th row of X is NaN, 224 where all are; formed again, 400 and 604).
// True where y may have changed, in any lane.
template <int IN, int NC, typename Base>
__device__ __forceinline__ bool lora_redo(const LoraArgs& L, int id, int m, int N, int n0,
                                          Base base, v4f (&y)[NC]) {
    bool sound = lora_nan(id, y);
    if (__builtin_expect(__ballot(sound) == 0, 1)) return false;
    const float* v = L.V + (size_t)m * L.R;
    if (sound)  // a row with a NaN in V has NaN results
        for (int r = 0; r < L.R; r += 8) {
            const v4f a = *reinterpret_cast<const v4f*>(v + r);
            const v4f b = *reinterpret_cast<const v4f*>(v + r + 4);
            sound = sound && !__builtin_isunordered(a[0], a[1]) &&
                    !__builtin_isunordered(a[2], a[3]) && !__builtin_isunordered(b[0], b[1]) &&
                    !__builtin_isunordered(b[2], b[3]);
        }
    if (__ballot(sound) == 0) return false;
    unsigned redo = 0;  // bit 4 c + q
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const v4f s = base(c);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (sound && y[c][q] != y[c][q]) {
                redo |= 1u << (4 * c + q);
                y[c][q] = s[q];
            }
    }
    const int G = (threadIdx.x & 63) >> 4;
#pragma clang loop unroll(disable)
    for (int k = 0; k < 4 * NC; ++k) {
        float sum = 0.0f;
        if ((redo >> k) & 1) {
            const size_t row = (size_t)id * N + n0 + 16 * (k >> 2) + 4 * G + (k & 3);
            const uint8_t* w = reinterpret_cast<const uint8_t*>(L.B) + row * L.R * 2;
#pragma clang loop unroll(disable)
            for (int r = 0; r < L.R; r += 8) {
                const v4i b = load16(w + 2 * r);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const unsigned h = ((unsigned)b[j >> 1] >> (16 * (j & 1))) & 0xFFFFu;
                    const float x = IN == 1 ? (float)__builtin_bit_cast(_Float16, (unsigned short)h)
                                            : __builtin_bit_cast(float, h << 16);
                    sum = fmaf(v[r + j], x, sum);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (k == 4 * c + q && ((redo >> k) & 1)) y[c][q] += sum;
    }
    return true;
}

}  // namespace w4a8
