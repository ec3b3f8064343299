// The streamed-tile kernel's body, shared by the plain kernels and those that
// add low-rank adapters in their epilogue.
#pragma once
#include <type_traits>

#include "device_common.h"
#include "ffn_common.h"
#include "launch.h"
#include "lora_common.h"

namespace w4a8 {

constexpr size_t kMaxLdsBytes = 160 * 1024;  // LDS one workgroup may hold on gfx950

// Panels (64 channels, four tiles) that NTW consecutive tiles can touch.
template <int NTW>
__host__ __device__ constexpr int stream_param_span() {
    return (NTW + 3) / 4 + 1;
}

__device__ __forceinline__ v4i buf_load_v4(__amdgpu_buffer_rsrc_t r, unsigned voff,
                                           unsigned soff) {
    return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}

// Swizzled 16-byte piece position of row R's piece c in a 16 x 128-byte X
// tile held in LDS (row stride 128 bytes): conflict-free for the row-wise
// writes and for the MFMA-layout reads below.
__device__ __forceinline__ int xpiece(int R, int c) {
    return R * 128 + 16 * (c ^ ((R & 7) ^ ((R >> 3) & 1)));
}

// W4A8 decode-shaped GEMM (M < 64).  One workgroup per NTW packed tiles
// (16 channels each) and one 16-row block of X (NTW and ks are chosen by
// the host from the shape); its `ks` waves take interleaved K-tiles (wave w:
// w, w + ks, ...), so at any moment a CU reads adjacent tiles of its channel
// rows.  Each wave keeps D K-tiles of weight loads in flight (a register
// ring refilled as each stage is consumed); the weight stream is loaded
// non-temporally.  The per-group parameters of the workgroup's tiles are
// copied to LDS once (whole 64-byte panel rows) when they fit.  X tiles
// (L2-resident) are loaded eight whole 128-byte rows per instruction and
// re-laid out through a per-wave LDS slot into the MFMA operand layout.
// The ks partial tiles are summed by all threads of the workgroup in wave
// order (exact).
// WK selects the weight kind (the rest of the kernel is shared):
//   kWkLQQ  LiquidQuant codes + group parameters, INT8 matrix cores;
//   kWkW8   the W8A8 comparison: INT8 weights in the 8-bit tile layout
//           (2 KiB per tile, a lane's 32 bytes as two 16-byte halves 1 KiB
//           apart), used as B operands without decode;
//   kWkF8   sign-magnitude INT4 codes -> e4m3 by byte table, X is e4m3,
//           one v_mfma_scale_f32_16x16x128_f8f6f4 per tile (unit scales),
//           float32 accumulation; epilogue scale sw[n];
//   kWkF8G  the same with per-group scales folded into the FP8 weights:
//           each tile's table is e4m3(|q| f) for the lane's channel and
//           group (fsc group-major [K/GROUP][N]; with 64-wide groups lane
//           quarter G lies in group 2 kt + G/2), loaded with the weights,
//           and the epilogue scales by tsc[0].
// OUT: 0 = fp16 (INT8 kinds) or bf16 (FP8 kinds), 1 = int32 or float32, 2 = bf16
// (W4A8).
constexpr int kWkLQQ = 0, kWkW8 = 1, kWkF8 = 2, kWkF8G = 3;

// LORA (1: fp16, 2: bfloat16 adapters; W4A8 to fp16 only): the epilogue adds
// each row's low-rank adapter to its scaled sums before the one rounding.
// HROWS (1 or 2; W4A8, one row block): X is not INT8 but the float32 rows `ffn` of
// that many rows with their partial maxima, and a wave quantises each K-tile as
// it comes to it (the rows' scales are taken once, behind the first loads).
// GLU (1: SiLU, 2: GELU; W4A8 only): the first half of a workgroup's tiles lie
// in the gate half of N = 2F, the others are the same ones of the up half, and
// the epilogue writes act(gate) up with the largest of each row's 16 channels.
template <int NTW, int D, int OUT, int GROUP, bool LDSP, int WK, int RB, int LORA, int GLU = 0,
          int HROWS = 0>
__device__ __forceinline__ void stream_body(
    const int8_t* __restrict__ X, const float* __restrict__ sx, const uint8_t* __restrict__ wq,
    const uint8_t* __restrict__ s_u8, const uint8_t* __restrict__ a_u8,
    const float* __restrict__ sw, void* __restrict__ Y, int M, int N, int K, int ks,
    const int* __restrict__ offsets, const float* __restrict__ fsc,
    const float* __restrict__ tsc, const LoraArgs& lora, const FfnRows& ffn = {}) {
    static_assert(GLU == 0 || (LORA == 0 && WK == kWkLQQ && NTW % 2 == 0), "pairs of tiles");
    static_assert(HROWS == 0 || (HROWS <= 2 && LORA == 0 && GLU == 0 && WK == kWkLQQ && RB == 1),
                  "one or two float rows");
    static_assert(LORA == 0 || (OUT == 0 && WK == kWkLQQ), "adapters: W4A8 to fp16");
    constexpr bool W8 = WK == kWkW8;
    constexpr bool F8 = WK == kWkF8 || WK == kWkF8G;
    using Acc = std::conditional_t<F8, v4f, v4i>;
    extern __shared__ int red[];
    // Grouped problems (offsets != nullptr): expert blockIdx.z owns rows
    // offsets[e] .. offsets[e+1]-1 of X and Y and the e-th slab of the
    // packed weights.  Rows are clamped to [0, M], so bad offsets can only
    // leave rows unwritten, never move an access out of the buffers.
    int row_lo = 0, row_hi = M;
    if (offsets) {
        const int e = blockIdx.z;
        row_lo = min(max(offsets[e], 0), M);
        row_hi = min(max(offsets[e + 1], row_lo), M);
        wq += (size_t)e * N * (W8 ? K : K / 2);
        s_u8 += (size_t)e * N * (K / GROUP);
        a_u8 += (size_t)e * N * (K / GROUP);
        sw += (size_t)e * N;
    }
    const int m0 = row_lo + blockIdx.y * (16 * RB);
    if (m0 >= row_hi) return;  // whole workgroup: no rows of this expert here
    // X through LDS pays where X is a large share of the loads (narrow
    // workgroups: 2 KB of X per K-tile against NTW KB of weights).
    constexpr bool kXlds = true;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, G = lane >> 4;
    const int KT = K / kTileK;
    const int groups = K / GROUP;
    // Workgroups are dealt round-robin to the eight XCDs (b -> b % 8), each
    // with its own L2: give workgroups b and b + 8 adjacent tile groups, so
    // the parameter panels that neighbouring groups share are read once per
    // XCD (when the group count is a multiple of 8).
    const int nwg = gridDim.x, b = blockIdx.x;
    const int g = (nwg & 7) ? b : (b & 7) * (nwg >> 3) + (b >> 3);
    constexpr int NTH = GLU ? NTW / 2 : NTW;  // tiles of one half
    const int nt0 = g * NTH;
    // tile t of the workgroup
    auto tile_of = [&](int t) {
        return t < NTH ? nt0 + t : N / 2 / kTileN + nt0 + t - NTH;
    };
    const int nk = (KT - wave + ks - 1) / ks;  // K-tiles of this wave (>= 1: ks <= KT)
    // i-th K-tile of this wave (i < nk)
    auto kt_of = [&](int i) { return wave + ks * i; };

    const __amdgpu_buffer_rsrc_t x_rsrc =
        HROWS ? __builtin_amdgcn_make_buffer_rsrc(ffn.h, (short)0, 4 * M * K, 0x00020000)
              : __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(X), (short)0, M * K,
                                                  0x00020000);
    const __amdgpu_buffer_rsrc_t w_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(wq), (short)0, (int)((size_t)N * K / (W8 ? 1 : 2)), 0x00020000);
    const __amdgpu_buffer_rsrc_t f_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<float*>(fsc), (short)0,
        WK == kWkF8G ? (int)((size_t)(K / GROUP) * N * sizeof(float)) : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t s_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(s_u8), (short)0, (int)((size_t)N * K / GROUP), 0x00020000);
    const __amdgpu_buffer_rsrc_t a_rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(a_u8), (short)0, (int)((size_t)N * K / GROUP), 0x00020000);
    // X loads (a row >= M lies past the buffer end and reads as 0).  With
    // the LDS re-layout, lane l takes 16-byte piece (l & 7) of rows
    // m0 + (l >> 3) and m0 + 8 + (l >> 3); otherwise lane (r, G) loads its
    // MFMA operand directly: row m0 + r, columns 32G .. 32G+31.
    // (HROWS: 64 / HROWS lanes take 2 HROWS consecutive elements each of a row)
    constexpr int HL = HROWS ? 64 / HROWS : 64;  // lanes of a row
    const int hrow = lane / HL, hcol = 2 * HROWS * (lane % HL);
    const unsigned xvoff =
        HROWS ? 4u * ((unsigned)hrow * (unsigned)K + (unsigned)hcol)
        : kXlds ? (unsigned)(m0 + (lane >> 3)) * (unsigned)K + 16u * (unsigned)(lane & 7)
              : (unsigned)(m0 + r) * (unsigned)K + 32u * (unsigned)G;
    const unsigned xvoff8 = kXlds ? xvoff + 8u * (unsigned)K : xvoff + 16u;
    const unsigned wvoff = (unsigned)lane * 16u;
    const int gsub = (GROUP == 64) ? (G >> 1) : 0;  // group within the K-tile

    // ---- LDS: [parameters (LDSP)] [one 2 KB X slot per wave]; the
    // reduction at the end reuses it from offset 0.
    const int p0 = nt0 >> 2;
    const int np = ((nt0 + NTH - 1) >> 2) - p0 + 1;
    uint8_t* lds_s = reinterpret_cast<uint8_t*>(red);
    // (GLU: the gate half's panels, then the up half's)
    constexpr int HALVES = GLU ? 2 : 1;
    uint8_t* lds_a = lds_s + (size_t)HALVES * np * groups * 64;
    const int pbytes = LDSP ? 2 * HALVES * stream_param_span<NTH>() * groups * 64 : 0;
    uint8_t* xslot = reinterpret_cast<uint8_t*>(red) + pbytes + wave * (2048 * RB);
    // MFMA operand layout: lane (r, G) holds row r, columns 32G .. 32G+31.
    const int xw0 = xpiece(lane >> 3, lane & 7), xw1 = xpiece(8 + (lane >> 3), lane & 7);
    const int xr0 = xpiece(r, 2 * G), xr1 = xpiece(r, 2 * G + 1);

    constexpr int WPT = W8 ? 2 : 1;  // 16-byte weight loads per lane and tile
    constexpr int NF = WK == kWkF8G ? NTW : 1;  // folded factors per stage
    struct Stage {
        v4i x0[RB], x1[RB];
        v4i w[NTW * WPT];
        float f[NF];
    };
    // The feed-forward forms run their K-tiles in one loop without drain copies
    // (a wave has few K-tiles there, and code that runs once is fetched at the
    // pace of instruction cache misses): a stage past the wave's last K-tile is
    // loaded from past the buffers' ends, which reads zeros and no memory (gate and
    // up of one row, 8192 x 28672: 40.6 -> 38.7 us).
    constexpr bool ONELOOP = GLU != 0 || HROWS != 0;
    auto issue = [&](int kt_, Stage& st) {
        const unsigned past = ONELOOP && kt_ >= KT ? 0x80000000u : 0u;
        const int kt = ONELOOP ? min(kt_, KT - 1) : kt_;
        const unsigned xvo = xvoff | past, xvo8 = xvoff8 | past, wvo = wvoff | past;
        const unsigned so = (unsigned)(kt * kTileK * (HROWS ? 4 : 1));
        if constexpr (HROWS == 1) {
            const auto v = __builtin_amdgcn_raw_buffer_load_b64(x_rsrc, xvo, so, 0);
            st.x0[0] = v4i{(int)v[0], (int)v[1], 0, 0};
        } else if constexpr (HROWS == 2) {
            st.x0[0] = buf_load_v4(x_rsrc, xvo, so);
        }
#pragma unroll
        for (int rb = 0; rb < (HROWS ? 0 : RB); ++rb) {
            const unsigned ro = 16u * (unsigned)rb * (unsigned)K;  // row block rb
            st.x0[rb] = __builtin_bit_cast(
                v4i, __builtin_amdgcn_raw_buffer_load_b128(x_rsrc, xvo + ro, so, 0));
            st.x1[rb] = __builtin_bit_cast(
                v4i, __builtin_amdgcn_raw_buffer_load_b128(x_rsrc, xvo8 + ro, so, 0));
        }
#pragma unroll
        for (int t = 0; t < NTW; ++t) {
            if constexpr (W8) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    st.w[2 * t + u] = __builtin_bit_cast(
                        v4i, __builtin_amdgcn_raw_buffer_load_b128(
                                 w_rsrc, wvoff,
                                 (unsigned)(((size_t)tile_of(t) * KT + kt) * 2048 + 1024 * u),
                                 kNonTemporal));
            } else {
                st.w[t] = __builtin_bit_cast(
                    v4i, __builtin_amdgcn_raw_buffer_load_b128(
                             w_rsrc, wvo, (unsigned)(((size_t)tile_of(t) * KT + kt) * kTileBytes),
                             kNonTemporal));
            }
            if constexpr (WK == kWkF8G) {
                // factor of this lane's channel and group, loaded with the
                // stage so using it waits for nothing younger
                const int gi = GROUP == 64 ? 2 * kt + (G >> 1) : kt;
                st.f[t] = __builtin_bit_cast(
                    float, __builtin_amdgcn_raw_buffer_load_b32(
                               f_rsrc, (unsigned)((size_t)gi * N + (nt0 + t) * kTileN + r) * 4u,
                               0u, 0));
            }
        }
    };
    auto params = [&](int kt, int t, unsigned& s, unsigned& a) {
        const int j = kt * (kTileK / GROUP) + gsub;
        const int nt = tile_of(t);
        if (LDSP) {
            const int first = t < NTH ? p0 : (N / 2 >> 6) + p0 - np;
            const int o = (((nt >> 2) - first) * groups + j) * 64 + 4 * r + (nt & 3);
            s = lds_s[o];
            a = lds_a[o];
        } else {
            const unsigned po = (unsigned)param_offset(nt * kTileN + r, j, groups);
            s = __builtin_amdgcn_raw_buffer_load_b8(s_rsrc, po, 0, 0);
            a = __builtin_amdgcn_raw_buffer_load_b8(a_rsrc, po, 0, 0);
        }
    };

    Acc acc[RB][NTW];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int t = 0; t < NTW; ++t) acc[rb][t] = Acc{};

    // (whole 16 bytes: the dynamic LDS behind it is read in such pieces)
    [[maybe_unused]] __shared__ alignas(16) unsigned htops[HROWS ? HROWS * 16 : 4];
    [[maybe_unused]] float hscale = 1.0f, hinv = 1.0f;  // of the lane's row
    // Multiply-accumulate of the K-tile held in stage S.
    auto consume = [&](const Stage& S, int kt) {
        v4i x0[RB], x1[RB];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            x0[rb] = S.x0[rb];
            x1[rb] = S.x1[rb];
            if constexpr (HROWS) {
                // the lane's codes; the other rows stay the zeros that were put
                // there at the start
                float v[4] = {};
#pragma unroll
                for (int j = 0; j < 2 * HROWS; ++j) {
                    const int b = S.x0[0][j];
                    v[j] = __builtin_bit_cast(float, b);
                }
                const unsigned q = quant4_fast(v[0], v[1], v[2], v[3], hscale, hinv);
                uint8_t* at = xslot + xpiece(hrow, hcol >> 4) + (hcol & 15);
                if constexpr (HROWS == 1) *reinterpret_cast<unsigned short*>(at) = (unsigned short)q;
                else *reinterpret_cast<unsigned*>(at) = q;
                x0[0] = *reinterpret_cast<const v4i*>(xslot + xr0);
                x1[0] = *reinterpret_cast<const v4i*>(xslot + xr1);
            } else if constexpr (kXlds) {
                // X tile -> MFMA layout through this wave's LDS slot (LDS
                // operations of one wave complete in order).
                uint8_t* xs = xslot + rb * 2048;
                *reinterpret_cast<v4i*>(xs + xw0) = S.x0[rb];
                *reinterpret_cast<v4i*>(xs + xw1) = S.x1[rb];
                x0[rb] = *reinterpret_cast<const v4i*>(xs + xr0);
                x1[rb] = *reinterpret_cast<const v4i*>(xs + xr1);
            }
        }
#pragma unroll
        for (int t = 0; t < NTW; ++t) {
            if constexpr (W8) {
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) {
                    acc[rb][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x0[rb], S.w[2 * t],
                                                                       acc[rb][t], 0, 0, 0);
                    acc[rb][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x1[rb], S.w[2 * t + 1],
                                                                       acc[rb][t], 0, 0, 0);
                }
                continue;
            } else if constexpr (F8) {
                unsigned lo = kE4m3LutLo, hi = kE4m3LutHi;
                if constexpr (WK == kWkF8G) e4m3_fold_table(S.f[t], lo, hi);
                const v4i w = S.w[t];
                const v8i Bf = v8i{(int)int4_to_e4m3_lo(w.x, lo, hi), (int)int4_to_e4m3_hi(w.x, lo, hi),
                                   (int)int4_to_e4m3_lo(w.y, lo, hi), (int)int4_to_e4m3_hi(w.y, lo, hi),
                                   (int)int4_to_e4m3_lo(w.z, lo, hi), (int)int4_to_e4m3_hi(w.z, lo, hi),
                                   (int)int4_to_e4m3_lo(w.w, lo, hi), (int)int4_to_e4m3_hi(w.w, lo, hi)};
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) {
                    const v8i A = v8i{x0[rb].x, x0[rb].y, x0[rb].z, x0[rb].w,
                                      x1[rb].x, x1[rb].y, x1[rb].z, x1[rb].w};
                    // formats 0/0 = e4m3 x e4m3; E8M0 scale 127 = 2^0 on both sides
                    acc[rb][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        A, Bf, acc[rb][t], 0, 0, 0, 127, 0, 127);
                }
                continue;
            }
            unsigned s, a;
            params(kt, t, s, a);
            const u16x2 s2 = u16x2{(unsigned short)s, (unsigned short)s};
            const unsigned short aa = (unsigned short)(a * 0x101u);
            const u16x2 a4 = u16x2{aa, aa};
            unsigned b[8];
            lqq_dequant8((unsigned)S.w[t].x, s2, a4, b[0], b[1]);
            lqq_dequant8((unsigned)S.w[t].y, s2, a4, b[2], b[3]);
            lqq_dequant8((unsigned)S.w[t].z, s2, a4, b[4], b[5]);
            lqq_dequant8((unsigned)S.w[t].w, s2, a4, b[6], b[7]);
            const v4i B0 = v4i{(int)b[0], (int)b[1], (int)b[2], (int)b[3]};
            const v4i B1 = v4i{(int)b[4], (int)b[5], (int)b[6], (int)b[7]};
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                acc[rb][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x0[rb], B0, acc[rb][t], 0, 0, 0);
                acc[rb][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x1[rb], B1, acc[rb][t], 0, 0, 0);
            }
        }
    };

    // Stage d holds this wave's K-tile i + d.  The steady-state loop has no
    // conditional work, so the load counter waits it needs are exact (one
    // stage at a time) and D stages stay in flight; the last 2D-1 K-tiles
    // at most are drained after it.
    Stage st[D];
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (ONELOOP || d < nk) issue(kt_of(d), st[d]);

    // Parameter copy, behind the first weight loads (panels p0 .. p0+np-1
    // are contiguous in the panel-order arrays).
    if (LDSP && WK == kWkLQQ) {
        const int n16 = np * groups * 4;  // 16-byte pieces per array and half
        const size_t base = (size_t)p0 * groups * 64;
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf) {
            const size_t from = base + (size_t)hf * (N / 2 >> 6) * groups * 64;
            const int to = hf * n16 * 16;
            for (int q = tid; q < n16; q += blockDim.x) {
                const v4i vs = *reinterpret_cast<const v4i*>(s_u8 + from + (size_t)q * 16);
                const v4i va = *reinterpret_cast<const v4i*>(a_u8 + from + (size_t)q * 16);
                *reinterpret_cast<v4i*>(lds_s + to + q * 16) = vs;
                *reinterpret_cast<v4i*>(lds_a + to + q * 16) = va;
            }
        }
        if constexpr (!HROWS) __syncthreads();
    }
    if constexpr (HROWS) {
        // largest of each row's parts: every wave takes a share of all rows
        unsigned top[HROWS] = {};
        for (int q = tid; q < ffn.ntops; q += blockDim.x)
#pragma unroll
            for (int m = 0; m < HROWS; ++m)
                top[m] = MaxU32{}(top[m], ffn.tops[(size_t)m * ffn.ntops + q]);
#pragma unroll
        for (int m = 0; m < HROWS; ++m) {
            top[m] = wave_reduce(top[m], MaxU32{});
            if (lane == 0) htops[m * 16 + wave] = top[m];
        }
        *reinterpret_cast<v4i*>(xslot + 32 * lane) = v4i{0, 0, 0, 0};
        *reinterpret_cast<v4i*>(xslot + 32 * lane + 16) = v4i{0, 0, 0, 0};
        __syncthreads();
        unsigned all = 0;
        for (int w = 0; w < ks; ++w) all = MaxU32{}(all, htops[hrow * 16 + w]);
        hscale = row_scale_bits(all);
        hinv = __fdiv_rn(1.0f, hscale);
    }

    if constexpr (ONELOOP) {
#pragma clang loop unroll(disable)
        for (int i = 0; i < nk; i += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                consume(st[d], min(kt_of(i + d), KT - 1));
                issue(kt_of(i + d + D), st[d]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    int i = ONELOOP ? nk : 0;
    for (; i + 2 * D <= nk; i += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            consume(st[d], kt_of(i + d));
            issue(kt_of(i + d + D), st[d]);
            // keep each refill right behind its stage's use (the scheduler
            // would otherwise sink every refill to the end of the iteration)
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int d = 0; d < D; ++d) {
        if (i + d < nk) {
            consume(st[d], kt_of(i + d));
            if (i + d + D < nk) issue(kt_of(i + d + D), st[d]);
        }
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (i + D + d < nk) consume(st[d], kt_of(i + D + d));

    // Sum the ks partial tiles: element e = ((rb * NTW + t) * 4 + v) * 64 + l
    // of wave w lives at red[w * RB * NTW * 256 + e] (reusing the parameter
    // LDS).
    // (float32 sums, for the FP8 kinds, are added in the same wave order.)
    using Sum = std::conditional_t<F8, float, int>;
    Sum* reds = reinterpret_cast<Sum*>(red);
    __syncthreads();
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int t = 0; t < NTW; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                reds[(((wave * RB + rb) * NTW + t) * 4 + v) * 64 + lane] = acc[rb][t][v];
    __syncthreads();
    if constexpr (LORA != 0) {
        // a wave takes whole 16 x 16 blocks, lane (r, G) row r and channels
        // 4G .. 4G + 3 (the adapters' product layout)
        for (int u = wave; u < RB * NTW; u += ks) {
            const int rb = u / NTW, t = u % NTW;
            const int m = m0 + 16 * rb + r, n = (nt0 + t) * kTileN;
            const bool live = m < row_hi;
            const int id = lora_id(lora, m, live);
            const float xs = live ? sx[m] : 0.0f;
            const float* ws = sw + n + 4 * G;  // (4-byte aligned only)
            v4i sum = v4i{0, 0, 0, 0};
            for (int w = 0; w < ks; ++w)
                sum += *reinterpret_cast<const v4i*>(
                    &red[((w * RB + rb) * NTW + t) * 256 + (r & 3) * 64 + 16 * (r >> 2) + 4 * G]);
            auto scaled = [&](int) {
                v4f s;
#pragma unroll
                for (int q = 0; q < 4; ++q) s[q] = ((float)sum[q] * xs) * ws[q];
                return s;
            };
            v4f y[1] = {scaled(0)};
            lora_add<LORA, false>(
                lora, id, N, n,
                [&](int s) {
                    float v[8];
                    lora_load_v(lora, m, id >= 0, s, v);
                    return lora_split<LORA>(v);
                },
                y);
            lora_redo<LORA>(lora, id, m, N, n, scaled, y);
            if (!live) continue;
            unsigned short h[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) h[q] = f32_to_f16_bits(y[0][q]);
            *reinterpret_cast<uint2*>(reinterpret_cast<unsigned short*>(Y) + (size_t)m * N + n +
                                      4 * G) =
                uint2{h[0] | ((unsigned)h[1] << 16), h[2] | ((unsigned)h[3] << 16)};
        }
        return;
    }
    if constexpr (GLU != 0) {
        // a wave's 64 elements are four rows of 16 channels of one tile pair
        constexpr int NPAIR = RB * NTH * 256;
        const int F = N / 2;
        for (int q = tid; q < NPAIR; q += blockDim.x) {
            const int rb = q / (NTH * 256), t = (q >> 8) % NTH, v = (q >> 6) & 3, l = q & 63;
            const int e = rb * (NTW * 256) + t * 256 + (q & 255);
            int sum[2] = {0, 0};
            for (int w = 0; w < ks; ++w) {
                sum[0] += red[w * (RB * NTW * 256) + e];
                sum[1] += red[w * (RB * NTW * 256) + NTH * 256 + e];
            }
            const int m = m0 + 16 * rb + 4 * (l >> 4) + v;
            const int n = (nt0 + t) * kTileN + (l & 15);
            const bool on = m < row_hi;
            const float x = on ? sx[m] : 0.0f;
            const float h =
                gated<GLU - 1>(((float)sum[0] * x) * sw[n], ((float)sum[1] * x) * sw[F + n]);
            const unsigned top = row16_reduce(abs_bits(h), MaxU32{});
            if (!on) continue;
            ffn.h[(size_t)m * F + n] = h;
            if ((l & 15) == 0) ffn.tops[(size_t)m * (F / 16) + n / 16] = top;
        }
        return;
    }
    const int nel = RB * NTW * 256;
    const float tval = WK == kWkF8G ? tsc[0] : 0.0f;
    for (int e = tid; e < nel; e += blockDim.x) {
        Sum sum = reds[e];
        for (int w = 1; w < ks; ++w) sum += reds[w * nel + e];
        const int rb = e / (NTW * 256), t = (e >> 8) % NTW, v = (e >> 6) & 3, l = e & 63;
        const int m = m0 + 16 * rb + 4 * (l >> 4) + v;  // accumulator row (X row)
        const int n = (nt0 + t) * kTileN + (l & 15);
        if (m < row_hi) {
            if constexpr (F8) {
                const float y = (sum * sx[m]) * (WK == kWkF8G ? tval : sw[n]);
                if (OUT == 1)
                    reinterpret_cast<float*>(Y)[(size_t)m * N + n] = y;
                else
                    reinterpret_cast<unsigned short*>(Y)[(size_t)m * N + n] = f32_to_bf16_bits(y);
            } else if (OUT == 1) {
                reinterpret_cast<int*>(Y)[(size_t)m * N + n] = sum;
            } else {
                float xs;
                if constexpr (HROWS) {
                    unsigned all = 0;
                    for (int w = 0; w < ks; ++w) all = MaxU32{}(all, htops[m * 16 + w]);
                    xs = row_scale_bits(all);
                } else {
                    xs = sx[m];
                }
                const float y = ((float)sum * xs) * sw[n];
                reinterpret_cast<unsigned short*>(Y)[(size_t)m * N + n] = f32_to_out16_bits<OUT>(y);
            }
        }
    }
}

}  // namespace w4a8
