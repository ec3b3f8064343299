// A whole mixture-of-experts layer on W4A8 weights for a few tokens.
//
//   Xq, sx = per-token INT8 of X                     (as w4a8_quant_act)
//   slot (t, j) with expert e = ids[t][j] in [0, E):
//     g, u = the two halves of (Xq[t] . W13[e]^T) sx[t] sw13[e]
//     h    = u g / (1 + exp(-g))                     (float32)
//     hq, sh = per-slot INT8 of h
//     y    = (hq . W2[e]^T) sh sw2[e]
//   Y[t] = sum_j weights[t][j] y(t, j)               (float32, j ascending)
//
// The weights of the chosen experts are the bulk of the bytes, so their stream
// bounds the layer.  A stream serves 16 rows of its expert, 32 or 64 where a
// batch has that many per expert; an expert with more rows repeats it.
#include "act_common.h"
#include "launch.h"
#include "mfma_common.h"
#include "stream_body.h"
#include "wave_common.h"

namespace w4a8 {

namespace {

// Head of the workspace: the experts that have slots, in order.
struct MoeActive {
    int expert, start, count, pad;
};
struct MoeHead {
    int active;  // experts with slots
    int total;   // slots with an expert
    int pad[2];
    MoeActive list[kMaxExperts];
};

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Workspace regions (every one starts on a 256-byte boundary).
struct MoeLayout {
    size_t slots, xq, sx, h, hq, sh, part, bytes;
    MoeLayout(int T, int k, int H, int F) {
        const size_t S = (size_t)T * k;
        size_t o = up256(sizeof(MoeHead));
        auto take = [&](size_t n) {
            const size_t at = o;
            o += up256(n);
            return at;
        };
        slots = take(S * sizeof(int));
        xq = take((size_t)T * H);
        sx = take((size_t)T * sizeof(float));
        h = take(S * F * sizeof(float));
        hq = take(S * F);
        sh = take(S * sizeof(float));
        part = take(S * H * sizeof(float));
        bytes = o;
    }
};

}  // namespace

template <int IN>
__device__ __forceinline__ void quant_row(const void* row, int K, int8_t* out, float* scale) {
    unsigned m = 0;
    for (int i = threadIdx.x; i < K / 8; i += blockDim.x) {
        const Row8<IN> r = load_row8<IN>(row, i);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = MaxU32{}(m, abs_bits(r.v[j]));
    }
    const float s = row_scale_bits(block_max_bits(m)), inv = __fdiv_rn(1.0f, s);
    if (threadIdx.x == 0) *scale = s;
    for (int i = threadIdx.x; i < K / 8; i += blockDim.x) {
        const Row8<IN> r = load_row8<IN>(row, i);
        reinterpret_cast<uint2*>(out)[i] =
            uint2{quant4_fast(r.v[0], r.v[1], r.v[2], r.v[3], s, inv),
                  quant4_fast(r.v[4], r.v[5], r.v[6], r.v[7], s, inv)};
    }
}

// Workgroup t < T quantises token t; workgroup T groups the slots.
template <int IN>
__global__ __launch_bounds__(1024) void moe_prepare_kernel(const void* __restrict__ X,
                                                           const int* __restrict__ ids, int T,
                                                           int E, int k, int H,
                                                           MoeHead* __restrict__ head,
                                                           int* __restrict__ slots,
                                                           int8_t* __restrict__ xq,
                                                           float* __restrict__ sx) {
    if ((int)blockIdx.x < T) {
        constexpr int EB = IN == 0 ? 4 : 2;
        const size_t t = blockIdx.x;
        quant_row<IN>(reinterpret_cast<const uint8_t*>(X) + t * H * EB, H, xq + t * H, sx + t);
        return;
    }
    extern __shared__ int lds[];
    const int S = T * k;
    int* hist = lds;
    int* cnt = hist + kGroupWaves * E;
    int* start = cnt + E;
    for (int i = threadIdx.x; i < kGroupWaves * E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    auto get = [&](int s) { return ids[s]; };
    group_count(hist, S, E, get);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int c = 0;
        for (int w = 0; w < kGroupWaves; ++w) c += hist[w * E + e];
        cnt[e] = c;
    }
    __syncthreads();
    expert_scan(cnt, start, E);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int p = start[e];
        for (int w = 0; w < kGroupWaves; ++w) {
            const int c = hist[w * E + e];
            hist[w * E + e] = p;
            p += c;
        }
    }
    __syncthreads();
    group_place(hist, S, E, get, [&](int p, int s) { slots[p] = s; });
    // the experts with slots, in order (one wave: a ballot counts those before)
    if (threadIdx.x < 64) {
        int n = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + threadIdx.x;
            const int c = e < E ? cnt[e] : 0;
            const uint64_t m = __ballot(c > 0);
            if (c > 0)
                head->list[n + __builtin_popcountll(m & ((1ull << threadIdx.x) - 1))] =
                    MoeActive{e, start[e], c, 0};
            n += __builtin_popcountll(m);
        }
        if (threadIdx.x == 0) {
            head->active = n;
            head->total = start[E];
        }
    }
}

// Per-slot INT8 of h (rows in grouped order).
__global__ __launch_bounds__(1024) void moe_quant_kernel(const float* __restrict__ h, int F,
                                                         const MoeHead* __restrict__ head,
                                                         int8_t* __restrict__ hq,
                                                         float* __restrict__ sh) {
    const size_t p = blockIdx.x;
    if ((int)p >= head->total) return;
    quant_row<0>(h + p * F, F, hq + p * F, sh + p);
}

// Workgroup -> group of channels.  Workgroups are dealt round-robin to the
// eight XCDs: give b and b + 8 neighbouring groups, so that a panel of group
// parameters (64 channels) is read into one XCD's L2.
__device__ __forceinline__ int channel_group(int b, int n) {
    return (n & 7) ? b : (b & 7) * (n >> 3) + (b >> 3);
}

// 16-channel tiles of each half per workgroup of the products (half a panel of
// group parameters).
constexpr int kMoeTiles = 2;

// One product of the layer for one expert and 32 channels of each half:
// HALVES = 2: the gate and up products of W13 (channel n and F + n), h = silu;
// HALVES = 1: the down product, scaled by the slot's weight, into part[slot].
// blockIdx.x: channel group, blockIdx.y: index into the active experts.  The
// `ks` waves take interleaved K-tiles and are summed in LDS (exact int32).
// Up to 16 RB rows share each decoded weight; the rows of an expert with more
// are dealt to the workgroups of blockIdx.z, and past those repeat the stream.
template <int HALVES, int RB, int D, int GROUP>
__global__ __launch_bounds__(512) void moe_product_kernel(
    const int8_t* __restrict__ Xq, const float* __restrict__ sx, const uint8_t* __restrict__ wq,
    const uint8_t* __restrict__ s_u8, const uint8_t* __restrict__ a_u8,
    const float* __restrict__ sw, const float* __restrict__ weights,
    const MoeHead* __restrict__ head, const int* __restrict__ slots, float* __restrict__ out,
    int N, int K, int k, int rows_in) {
    constexpr int NT = kMoeTiles, TT = HALVES * NT;  // weight tiles of the workgroup
    extern __shared__ int red[];
    if ((int)blockIdx.y >= head->active) return;
    const MoeActive act = head->list[blockIdx.y];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ks = blockDim.x >> 6;
    const int r = lane & 15, G = lane >> 4;
    const int KT = K / kTileK, groups = K / GROUP;
    const size_t e = act.expert;
    const int nh = N / HALVES;  // channels of one half
    const int part = blockIdx.z, sharers = gridDim.z;
    if (16 * RB * part >= act.count) return;
    const int nt0 = channel_group(blockIdx.x, gridDim.x) * NT;
    const int nk = wave < KT ? (KT - wave + ks - 1) / ks : 0;
    auto kt_of = [&](int i) { return wave + ks * i; };

    const __amdgpu_buffer_rsrc_t x_rsrc = buf_rsrc(Xq, (unsigned)rows_in * (unsigned)K);
    const __amdgpu_buffer_rsrc_t w_rsrc =
        buf_rsrc(wq + e * ((size_t)N * K / 2), (unsigned)((size_t)N * K / 2));
    const unsigned pbytes = (unsigned)((size_t)N * groups);
    const __amdgpu_buffer_rsrc_t s_rsrc = buf_rsrc(s_u8 + e * pbytes, pbytes);
    const __amdgpu_buffer_rsrc_t a_rsrc = buf_rsrc(a_u8 + e * pbytes, pbytes);
    const unsigned wvoff = (unsigned)lane * 16u;
    const unsigned pvoff = 4u * (unsigned)r + (GROUP == 64 ? 64u * (unsigned)(G >> 1) : 0u);
    auto tile_of = [&](int t) { return t < NT ? nt0 + t : nh / kTileN + nt0 + t - NT; };

    uint8_t* xslot = reinterpret_cast<uint8_t*>(red) + wave * (2048 * RB);
    const int xw0 = xpiece(lane >> 3, lane & 7), xw1 = xpiece(8 + (lane >> 3), lane & 7);
    const int xr0 = xpiece(r, 2 * G), xr1 = xpiece(r, 2 * G + 1);

    struct Stage {
        v4i x0[RB], x1[RB], w[TT];
        unsigned s[HALVES], a[HALVES];
    };
    for (int r0 = 16 * RB * part; r0 < act.count; r0 += 16 * RB * sharers) {
        // Rows (lane / 8) and 8 + (lane / 8) of row block rb, 16-byte piece
        // lane % 8: the row's token (W13) or its own place (W2).  Absent rows
        // get an offset past the buffer, which reads 0.
        unsigned xoff[RB][2];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int i = r0 + 16 * rb + 8 * u + (lane >> 3);
                unsigned row = act.start + i;
                if (HALVES == 2 && i < act.count) row = (unsigned)slots[row] / (unsigned)k;
                xoff[rb][u] = i < act.count ? row * (unsigned)K + 16u * (unsigned)(lane & 7)
                                            : 0xFFFFFF00u;
            }
        auto issue = [&](int kt, Stage& st) {
#pragma unroll
            for (int t = 0; t < TT; ++t)
                st.w[t] = __builtin_bit_cast(
                    v4i, __builtin_amdgcn_raw_buffer_load_b128(
                             w_rsrc, wvoff,
                             (unsigned)(((size_t)tile_of(t) * KT + kt) * kTileBytes),
                             kNonTemporal));
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf) {
                const unsigned po = 64u * ((unsigned)(tile_of(hf * NT) >> 2) * (unsigned)groups +
                                           (unsigned)(kt * (kTileK / GROUP)));
                st.s[hf] = buf_load4(s_rsrc, pvoff, po);
                st.a[hf] = buf_load4(a_rsrc, pvoff, po);
            }
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                st.x0[rb] = buf_load16(x_rsrc, xoff[rb][0], (unsigned)(kt * kTileK));
                st.x1[rb] = buf_load16(x_rsrc, xoff[rb][1], (unsigned)(kt * kTileK));
            }
        };
        v4i acc[RB][TT];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[rb][t] = v4i{0, 0, 0, 0};
        auto consume = [&](const Stage& S) {
            // X tiles -> matrix-core layout (lane (r, G): row r, columns
            // 32 G .. + 31) through this wave's LDS slots; LDS operations of
            // one wave complete in order
            v4i x0[RB], x1[RB];
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                uint8_t* xs = xslot + rb * 2048;
                *reinterpret_cast<v4i*>(xs + xw0) = S.x0[rb];
                *reinterpret_cast<v4i*>(xs + xw1) = S.x1[rb];
                x0[rb] = *reinterpret_cast<const v4i*>(xs + xr0);
                x1[rb] = *reinterpret_cast<const v4i*>(xs + xr1);
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int b = (nt0 & 3) + t % NT;
                const u16x2 s2 = scale_pair(S.s[t / NT], b), a4 = offset_quad(S.a[t / NT], b);
                unsigned q[8];
                lqq_dequant8((unsigned)S.w[t].x, s2, a4, q[0], q[1]);
                lqq_dequant8((unsigned)S.w[t].y, s2, a4, q[2], q[3]);
                lqq_dequant8((unsigned)S.w[t].z, s2, a4, q[4], q[5]);
                lqq_dequant8((unsigned)S.w[t].w, s2, a4, q[6], q[7]);
                const v4i B0 = v4i{(int)q[0], (int)q[1], (int)q[2], (int)q[3]};
                const v4i B1 = v4i{(int)q[4], (int)q[5], (int)q[6], (int)q[7]};
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) {
                    acc[rb][t] =
                        __builtin_amdgcn_mfma_i32_16x16x64_i8(x0[rb], B0, acc[rb][t], 0, 0, 0);
                    acc[rb][t] =
                        __builtin_amdgcn_mfma_i32_16x16x64_i8(x1[rb], B1, acc[rb][t], 0, 0, 0);
                }
            }
        };
        Stage st[D];
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (d < nk) issue(kt_of(d), st[d]);
        int i = 0;
        for (; i + 2 * D <= nk; i += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                consume(st[d]);
                issue(kt_of(i + d + D), st[d]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (i + d < nk) {
                consume(st[d]);
                if (i + d + D < nk) issue(kt_of(i + d + D), st[d]);
            }
        }
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (i + D + d < nk) consume(st[d]);

        // Sums over the waves, one row block at a time: element
        // (t * 4 + v) * 64 + l of wave w at red[w * TT * 256 + ...].
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            __syncthreads();
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    red[((wave * TT + t) * 4 + v) * 64 + lane] = acc[rb][t][v];
            __syncthreads();
            for (int q = tid; q < NT * 256; q += blockDim.x) {
                const int t = q >> 8, v = (q >> 6) & 3, l = q & 63;
                const int i_row = r0 + 16 * rb + 4 * (l >> 4) + v;
                if (i_row >= act.count) continue;
                const int p = act.start + i_row;  // place in grouped order
                const int slot = slots[p];
                const int n = (nt0 + t) * kTileN + (l & 15);
                int sum[HALVES];
#pragma unroll
                for (int hf = 0; hf < HALVES; ++hf) {
                    sum[hf] = 0;
                    for (int w = 0; w < ks; ++w) sum[hf] += red[(w * TT + hf * NT) * 256 + q];
                }
                if constexpr (HALVES == 2) {
                    const float x = sx[slot / k];
                    const float g = ((float)sum[0] * x) * sw[e * N + n];
                    const float u = ((float)sum[HALVES - 1] * x) * sw[e * N + nh + n];
                    out[(size_t)p * nh + n] = g / (1.0f + expf(-g)) * u;
                } else {
                    const float w = weights[slot];
                    const float y = ((float)sum[0] * sx[p]) * sw[e * N + n];
                    out[(size_t)slot * N + n] = w != 0.0f ? w * y : 0.0f;
                }
            }
        }
        // the sums lie over the X slots: all of them are added up before the
        // next rows' tiles go there
        __syncthreads();
    }
}

// Y[t] = the sum of the token's slots in order (float32, rounded once).
template <int OUT>
__global__ __launch_bounds__(256) void moe_combine_kernel(const float* __restrict__ part,
                                                          const int* __restrict__ ids, int E,
                                                          int k, int H, void* __restrict__ Y) {
    const size_t t = blockIdx.y;
    const int n = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (n >= H) return;
    v4f sum = v4f{0, 0, 0, 0};
    for (int j = 0; j < k; ++j) {
        const int e = ids[t * k + j];
        if (e >= 0 && e < E) sum += *reinterpret_cast<const v4f*>(part + (t * k + j) * H + n);
    }
    if constexpr (OUT == 0) {
        *reinterpret_cast<v4f*>(reinterpret_cast<float*>(Y) + t * H + n) = sum;
    } else {
        unsigned short b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = sum[i];
            b[i] = OUT == 1 ? f32_to_f16_bits(f) : f32_to_bf16_bits(f);
        }
        *reinterpret_cast<uint2*>(reinterpret_cast<unsigned short*>(Y) + t * H + n) =
            uint2{b[0] | ((unsigned)b[1] << 16), b[2] | ((unsigned)b[3] << 16)};
    }
}

// ---------------------------------------------------------------------------
// Few slots: every workgroup finds its expert's slots among the ids and
// quantises their rows itself, into LDS (row stride K + 16 bytes), while the
// first weights are in flight.  That saves the launches that prepare the
// rows: one token takes two launches, a few tokens three.
// ---------------------------------------------------------------------------
constexpr int kMaskSlots = 64;  // slots that one wave's ballots can find

// The slots of lane-wise ids (lane = slot): one bit per expert's first slot.
struct FewSlots {
    int id;                // of slot `lane`, -1: none
    unsigned long long peers;  // slots of the same expert
    unsigned long long first;  // uniform: the experts' first slots
};
__device__ __forceinline__ FewSlots few_slots(const int* ids, int S, int E) {
    const int lane = threadIdx.x & 63;
    FewSlots f;
    f.id = lane < S ? ids[lane] : -1;
    if (f.id >= E) f.id = -1;
    f.peers = same_expert_lanes(f.id, f.id >= 0, expert_bits(E));
    f.first = __ballot(f.id >= 0 && __builtin_ctzll(f.peers) == lane);
    return f;
}
__device__ __forceinline__ unsigned long long readlane64(unsigned long long v, int l) {
    return (unsigned long long)(unsigned)__builtin_amdgcn_readlane((int)(v >> 32), l) << 32 |
           (unsigned)__builtin_amdgcn_readlane((int)v, l);
}
// Position of the n-th set bit of a mask that has more than n.
__device__ __forceinline__ int nth_bit(unsigned long long m, int n) {
    for (int i = 0; i < n; ++i) m &= m - 1;
    return __builtin_ctzll(m);
}

// INT8 of a row by `waves` waves of which this is the w-th, into LDS; two
// passes over the row, the second from cache.  `part` holds one value per
// wave of the workgroup; every wave of the workgroup calls this (it holds a
// barrier), with on = false for those without a row.
template <int IN>
__device__ __forceinline__ float quant_row_lds(bool on, const void* row, int K, int w, int waves,
                                               int8_t* out, unsigned* part) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    unsigned m = 0;
    if (on)
#pragma unroll 2
        for (int i = w * 64 + lane; i < K / 8; i += waves * 64) {
            const Row8<IN> r = load_row8<IN>(row, i);
#pragma unroll
            for (int j = 0; j < 8; ++j) m = MaxU32{}(m, abs_bits(r.v[j]));
        }
    m = wave_reduce(m, MaxU32{});
    if (lane == 0) part[wave] = m;
    __syncthreads();
    if (!on) return 0.0f;
    for (int i = 0; i < waves; ++i) m = MaxU32{}(m, part[wave - w + i]);
    const float s = row_scale_bits(m), inv = __fdiv_rn(1.0f, s);
#pragma unroll 2
    for (int i = w * 64 + lane; i < K / 8; i += waves * 64) {
        const Row8<IN> r = load_row8<IN>(row, i);
        reinterpret_cast<uint2*>(out)[i] =
            uint2{quant4_fast(r.v[0], r.v[1], r.v[2], r.v[3], s, inv),
                  quant4_fast(r.v[4], r.v[5], r.v[6], r.v[7], s, inv)};
    }
    return s;
}

// One product of one expert (the blockIdx.y-th of the chosen ones) and 32
// channels of each half, the rows quantised by the workgroup itself:
// HALVES = 2: gate and up of the slots' tokens (rows of X), into h[slot][N / 2];
// HALVES = 1: down of the slots (rows of h), times the slot's weight, into
// part[slot][N].  `cap` rows at a time (more slots of an expert repeat its
// stream).
template <int HALVES, int IN, int GROUP>
__global__ __launch_bounds__(256, 4) void moe_few_kernel(
    const void* __restrict__ X, const int* __restrict__ ids, const float* __restrict__ weights,
    const uint8_t* __restrict__ wq, const uint8_t* __restrict__ s_u8,
    const uint8_t* __restrict__ a_u8, const float* __restrict__ sw, float* __restrict__ out, int S,
    int E, int k, int N, int K, int cap) {
    constexpr int NT = kMoeTiles, TT = HALVES * NT, D = HALVES == 2 ? 2 : 4, WAVES = 4;
    extern __shared__ __attribute__((aligned(16))) uint8_t few_lds[];
    uint8_t* const lds = few_lds;
    __shared__ float scales[16];
    __shared__ unsigned part[WAVES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, G = lane >> 4;
    const FewSlots f = few_slots(ids, S, E);
    if ((int)blockIdx.y >= __builtin_popcountll(f.first)) return;
    const int first = nth_bit(f.first, blockIdx.y);
    const int e = __builtin_amdgcn_readlane(f.id, first);
    unsigned long long mine = readlane64(f.peers, first);  // its slots

    const int nh = N / HALVES;  // channels of one half
    const int KT = K / kTileK, groups = K / GROUP, nt0 = channel_group(blockIdx.x, gridDim.x) * NT;
    const int nk = wave < KT ? (KT - wave + WAVES - 1) / WAVES : 0;
    const __amdgpu_buffer_rsrc_t w_rsrc =
        buf_rsrc(wq + (size_t)e * ((size_t)N * K / 2), (unsigned)((size_t)N * K / 2));
    const unsigned pbytes = (unsigned)((size_t)N * groups);
    const __amdgpu_buffer_rsrc_t s_rsrc = buf_rsrc(s_u8 + (size_t)e * pbytes, pbytes);
    const __amdgpu_buffer_rsrc_t a_rsrc = buf_rsrc(a_u8 + (size_t)e * pbytes, pbytes);
    const unsigned pvoff = 4u * (unsigned)r + (GROUP == 64 ? 64u * (unsigned)(G >> 1) : 0u);
    auto tile_of = [&](int t) { return t < NT ? nt0 + t : nh / kTileN + nt0 + t - NT; };
    struct Stage {
        v4i w[TT];
        unsigned s[HALVES], a[HALVES];
    };
    auto issue = [&](int i, Stage& st) {
        const int kt = wave + WAVES * i;
#pragma unroll
        for (int t = 0; t < TT; ++t)
            st.w[t] = __builtin_bit_cast(
                v4i, __builtin_amdgcn_raw_buffer_load_b128(
                         w_rsrc, (unsigned)lane * 16u,
                         (unsigned)(((size_t)tile_of(t) * KT + kt) * kTileBytes), kNonTemporal));
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf) {
            const unsigned po = 64u * ((unsigned)(tile_of(hf * NT) >> 2) * (unsigned)groups +
                                       (unsigned)(kt * (kTileK / GROUP)));
            st.s[hf] = buf_load4(s_rsrc, pvoff, po);
            st.a[hf] = buf_load4(a_rsrc, pvoff, po);
        }
    };
    while (mine) {  // the next slots, at most cap (<= 16)
        const int count = min(cap, __builtin_popcountll(mine));
        Stage st[D];
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (d < nk) issue(d, st[d]);

        // the rows, behind 16 bytes of zeros for the absent ones
        const int stride = K + 16;
        int8_t* rows = reinterpret_cast<int8_t*>(lds) + 16;
        if (tid < 4) reinterpret_cast<int*>(lds)[tid] = 0;
        constexpr int EB = IN == 0 ? 4 : 2;
        for (int i = 0; i < count; ++i) {
            const int slot = nth_bit(mine, i), row = HALVES == 2 ? slot / k : slot;
            const float s =
                quant_row_lds<IN>(true, reinterpret_cast<const uint8_t*>(X) + (size_t)row * K * EB, K,
                                  wave, WAVES, rows + i * stride, part);
            if (tid == 0) scales[i] = s;
            __syncthreads();
        }
        const int8_t* xrow = r < count ? rows + r * stride + 32 * G : nullptr;

        v4i acc[TT];
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[t] = v4i{0, 0, 0, 0};
        auto consume = [&](int i, const Stage& S_) {
            const int8_t* x = xrow ? xrow + (wave + WAVES * i) * kTileK : reinterpret_cast<int8_t*>(lds);
            const v4i x0 = *reinterpret_cast<const v4i*>(x);
            const v4i x1 = *reinterpret_cast<const v4i*>(xrow ? x + 16 : x);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int b = (nt0 & 3) + t % NT;
                const u16x2 s2 = scale_pair(S_.s[t / NT], b), a4 = offset_quad(S_.a[t / NT], b);
                unsigned q[8];
                lqq_dequant8((unsigned)S_.w[t].x, s2, a4, q[0], q[1]);
                lqq_dequant8((unsigned)S_.w[t].y, s2, a4, q[2], q[3]);
                lqq_dequant8((unsigned)S_.w[t].z, s2, a4, q[4], q[5]);
                lqq_dequant8((unsigned)S_.w[t].w, s2, a4, q[6], q[7]);
                acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                    x0, v4i{(int)q[0], (int)q[1], (int)q[2], (int)q[3]}, acc[t], 0, 0, 0);
                acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(
                    x1, v4i{(int)q[4], (int)q[5], (int)q[6], (int)q[7]}, acc[t], 0, 0, 0);
            }
        };
        int i = 0;
        for (; i + 2 * D <= nk; i += D) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                consume(i + d, st[d]);
                issue(i + d + D, st[d]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (i + d < nk) {
                consume(i + d, st[d]);
                if (i + d + D < nk) issue(i + d + D, st[d]);
            }
        }
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (i + D + d < nk) consume(i + D + d, st[d]);

        __syncthreads();  // all waves have read the rows
        int* red = reinterpret_cast<int*>(lds);
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int v = 0; v < 4; ++v) red[((wave * TT + t) * 4 + v) * 64 + lane] = acc[t][v];
        __syncthreads();
        for (int q = tid; q < NT * 256; q += 256) {
            const int t = q >> 8, l = q & 63, row = 4 * (l >> 4) + ((q >> 6) & 3);
            if (row >= count) continue;
            const int n = (nt0 + t) * kTileN + (l & 15), slot = nth_bit(mine, row);
            int sum[HALVES];
#pragma unroll
            for (int hf = 0; hf < HALVES; ++hf) {
                sum[hf] = 0;
                for (int w = 0; w < WAVES; ++w) sum[hf] += red[(w * TT + hf * NT) * 256 + q];
            }
            const float x = scales[row];
            const float y = ((float)sum[0] * x) * sw[(size_t)e * N + n];
            if constexpr (HALVES == 2) {
                const float u = ((float)sum[HALVES - 1] * x) * sw[(size_t)e * N + nh + n];
                out[(size_t)slot * nh + n] = y / (1.0f + expf(-y)) * u;
            } else {
                const float w = weights[slot];
                out[(size_t)slot * N + n] = w != 0.0f ? w * y : 0.0f;
            }
        }
        for (int i = 0; i < count; ++i) mine &= mine - 1;
        __syncthreads();  // the sums have been read
    }
}

// One token: the down products of its k slots for 16 channels and their
// weighted sum.  The 16 waves stream the chosen experts' tiles one after the
// other (a wave's K-tiles of all experts are one sequence, so the pipeline
// does not drain between them).  P (a power of two, at least k) rows are
// quantised at once.
template <int OUT, int GROUP>
__global__ __launch_bounds__(1024) void moe_few_down_kernel(
    const float* __restrict__ h, const int* __restrict__ ids, const float* __restrict__ weights,
    const uint8_t* __restrict__ wq, const uint8_t* __restrict__ s_u8,
    const uint8_t* __restrict__ a_u8, const float* __restrict__ sw, void* __restrict__ Y, int E,
    int S, int H, int K, int P) {
    constexpr int D = 4, WAVES = 16;
    extern __shared__ __attribute__((aligned(16))) uint8_t few_lds[];
    uint8_t* const lds = few_lds;
    __shared__ float scales[kMaxTopK];
    __shared__ unsigned part[WAVES];
    __shared__ float ys[kMaxTopK * 16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, G = lane >> 4;
    const FewSlots f = few_slots(ids, S, E);
    const int KT = K / kTileK, groups = K / GROUP, nt = channel_group(blockIdx.x, gridDim.x);
    const int nk = wave < KT ? (KT - wave + WAVES - 1) / WAVES : 0;
    const int total = nk * __builtin_popcountll(f.first);
    const size_t wbytes = (size_t)H * K / 2, pbytes = (size_t)H * groups;
    const unsigned pvoff = 4u * (unsigned)r + (GROUP == 64 ? 64u * (unsigned)(G >> 1) : 0u);
    struct Stage {
        v4i w;
        unsigned s, a;
    };
    // the sequence's next K-tile to load: of expert `in_e`
    unsigned in_first = (unsigned)f.first;  // k <= 16 slots
    int in_i = 0, in_e = in_first ? __builtin_amdgcn_readlane(f.id, __builtin_ctz(in_first)) : 0;
    auto issue = [&](Stage& st) {
        const int kt = wave + WAVES * in_i;
        const __amdgpu_buffer_rsrc_t w_rsrc = buf_rsrc(wq + in_e * wbytes, (unsigned)wbytes);
        const __amdgpu_buffer_rsrc_t s_rsrc = buf_rsrc(s_u8 + in_e * pbytes, (unsigned)pbytes);
        const __amdgpu_buffer_rsrc_t a_rsrc = buf_rsrc(a_u8 + in_e * pbytes, (unsigned)pbytes);
        st.w = __builtin_bit_cast(
            v4i, __builtin_amdgcn_raw_buffer_load_b128(
                     w_rsrc, (unsigned)lane * 16u,
                     (unsigned)(((size_t)nt * KT + kt) * kTileBytes), kNonTemporal));
        const unsigned po = 64u * ((unsigned)(nt >> 2) * (unsigned)groups +
                                   (unsigned)(kt * (kTileK / GROUP)));
        st.s = buf_load4(s_rsrc, pvoff, po);
        st.a = buf_load4(a_rsrc, pvoff, po);
        if (++in_i == nk) {
            in_i = 0;
            in_first &= in_first - 1;
            if (in_first) in_e = __builtin_amdgcn_readlane(f.id, __builtin_ctz(in_first));
        }
    };
    Stage st[D];
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (d < total) issue(st[d]);

    // h rows in LDS: 16 bytes of zeros, then row s at s * stride
    const int stride = K + 16;
    int8_t* rows = reinterpret_cast<int8_t*>(lds) + 16;
    if (tid < 4) reinterpret_cast<int*>(lds)[tid] = 0;
    {
        const int per = WAVES / P, s = wave / per;  // P <= 16
        const bool on = s < S && __builtin_amdgcn_readlane(f.id, s & 15) >= 0;
        const float sc = quant_row_lds<0>(on, h + (size_t)s * K, K, wave % per, per,
                                          rows + (size_t)s * stride, part);
        if (on && wave % per == 0 && lane == 0) scales[s] = sc;
    }
    int* red = reinterpret_cast<int*>(lds + 16 + (size_t)S * stride) + wave * S * 16;
    for (int q = lane; q < S * 16; q += 64) red[q] = 0;
    __syncthreads();

    // the expert being multiplied: its slots and this lane's row of them
    unsigned out_first = (unsigned)f.first, mine = 0;
    int out_i = 0;
    const int8_t* xrow = nullptr;
    auto enter = [&]() {
        mine = (unsigned)__builtin_amdgcn_readlane((int)f.peers, __builtin_ctz(out_first));
        const bool has = r < __builtin_popcount(mine);
        unsigned m = mine;
        for (int q = 0; q < r && has; ++q) m &= m - 1;
        xrow = has ? rows + (size_t)__builtin_ctz(m) * stride + 32 * G : nullptr;
    };
    v4i acc = v4i{0, 0, 0, 0};
    auto consume = [&](const Stage& S_) {
        if (out_i == 0) enter();
        const int8_t* x =
            xrow ? xrow + (wave + WAVES * out_i) * kTileK : reinterpret_cast<int8_t*>(lds);
        const v4i x0 = *reinterpret_cast<const v4i*>(x);
        const v4i x1 = *reinterpret_cast<const v4i*>(xrow ? x + 16 : x);
        const u16x2 s2 = scale_pair(S_.s, nt & 3), a4 = offset_quad(S_.a, nt & 3);
        unsigned q[8];
        lqq_dequant8((unsigned)S_.w.x, s2, a4, q[0], q[1]);
        lqq_dequant8((unsigned)S_.w.y, s2, a4, q[2], q[3]);
        lqq_dequant8((unsigned)S_.w.z, s2, a4, q[4], q[5]);
        lqq_dequant8((unsigned)S_.w.w, s2, a4, q[6], q[7]);
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
            x0, v4i{(int)q[0], (int)q[1], (int)q[2], (int)q[3]}, acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
            x1, v4i{(int)q[4], (int)q[5], (int)q[6], (int)q[7]}, acc, 0, 0, 0);
        if (++out_i == nk) {  // the expert's last K-tile of this wave
            out_i = 0;
            out_first &= out_first - 1;
            unsigned m = mine;
            for (int row = 0; m; ++row, m &= m - 1)  // uniform: its slots in order
                if (G == row >> 2) {
                    const int v = row & 3;
                    red[__builtin_ctz(m) * 16 + r] =
                        v == 0 ? acc[0] : v == 1 ? acc[1] : v == 2 ? acc[2] : acc[3];
                }
            acc = v4i{0, 0, 0, 0};
        }
    };
    int i = 0;
    for (; i + 2 * D <= total; i += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            consume(st[d]);
            issue(st[d]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int d = 0; d < D; ++d) {
        if (i + d < total) {
            consume(st[d]);
            if (i + d + D < total) issue(st[d]);
        }
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (i + D + d < total) consume(st[d]);
    __syncthreads();
    if (tid < S * 16) {
        const int s = tid >> 4, n = nt * kTileN + (tid & 15);
        const int* all = reinterpret_cast<const int*>(lds + 16 + (size_t)S * stride);
        int sum = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) sum += all[w * S * 16 + tid];
        const int e = ids[s];
        float y = 0.0f;
        if (e >= 0 && e < E) {
            const float w = weights[s];
            y = ((float)sum * scales[s]) * sw[(size_t)e * H + n];
            y = w != 0.0f ? w * y : 0.0f;
        }
        ys[tid] = y;
    }
    __syncthreads();
    if (tid < 16) {
        const int n = nt * kTileN + tid;
        float y = 0.0f;
        for (int j = 0; j < S; ++j) y += ys[j * 16 + tid];
        if constexpr (OUT == 0)
            reinterpret_cast<float*>(Y)[n] = y;
        else
            reinterpret_cast<unsigned short*>(Y)[n] =
                OUT == 1 ? f32_to_f16_bits(y) : f32_to_bf16_bits(y);
    }
}

size_t moe_workspace(int T, int k, int H, int F) { return MoeLayout(T, k, H, F).bytes; }

namespace {

// Rows that few experts exceed: the slots per expert a batch has on average
// and three of their standard deviations, or a row per token.
float most_rows(int T, int S, int E) {
    const float avg = (float)S / (float)E;
    return fminf(avg + 3.0f * sqrtf(avg), (float)T);
}

// The kernels that quantise their own rows run while the rows leave room for
// four workgroups per CU (at 66 KiB, two per CU, 32 tokens over 16 experts of
// 4096 x 2048 took 77 us against 54 with prepared rows).  Otherwise, in us,
// prepared rows / rows of their own / one token in two launches:
//   8 experts 14336 x 4096, top 2:   1 token 48.3 / 46.2 / 42.3, 2: 76.9 / 73.0
//   64 experts 1408 x 2048, top 6:   1 token 24.8 / 18.5 / 18.3, 2: 26.7 / 22.0,
//                                    8: 44.1 / 42.2
//   16 experts 4096 x 2048, top 2:   1 token 23.4 / 17.5 / 16.2, 4: 35.6 / 30.0
// (the two-launch form lost to three from two tokens on: 22.1 against 21.1).
constexpr size_t kFewLds = 40 * 1024;

// Row blocks of 16 that share a decoded weight.  us with one / two / four
// blocks (means of two routings):
//   24 tokens, two of 8 experts 4096 x 2048 (6 slots per expert): 36.7 / 38.5 / 47
//   32 tokens, two of 8 experts 14336 x 4096 (8):                 140 / 142 / 186
//   48 tokens, two of 8 experts 4096 x 2048 (12):                 46.4 / 42.4 / 50.7
//   131 tokens, two of 16 experts 6400 x 4096 (16):               186 / 148 / 187
//   200 tokens, two of 8 experts 4096 x 2048 (50):                87.7 / 69.8 / 76.7
//   250 tokens, two of 8 experts 6400 x 4096 (62):                275 / 183 / 172
int row_blocks(int T, int S, int E) {
    return most_rows(T, S, E) <= 18.0f ? 1 : (float)S <= 56.0f * (float)E ? 2 : 4;
}

// Workgroups that share an expert's rows where they exceed the blocks: routing
// is uneven (131 tokens, two of 16 experts, up to 50 of 262 slots on one: 170
// us with one, 155 with these), and one that finds no rows of its own leaves
// at once.  They come last in the grid: interleaved with the others, two or
// four of them left half or most of the CUs idle (209 and 361 us), since
// consecutive workgroups are dealt to the shader engines in turn.
int row_sharers(int T, int rb) {
    const int all = (T + 16 * rb - 1) / (16 * rb);
    return all < 4 ? all : 4;
}

// Waves splitting K: four, eight for
// the down product of wide experts (14336 x 4096, one token: the layer in
// 47.5 us against 50.5).
template <int HALVES, int RB, int D>
void launch_product(const int8_t* xq, const float* sx, const MoeWeights& w, const float* weights,
                    const MoeHead* head, const int* slots, float* out, int N, int K, int k,
                    int rows_in, int experts, int group, int sharers, hipStream_t st) {
    constexpr int NT = kMoeTiles;
    const int ks = HALVES == 1 && RB == 1 && K >= 64 * kTileK ? 8 : 4;
    const dim3 grid(N / HALVES / (kTileN * NT), experts, sharers), block(64 * ks);
    // X slots, then the sums of one row block
    const size_t xbytes = (size_t)ks * 2048 * RB;
    const size_t rbytes = (size_t)ks * HALVES * NT * 256 * sizeof(int);
    const size_t lds = xbytes > rbytes ? xbytes : rbytes;
    if (group == 64)
        hipLaunchKernelGGL((moe_product_kernel<HALVES, RB, D, 64>), grid, block, lds, st, xq,
                           sx, w.wq, w.s_u8, w.a_u8, w.sw, weights, head, slots, out, N, K, k,
                           rows_in);
    else
        hipLaunchKernelGGL((moe_product_kernel<HALVES, RB, D, 128>), grid, block, lds, st, xq,
                           sx, w.wq, w.s_u8, w.a_u8, w.sw, weights, head, slots, out, N, K, k,
                           rows_in);
}

// LDS of the kernels that quantise their own rows (`rows` of K elements).
size_t few_rows_lds(int rows, int K) { return 16 + (size_t)rows * (K + 16); }

template <int HALVES, int IN, int GROUP>
void launch_few_type(const void* X, const int* ids, const float* weights, const MoeWeights& w,
                     float* out, int S, int E, int k, int N, int K, int cap, hipStream_t st) {
    const dim3 grid(N / HALVES / (kTileN * kMoeTiles), E < S ? E : S);
    const size_t red = (size_t)4 * HALVES * kMoeTiles * 256 * sizeof(int);  // the sums, over the rows
    const size_t lds = few_rows_lds(cap, K);
    hipLaunchKernelGGL((moe_few_kernel<HALVES, IN, GROUP>), grid, dim3(256), lds > red ? lds : red,
                       st, X, ids, weights, w.wq, w.s_u8, w.a_u8, w.sw, out, S, E, k, N, K, cap);
}

template <int GROUP>
void launch_few_up(const void* X, int in_type, const int* ids, const MoeWeights& w, float* h,
                   int S, int E, int k, int F, int H, int cap, hipStream_t st) {
    if (in_type == 1)
        launch_few_type<2, 1, GROUP>(X, ids, nullptr, w, h, S, E, k, 2 * F, H, cap, st);
    else if (in_type == 2)
        launch_few_type<2, 2, GROUP>(X, ids, nullptr, w, h, S, E, k, 2 * F, H, cap, st);
    else
        launch_few_type<2, 0, GROUP>(X, ids, nullptr, w, h, S, E, k, 2 * F, H, cap, st);
}

size_t few_down_lds(int k, int F) {
    return few_rows_lds(k, F) + (size_t)16 * k * 16 * sizeof(int);
}

template <int GROUP>
void launch_few_down(const float* h, const int* ids, const float* weights, int E, int k,
                     const MoeWeights& w, void* Y, int out_type, int H, int F, hipStream_t st) {
    int P = 1;
    while (P < k) P *= 2;
#define FEW_DOWN(O)                                                                            \
    hipLaunchKernelGGL((moe_few_down_kernel<O, GROUP>), dim3(H / kTileN), dim3(1024),          \
                       few_down_lds(k, F), st, h, ids, weights, w.wq, w.s_u8, w.a_u8, w.sw, Y, \
                       E, k, H, F, P)
    if (out_type == 1) FEW_DOWN(1);
    else if (out_type == 2) FEW_DOWN(2);
    else FEW_DOWN(0);
#undef FEW_DOWN
}

void launch_combine(const float* part, const int* ids, int T, int E, int k, int H, void* Y,
                    int out_type, hipStream_t st) {
    const dim3 grid((H / 4 + 255) / 256, T);
    if (out_type == 1)
        hipLaunchKernelGGL(moe_combine_kernel<1>, grid, dim3(256), 0, st, part, ids, E, k, H, Y);
    else if (out_type == 2)
        hipLaunchKernelGGL(moe_combine_kernel<2>, grid, dim3(256), 0, st, part, ids, E, k, H, Y);
    else
        hipLaunchKernelGGL(moe_combine_kernel<0>, grid, dim3(256), 0, st, part, ids, E, k, H, Y);
}

}  // namespace

hipError_t launch_moe(const void* X, int in_type, const int* ids, const float* weights, int T,
                      int E, int k, const MoeWeights& w13, const MoeWeights& w2, void* Y,
                      int out_type, int H, int F, int group, void* workspace, hipStream_t st) {
    const MoeLayout lay(T, k, H, F);
    uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
    MoeHead* head = reinterpret_cast<MoeHead*>(ws);
    int* slots = reinterpret_cast<int*>(ws + lay.slots);
    int8_t* xq = reinterpret_cast<int8_t*>(ws + lay.xq);
    float* sx = reinterpret_cast<float*>(ws + lay.sx);
    float* h = reinterpret_cast<float*>(ws + lay.h);
    int8_t* hq = reinterpret_cast<int8_t*>(ws + lay.hq);
    float* sh = reinterpret_cast<float*>(ws + lay.sh);
    float* part = reinterpret_cast<float*>(ws + lay.part);
    const int S = T * k, experts = E < S ? E : S;
    // rows of an expert that one stream has to serve, a power of two; the
    // kernels that quantise their own rows take those and their elements
    int cap = 1;
    while (cap < 16 && (float)cap < most_rows(T, S, E)) cap *= 2;
    const bool up = S <= kMaskSlots && few_rows_lds(cap, H) <= kFewLds;
    const bool join = T == 1 && few_down_lds(k, F) <= 144 * 1024;
    const bool down = S <= kMaskSlots && few_rows_lds(cap, F) <= kFewLds;
    if (up && (join || down)) {
        if (group == 64) launch_few_up<64>(X, in_type, ids, w13, h, S, E, k, F, H, cap, st);
        else launch_few_up<128>(X, in_type, ids, w13, h, S, E, k, F, H, cap, st);
        if (join) {
            if (group == 64) launch_few_down<64>(h, ids, weights, E, k, w2, Y, out_type, H, F, st);
            else launch_few_down<128>(h, ids, weights, E, k, w2, Y, out_type, H, F, st);
            return hipGetLastError();
        }
        if (group == 64)
            launch_few_type<1, 0, 64>(h, ids, weights, w2, part, S, E, k, H, F, cap, st);
        else
            launch_few_type<1, 0, 128>(h, ids, weights, w2, part, S, E, k, H, F, cap, st);
        launch_combine(part, ids, T, E, k, H, Y, out_type, st);
        return hipGetLastError();
    }
    const size_t lds = ((size_t)kGroupWaves * E + 2 * E + 1) * sizeof(int);
#define PREPARE(I)                                                                              \
    hipLaunchKernelGGL((moe_prepare_kernel<I>), dim3(T + 1), dim3(1024), lds, st, X, ids, T, E, \
                       k, H, head, slots, xq, sx)
    if (in_type == 1) PREPARE(1);
    else if (in_type == 2) PREPARE(2);
    else PREPARE(0);
#undef PREPARE
    const int rb = row_blocks(T, S, E), sharers = row_sharers(T, rb);
    if (rb == 1)
        launch_product<2, 1, 2>(xq, sx, w13, weights, head, slots, h, 2 * F, H, k, T, experts, group,
                                sharers, st);
    else if (rb == 2)
        launch_product<2, 2, 1>(xq, sx, w13, weights, head, slots, h, 2 * F, H, k, T, experts, group,
                                sharers, st);
    else
        launch_product<2, 4, 1>(xq, sx, w13, weights, head, slots, h, 2 * F, H, k, T, experts, group,
                                sharers, st);
    hipLaunchKernelGGL(moe_quant_kernel, dim3(S), dim3(1024), 0, st, h, F, head, hq, sh);
    if (rb == 1)
        launch_product<1, 1, 2>(hq, sh, w2, weights, head, slots, part, H, F, k, S, experts, group,
                                sharers, st);
    else if (rb == 2)
        launch_product<1, 2, 2>(hq, sh, w2, weights, head, slots, part, H, F, k, S, experts, group,
                                sharers, st);
    else
        launch_product<1, 4, 2>(hq, sh, w2, weights, head, slots, part, H, F, k, S, experts, group,
                                sharers, st);
    launch_combine(part, ids, T, E, k, H, Y, out_type, st);
    return hipGetLastError();
}

}  // namespace w4a8
