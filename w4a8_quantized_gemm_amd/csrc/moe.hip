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
// Every weight of a chosen expert is read once from HBM and nothing else is
// of its size, so the weight stream bounds the layer.
#include "act_common.h"
#include "launch.h"
#include "mfma_common.h"
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
// Scale of a row: max / 127, 1 for an all-zero row, and NaN for a row with
// an element that is not finite (all of the row's results are NaN then).
__device__ __forceinline__ float row_scale_bits(unsigned m) {
    if (m >= 0x7F800000u) return __builtin_nanf("");
    return scale_of(__builtin_bit_cast(float, m), 127.0f);
}

template <int IN>
__device__ __forceinline__ void quant_row(const void* row, int K, int8_t* out, float* scale) {
    unsigned m = 0;
    for (int i = threadIdx.x; i < K / 8; i += blockDim.x) {
        const Row8<IN> r = load_row8<IN>(row, i);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = MaxU32{}(m, abs_bits(r.v[j]));
    }
    const float s = row_scale_bits(block_max_bits(m));
    if (threadIdx.x == 0) *scale = s;
    uint2* o = reinterpret_cast<uint2*>(out);
    for (int i = threadIdx.x; i < K / 8; i += blockDim.x) {
        const Row8<IN> r = load_row8<IN>(row, i);
        unsigned b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = (unsigned)(quant_sym(r.v[j], s, 127.0f) & 0xFF);
        o[i] = uint2{b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24),
                     b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24)};
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

// One product of the layer for one expert and 16 NT channels of each half:
// HALVES = 2: the gate and up products of W13 (channel n and F + n), h = silu;
// HALVES = 1: the down product, scaled by the slot's weight, into part[slot].
// blockIdx.x: channel group, blockIdx.y: index into the active experts.  The
// `ks` waves take interleaved K-tiles and are summed in LDS (exact int32).
// Up to 16 RB rows share each decoded weight; more rows repeat the stream.
template <int HALVES, int NT, int RB, int D, int GROUP>
__global__ __launch_bounds__(256) void moe_product_kernel(
    const int8_t* __restrict__ Xq, const float* __restrict__ sx, const uint8_t* __restrict__ wq,
    const uint8_t* __restrict__ s_u8, const uint8_t* __restrict__ a_u8,
    const float* __restrict__ sw, const float* __restrict__ weights,
    const MoeHead* __restrict__ head, const int* __restrict__ slots, float* __restrict__ out,
    int N, int K, int k, int rows_in) {
    constexpr int TT = HALVES * NT;  // weight tiles of the workgroup
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
    const int nt0 = blockIdx.x * NT;
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

    struct Stage {
        v4i x0[RB], x1[RB], w[TT];
        unsigned s[HALVES], a[HALVES];
    };
    for (int r0 = 0; r0 < act.count; r0 += 16 * RB) {
        // row r of row block rb: its token (W13) or its own place (W2)
        unsigned xoff[RB];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            const int i = r0 + 16 * rb + r;
            unsigned row = 0xFFFFFFFFu;
            if (i < act.count) row = act.start + i;
            if (HALVES == 2 && i < act.count) row = (unsigned)slots[act.start + i] / (unsigned)k;
            xoff[rb] = i < act.count ? row * (unsigned)K + 32u * (unsigned)G : 0xFFFFFFE0u;
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
                // an absent row's offset lies past the buffer and reads 0
                const unsigned xo = xoff[rb] == 0xFFFFFFE0u ? xoff[rb] : xoff[rb] + kt * kTileK;
                st.x0[rb] = buf_load16(x_rsrc, xo, 0);
                st.x1[rb] = buf_load16(x_rsrc, xo + 16u, 0);
            }
        };
        v4i acc[RB][TT];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int t = 0; t < TT; ++t) acc[rb][t] = v4i{0, 0, 0, 0};
        auto consume = [&](const Stage& S) {
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int b = (NT == 4 ? t % NT : (nt0 & 3) + t % NT);
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
                        __builtin_amdgcn_mfma_i32_16x16x64_i8(S.x0[rb], B0, acc[rb][t], 0, 0, 0);
                    acc[rb][t] =
                        __builtin_amdgcn_mfma_i32_16x16x64_i8(S.x1[rb], B1, acc[rb][t], 0, 0, 0);
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

size_t moe_workspace(int T, int k, int H, int F) { return MoeLayout(T, k, H, F).bytes; }

namespace {

template <int HALVES, int NT, int RB, int D>
void launch_product(const int8_t* xq, const float* sx, const MoeWeights& w, const float* weights,
                    const MoeHead* head, const int* slots, float* out, int N, int K, int k,
                    int rows_in, int experts, int group, hipStream_t st) {
    const dim3 grid(N / HALVES / (kTileN * NT), experts), block(256);
    const size_t lds = (size_t)4 * HALVES * NT * 256 * sizeof(int);
    if (group == 64)
        hipLaunchKernelGGL((moe_product_kernel<HALVES, NT, RB, D, 64>), grid, block, lds, st, xq,
                           sx, w.wq, w.s_u8, w.a_u8, w.sw, weights, head, slots, out, N, K, k,
                           rows_in);
    else
        hipLaunchKernelGGL((moe_product_kernel<HALVES, NT, RB, D, 128>), grid, block, lds, st, xq,
                           sx, w.wq, w.s_u8, w.a_u8, w.sw, weights, head, slots, out, N, K, k,
                           rows_in);
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
    const size_t lds = ((size_t)kGroupWaves * E + 2 * E + 1) * sizeof(int);
#define PREPARE(I)                                                                              \
    hipLaunchKernelGGL((moe_prepare_kernel<I>), dim3(T + 1), dim3(1024), lds, st, X, ids, T, E, \
                       k, H, head, slots, xq, sx)
    if (in_type == 1) PREPARE(1);
    else if (in_type == 2) PREPARE(2);
    else PREPARE(0);
#undef PREPARE
    launch_product<2, 2, 1, 2>(xq, sx, w13, weights, head, slots, h, 2 * F, H, k, T, experts,
                               group, st);
    hipLaunchKernelGGL(moe_quant_kernel, dim3(S), dim3(1024), 0, st, h, F, head, hq, sh);
    launch_product<1, 2, 1, 2>(hq, sh, w2, weights, head, slots, part, H, F, k, S, experts, group,
                               st);
    const dim3 grid((H / 4 + 255) / 256, T);
    if (out_type == 1)
        hipLaunchKernelGGL(moe_combine_kernel<1>, grid, dim3(256), 0, st, part, ids, E, k, H, Y);
    else if (out_type == 2)
        hipLaunchKernelGGL(moe_combine_kernel<2>, grid, dim3(256), 0, st, part, ids, E, k, H, Y);
    else
        hipLaunchKernelGGL(moe_combine_kernel<0>, grid, dim3(256), 0, st, part, ids, E, k, H, Y);
    return hipGetLastError();
}

}  // namespace w4a8
