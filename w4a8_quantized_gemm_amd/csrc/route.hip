// Top-k gating of a mixture-of-experts layer, and the grouping of the chosen
// (token, expert) slots by expert.
//
// Per token, with e_i = exp(x_i - max x) over the available experts (logit
// above -inf and not NaN):
//   choice j = the expert with the j-th largest logit (ties: lowest index),
//   weight j = e_j / sum_i e_i, or e_j / (sum of the chosen) if renormalised.
// The logits are mapped to unsigned integers of the same order (0 = not
// available), so a choice is an integer maximum over the wave and a ballot
// of the lanes that hold it; the first set bit is the lowest index.
//
// The work is a few integer steps per logit and a chain of k wave maxima per
// token: latency bounds a decode call (one launch of one workgroup, ids kept
// in LDS), the chain bounds a prefill call (two launches: choices and counts
// per block of tokens, then places).
#include "act_common.h"
#include "launch.h"
#include "wave_common.h"

namespace w4a8 {

namespace {

constexpr int kThreads = 64 * kGroupWaves;

// Order-preserving map of a logit to an unsigned integer; -inf and NaN give
// 0, and the two zeros are equal.
__device__ __forceinline__ unsigned logit_key(float x) {
    const unsigned u = __builtin_bit_cast(unsigned, x + 0.0f);
    const unsigned k = u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
    return (x > -__builtin_inff()) ? k : 0u;  // false for NaN
}
__device__ __forceinline__ float key_logit(unsigned k) {
    return __builtin_bit_cast(float, k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
// exp(x - top); an infinite top has only infinite equals, all of weight 1.
__device__ __forceinline__ float gate_exp(float x, float top) {
    return x == top ? 1.0f : expf(x - top);
}

template <int IN>
__device__ __forceinline__ float load_logit(const void* p, size_t i) {
    if constexpr (IN == 0) return reinterpret_cast<const float*>(p)[i];
    const unsigned h = reinterpret_cast<const unsigned short*>(p)[i];
    if constexpr (IN == 1) return (float)__builtin_bit_cast(_Float16, (unsigned short)h);
    return __builtin_bit_cast(float, h << 16);
}

// Choices of one lane: lane j of a token's lanes holds choice j.
struct Choice {
    int id;
    float w;
};

// Keys of one token per wave, up to 64 VPL experts: lane l holds experts
// 64 i + l.
template <int IN, int VPL>
__device__ __forceinline__ void load_keys(const void* logits, size_t t, size_t T, int E,
                                          unsigned (&key)[VPL]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int e = 64 * i + lane;
        key[i] = t < T && e < E ? logit_key(load_logit<IN>(logits, t * E + e)) : 0u;
    }
}

template <int VPL>
__device__ __forceinline__ Choice choose_wave(unsigned (&key)[VPL], int k, bool renorm) {
    const int lane = threadIdx.x & 63;
    unsigned all = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) all = MaxU32{}(all, key[i]);
    unsigned best = wave_reduce(all, MaxU32{});
    const float top = key_logit(best);
    float sum = 0.0f;
    if (!renorm) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            sum += key[i] ? gate_exp(key_logit(key[i]), top) : 0.0f;
        sum = wave_sum(sum);
    }
    Choice c{-1, 0.0f};
    unsigned mine = 0;  // key of the lane's choice
    for (int j = 0; j < k && best != 0; ++j) {
        int id = -1;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const uint64_t m = __ballot(key[i] == best);
            if (id < 0 && m) id = 64 * i + __builtin_ctzll(m);
        }
        if (lane == j) {
            c.id = id;
            mine = best;
        }
        all = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            if (64 * i + lane == id) key[i] = 0u;
            all = MaxU32{}(all, key[i]);
        }
        best = wave_reduce(all, MaxU32{});
    }
    c.w = mine ? gate_exp(key_logit(mine), top) : 0.0f;
    if (renorm) sum = wave_sum(c.w);
    c.w = c.id >= 0 ? __fdiv_rn(c.w, sum) : 0.0f;
    return c;
}

// Four tokens per wave, up to 16 experts: the 16 lanes of a row hold a
// token's experts.
__device__ __forceinline__ Choice choose_row(unsigned key, int k, bool renorm) {
    const int lane = threadIdx.x & 63, e = lane & 15, row = lane >> 4;
    unsigned best = row16_reduce(key, MaxU32{});
    const float top = key_logit(best);
    float sum = 0.0f;
    if (!renorm) sum = row16_sum(key ? gate_exp(key_logit(key), top) : 0.0f);
    Choice c{-1, 0.0f};
    unsigned mine = 0;  // key of the lane's choice
    for (int j = 0; j < k; ++j) {
        const unsigned m = (unsigned)(__ballot(key == best) >> (16 * row)) & 0xFFFFu;
        const int id = best ? __builtin_ctz(m) : -1;  // best is some lane's key, so m != 0
        if (e == j) {
            c.id = id;
            mine = best;
        }
        if (e == id) key = 0u;
        best = row16_reduce(key, MaxU32{});
    }
    c.w = mine ? gate_exp(key_logit(mine), top) : 0.0f;
    if (renorm) sum = row16_sum(c.w);
    c.w = c.id >= 0 ? __fdiv_rn(c.w, sum) : 0.0f;
    return c;
}

// Choices of tokens [lo, hi) by all waves of the workgroup; seen(slot, id)
// for each, slots counted from t0's.
template <int IN, int VPL, typename Seen>
__device__ __forceinline__ void choose_tokens(const void* logits, size_t lo, size_t hi, int E,
                                              int k, bool renorm, int* ids, float* weights,
                                              Seen seen) {
    constexpr int PW = VPL == 0 ? 4 : 1;  // tokens per wave
    constexpr int AHEAD = 4;              // steps whose logits are loaded together
    constexpr int KEYS = VPL == 0 ? 1 : VPL;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int j = VPL == 0 ? lane & 15 : lane, row = VPL == 0 ? lane >> 4 : 0;
    constexpr size_t STEP = PW * kGroupWaves;
    for (size_t t0 = lo + PW * wave; t0 < hi; t0 += AHEAD * STEP) {
        unsigned key[AHEAD][KEYS];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const size_t t = t0 + i * STEP + row;
            if constexpr (VPL == 0)
                key[i][0] = t < hi && j < E ? logit_key(load_logit<IN>(logits, t * E + j)) : 0u;
            else
                load_keys<IN>(logits, t, hi, E, key[i]);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (t0 + i * STEP >= hi) break;
            Choice c;
            if constexpr (VPL == 0) c = choose_row(key[i][0], k, renorm);
            else c = choose_wave(key[i], k, renorm);
            const size_t t = t0 + i * STEP + row;
            if (t < hi && j < k) {
                ids[t * k + j] = c.id;
                weights[t * k + j] = c.w;
                seen((int)(t - lo) * k + j, c.id);
            }
        }
    }
}

}  // namespace

// All of a small call in one workgroup: choices (ids kept in LDS), counts,
// places.
template <int IN, int VPL>
__global__ __launch_bounds__(kThreads) void route_small_kernel(
    const void* __restrict__ logits, int T, int E, int k, int renorm, int* __restrict__ ids,
    float* __restrict__ weights, int* __restrict__ offsets, int* __restrict__ rows) {
    extern __shared__ int lds[];
    const int S = T * k;
    int* hist = lds;                        // [waves][E]
    int* cnt = hist + kGroupWaves * E;      // [E]
    int* start = cnt + E;                   // [E + 1]
    int* sid = start + E + 1;               // [S]
    for (int i = threadIdx.x; i < kGroupWaves * E; i += kThreads) hist[i] = 0;
    choose_tokens<IN, VPL>(logits, 0, T, E, k, renorm != 0, ids, weights,
                           [&](int s, int id) { sid[s] = id; });
    __syncthreads();
    auto get = [&](int s) { return sid[s]; };
    group_count(hist, S, E, get);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) {
        int c = 0;
        for (int w = 0; w < kGroupWaves; ++w) c += hist[w * E + e];
        cnt[e] = c;
    }
    __syncthreads();
    expert_scan(cnt, start, E);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) {
        int p = start[e];
        offsets[e] = p;
        for (int w = 0; w < kGroupWaves; ++w) {
            const int c = hist[w * E + e];
            hist[w * E + e] = p;
            p += c;
        }
    }
    if (threadIdx.x == 0) offsets[E] = start[E];
    __syncthreads();
    group_place(hist, S, E, get, [&](int p, int s) { rows[p] = s; });
    for (int p = start[E] + threadIdx.x; p < S; p += kThreads) rows[p] = -1;
}

// Larger calls, first launch: choices of `tb` tokens per workgroup and how
// many of its slots each expert got (counts[block][E]).
template <int IN, int VPL>
__global__ __launch_bounds__(kThreads) void route_choose_kernel(
    const void* __restrict__ logits, int T, int E, int k, int renorm, int tb,
    int* __restrict__ ids, float* __restrict__ weights, int* __restrict__ counts) {
    extern __shared__ int lds[];
    for (int e = threadIdx.x; e < E; e += kThreads) lds[e] = 0;
    __syncthreads();
    const size_t lo = (size_t)blockIdx.x * tb;
    const size_t hi = min(lo + tb, (size_t)T);
    choose_tokens<IN, VPL>(logits, lo, hi, E, k, renorm != 0, ids, weights, [&](int, int id) {
        if (id >= 0) atomicAdd(&lds[id], 1);  // a count: no order
    });
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kThreads) counts[(size_t)blockIdx.x * E + e] = lds[e];
}

// Second launch: every workgroup adds up the counts (its own first slot of
// an expert lies behind those of the earlier blocks) and places its slots.
__global__ __launch_bounds__(kThreads) void route_place_kernel(
    const int* __restrict__ ids, const int* __restrict__ counts, int T, int E, int k, int tb,
    int* __restrict__ offsets, int* __restrict__ rows) {
    extern __shared__ int lds[];
    int* hist = lds;
    int* cnt = hist + kGroupWaves * E;
    int* start = cnt + E;
    const size_t lo = (size_t)blockIdx.x * tb;
    const int S = (int)(min(lo + tb, (size_t)T) - lo) * k;
    const int* bid = ids + lo * k;
    for (int i = threadIdx.x; i < kGroupWaves * E; i += kThreads) hist[i] = 0;
    // totals, and the slots of earlier blocks: part-th of the blocks per group
    // of E threads, joined by integer adds in LDS
    int* before = start + E + 1;
    for (int e = threadIdx.x; e < E; e += kThreads) cnt[e] = before[e] = 0;
    __syncthreads();
    const int parts = kThreads / E, part = threadIdx.x / E, pe = threadIdx.x % E;
    if (part < parts) {
        int all = 0, mine = 0;
        for (int b = part; b < (int)gridDim.x; b += 8 * parts) {
            int c[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int bu = b + u * parts;
                c[u] = bu < (int)gridDim.x ? counts[(size_t)bu * E + pe] : 0;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                all += c[u];
                mine += b + u * parts < (int)blockIdx.x ? c[u] : 0;
            }
        }
        atomicAdd(&cnt[pe], all);
        atomicAdd(&before[pe], mine);
    }
    __syncthreads();
    expert_scan(cnt, start, E);
    auto get = [&](int s) { return bid[s]; };
    group_count(hist, S, E, get);
    __syncthreads();
    if ((int)threadIdx.x < E) {
        int p = start[threadIdx.x] + before[threadIdx.x];
        for (int w = 0; w < kGroupWaves; ++w) {
            const int c = hist[w * E + threadIdx.x];
            hist[w * E + threadIdx.x] = p;
            p += c;
        }
    }
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= E; e += kThreads) offsets[e] = start[e];
    __syncthreads();
    const int first = (int)(lo * k);
    group_place(hist, S, E, get, [&](int p, int s) { rows[p] = first + s; });
    const long long all = (long long)T * k;
    for (long long p = start[E] + (long long)blockIdx.x * kThreads + threadIdx.x; p < all;
         p += (long long)gridDim.x * kThreads)
        rows[p] = -1;
}

namespace {

template <int IN, int VPL>
hipError_t route_run(const void* logits, int T, int E, int k, int renorm, int* ids,
                     float* weights, int* offsets, int* rows, const RoutePlan& plan, int* counts,
                     hipStream_t st) {
    const size_t group_lds = ((size_t)kGroupWaves * E + 3 * E + 1) * sizeof(int);
    if (plan.blocks == 1) {
        hipLaunchKernelGGL((route_small_kernel<IN, VPL>), dim3(1), dim3(kThreads),
                           group_lds + (size_t)T * k * sizeof(int), st, logits, T, E, k, renorm,
                           ids, weights, offsets, rows);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((route_choose_kernel<IN, VPL>), dim3(plan.blocks), dim3(kThreads),
                       E * sizeof(int), st, logits, T, E, k, renorm, plan.tokens, ids, weights,
                       counts);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(route_place_kernel, dim3(plan.blocks), dim3(kThreads), group_lds, st, ids,
                       counts, T, E, k, plan.tokens, offsets, rows);
    return hipGetLastError();
}

template <int IN>
hipError_t route_type(const void* logits, int T, int E, int k, int renorm, int* ids,
                      float* weights, int* offsets, int* rows, const RoutePlan& plan, int* counts,
                      hipStream_t st) {
#define ROUTE(V) \
    return route_run<IN, V>(logits, T, E, k, renorm, ids, weights, offsets, rows, plan, counts, st)
    if (E <= 16) ROUTE(0);
    if (E <= 64) ROUTE(1);
    if (E <= 128) ROUTE(2);
    if (E <= 256) ROUTE(4);
    ROUTE(8);
#undef ROUTE
}

}  // namespace

// One workgroup while every wave makes one step (its 16 waves share a CU: at
// four steps each, 61 tokens of 128 experts took 16 us against 9 in two
// launches over many CUs); else blocks of at least 32 tokens (16 for small
// calls), at most 512 blocks.
RoutePlan plan_route(int T, int E, int k) {
    RoutePlan p;
    const int per_pass = kGroupWaves * (E <= 16 ? 4 : 1);
    if (T <= per_pass) {
        p.blocks = 1;
        p.tokens = T;
        p.workspace = 0;
        return p;
    }
    p.tokens = T <= 2048 ? 16 : 32 * (int)((T + 32LL * 512 - 1) / (32 * 512));
    p.blocks = (int)(((long long)T + p.tokens - 1) / p.tokens);
    p.workspace = (size_t)p.blocks * E * sizeof(int);
    return p;
}

hipError_t launch_route(const void* logits, int in_type, int T, int E, int k, int renorm,
                        int* ids, float* weights, int* offsets, int* rows, void* workspace,
                        hipStream_t st) {
    const RoutePlan plan = plan_route(T, E, k);
    int* counts = reinterpret_cast<int*>(workspace);
    if (in_type == 1)
        return route_type<1>(logits, T, E, k, renorm, ids, weights, offsets, rows, plan, counts, st);
    if (in_type == 2)
        return route_type<2>(logits, T, E, k, renorm, ids, weights, offsets, rows, plan, counts, st);
    return route_type<0>(logits, T, E, k, renorm, ids, weights, offsets, rows, plan, counts, st);
}

}  // namespace w4a8
