// Reductions over a wave of 64 lanes, and the grouping of slots by expert.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a8 {

// Butterfly over the 16 lanes of a row: each step combines a lane with the
// one a data-parallel-primitive permutation names (quad swaps, then halves
// and rows mirrored).  Both sides of a pair form the same sum of two, so
// every lane ends with the same bits.
template <typename F>
__device__ __forceinline__ unsigned row16_reduce(unsigned v, F f) {
    v = f(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));   // quad 1 0 3 2
    v = f(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));   // quad 2 3 0 1
    v = f(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));  // half row mirror
    v = f(v, (unsigned)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));  // row mirror
    return v;
}
template <typename F>
__device__ __forceinline__ unsigned wave_reduce(unsigned v, F f) {
    v = row16_reduce(v, f);
    const unsigned a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const unsigned c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    return f(f(a, b), f(c, d));
}

struct MaxU32 {
    __device__ unsigned operator()(unsigned a, unsigned b) const { return a > b ? a : b; }
};
struct SumF32 {
    __device__ unsigned operator()(unsigned a, unsigned b) const {
        return __builtin_bit_cast(unsigned,
                                  __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
    }
};
__device__ __forceinline__ float row16_sum(float v) {
    return __builtin_bit_cast(float, row16_reduce(__builtin_bit_cast(unsigned, v), SumF32{}));
}
__device__ __forceinline__ float wave_sum(float v) {
    return __builtin_bit_cast(float, wave_reduce(__builtin_bit_cast(unsigned, v), SumF32{}));
}

constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 16;
constexpr int kGroupWaves = 16;  // waves of the workgroups that group slots

// Slots (token, choice) are grouped by a stable counting sort: wave w of the
// workgroup takes the w-th run of consecutive slots, 64 at a time; the lanes
// of a chunk that hold the same expert find each other by one ballot per bit
// of its number, so a slot's place is (slots of smaller experts) + (its
// expert's slots in earlier runs) + (in earlier chunks of the run) + (in
// lower lanes), without an atomic, and the order is the slots' own.
__device__ __forceinline__ uint64_t same_expert_lanes(int id, bool valid, int bits) {
    uint64_t peers = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
        const bool one = (id >> b) & 1;
        const uint64_t m = __ballot(one);
        peers &= one ? m : ~m;
    }
    return peers;
}

__device__ __forceinline__ int expert_bits(int E) { return E > 1 ? 32 - __builtin_clz(E - 1) : 0; }

// Slots per wave: a whole number of chunks.
__device__ __forceinline__ int group_run(int S) {
    return (S + 64 * kGroupWaves - 1) / (64 * kGroupWaves) * 64;
}

// hist[wave][E] (zeroed by the caller, published by a barrier): this wave's
// slots of every expert.
// get(s): the expert of slot s < S; values outside [0, E) are no expert.
template <typename Get>
__device__ __forceinline__ void group_count(int* hist, int S, int E, Get get) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int run = group_run(S), bits = expert_bits(E);
    int* h = hist + wave * E;
    const int end = min(S, (wave + 1) * run);
    for (int s0 = wave * run; s0 < end; s0 += 64) {
        const int s = s0 + lane;
        const int id = s < end ? get(s) : -1;
        const bool valid = id >= 0 && id < E;
        const uint64_t peers = same_expert_lanes(id, valid, bits);
        if (valid && __builtin_ctzll(peers) == lane) h[id] += __builtin_popcountll(peers);
        __builtin_amdgcn_wave_barrier();
    }
}

// After hist[wave][e] has become the place of this wave's first slot of e:
// put(place, slot) for every slot with an expert.
template <typename Get, typename Put>
__device__ __forceinline__ void group_place(int* hist, int S, int E, Get get, Put put) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int run = group_run(S), bits = expert_bits(E);
    int* h = hist + wave * E;
    const int end = min(S, (wave + 1) * run);
    for (int s0 = wave * run; s0 < end; s0 += 64) {
        const int s = s0 + lane;
        const int id = s < end ? get(s) : -1;
        const bool valid = id >= 0 && id < E;
        const uint64_t peers = same_expert_lanes(id, valid, bits);
        const int rank = __builtin_popcountll(peers & ((1ull << lane) - 1));
        int base = 0;
        if (valid) base = h[id];
        __builtin_amdgcn_wave_barrier();
        if (valid && rank == 0) h[id] = base + __builtin_popcountll(peers);
        __builtin_amdgcn_wave_barrier();
        if (valid) put(base + rank, s);
    }
}

// Exclusive prefix sum of cnt[0 .. E) (E <= 512, LDS) into start[0 .. E], by
// the first wave of the workgroup; the caller's barriers stand around it.
__device__ __forceinline__ void expert_scan(const int* cnt, int* start, int E) {
    if (threadIdx.x >= 64) return;
    const int lane = threadIdx.x;
    constexpr int PER = kMaxExperts / 64;
    int c[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane * PER + i;
        c[i] = e < E ? cnt[e] : 0;
        sum += c[i];
    }
    int pre = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(pre, off, 64);
        if (lane >= off) pre += v;
    }
    const int total = __shfl(pre, 63, 64);
    pre -= sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane * PER + i;
        if (e < E) start[e] = pre;
        pre += c[i];
    }
    if (lane == 0) start[E] = total;
}

}  // namespace w4a8
