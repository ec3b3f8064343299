// Device helpers of the kernels that quantise rows: symmetric scales and
// codes, loads of float32 / fp16 / bf16 elements widened to float32, and the
// largest value of a workgroup.
#pragma once
#include "device_common.h"

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

}  // namespace w4a8
