// rows.cuh -- rows of elements as packed pairs of floats, and sums over the lanes that
// hold a row: what the kernels that norm rows share.
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"

namespace diffattn {

// 16 bytes of elements, N of them, as N / 2 packed pairs of floats (two elements an
// instruction: at an SM's share of the HBM rate the arithmetic is half of the time).
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void unpack(uint4 v, uint64_t* x) {
        x[0] = f2_from_bits(v.x, v.y);
        x[1] = f2_from_bits(v.z, v.w);
    }
    __device__ static __forceinline__ uint4 pack(const uint64_t* x) {
        return make_uint4((uint32_t)x[0], (uint32_t)(x[0] >> 32), (uint32_t)x[1], (uint32_t)(x[1] >> 32));
    }
    __device__ static __forceinline__ float get(float v) { return v; }
    __device__ static __forceinline__ float put(float v) { return v; }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void unpack(uint4 v, uint64_t* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = f2_from_bits(w[i] << 16, w[i] & 0xffff0000u);
    }
    __device__ static __forceinline__ uint4 pack(const uint64_t* x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(f2_lo(x[i]), f2_hi(x[i]));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ static __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    __device__ static __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

// V floats as V / 2 packed pairs.
template <int V>
__device__ __forceinline__ void load_pairs(const float* p, uint64_t* x) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
        x[2 * i] = f2_from_bits(v.x, v.y);
        x[2 * i + 1] = f2_from_bits(v.z, v.w);
    }
}

// Sum of both halves of V packed pairs.
template <int V>
__device__ __forceinline__ float pair_sum(const uint64_t* x) {
    uint64_t s = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) s = f2_add(s, x[i]);
    return f2_lo(s) + f2_hi(s);
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

}  // namespace diffattn
