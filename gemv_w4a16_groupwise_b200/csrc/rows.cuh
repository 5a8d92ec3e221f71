// Rows of bf16 held in the registers of a thread block, and reductions over
// the block.
#pragma once

#include "common.cuh"

namespace w4 {

constexpr int kRowMaxC = 16384;   // 1024 threads x 2 vectors of 8

// Elements of one thread: V vectors of VEC consecutive columns, T vectors
// apart.  VEC = 8 needs C % 8 == 0 (16-byte aligned rows); VEC = 1 serves
// the other widths.
template <int T, int V, int VEC>
struct RowSpan {
    static constexpr int E = V * VEC;                       // elements of a thread
    static constexpr int W = VEC == 8 ? V * 4 : (V + 1) / 2;   // packed words
    __device__ static __forceinline__ int col(int j) {      // first column of vector j
        return (j * T + static_cast<int>(threadIdx.x)) * VEC;
    }
    __device__ static __forceinline__ float get(const uint32_t (&p)[W], int e) {
        return __uint_as_float((e & 1) ? (p[e >> 1] & 0xFFFF0000u) : (p[e >> 1] << 16));
    }
    __device__ static __forceinline__ void put(uint32_t (&p)[W], int e, uint16_t b) {
        if (e & 1) p[e >> 1] = (p[e >> 1] & 0xFFFFu) | (static_cast<uint32_t>(b) << 16);
        else p[e >> 1] = (p[e >> 1] & 0xFFFF0000u) | b;
    }
    __device__ static __forceinline__ void load(uint32_t (&p)[W], const uint16_t* row, int C) {
#pragma unroll
        for (int i = 0; i < W; ++i) p[i] = 0u;              // columns past C read as 0
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = col(j);
            if (c < C) {
                if constexpr (VEC == 8) {
                    const uint4 v = *reinterpret_cast<const uint4*>(row + c);
                    p[4 * j] = v.x;
                    p[4 * j + 1] = v.y;
                    p[4 * j + 2] = v.z;
                    p[4 * j + 3] = v.w;
                } else {
                    put(p, j, row[c]);
                }
            }
        }
    }
    __device__ static __forceinline__ void store(const uint32_t (&p)[W], uint16_t* row, int C) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = col(j);
            if (c < C) {
                if constexpr (VEC == 8)
                    *reinterpret_cast<uint4*>(row + c) = make_uint4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
                else
                    row[c] = static_cast<uint16_t>((j & 1) ? p[j >> 1] >> 16 : p[j >> 1] & 0xFFFFu);
            }
        }
    }
};

__device__ __forceinline__ uint16_t to_bf16_bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// Sum over the block's T threads in a fixed order, in every thread.  `buf`
// alternates between calls, so that one barrier per call is enough.
template <int T>
__device__ __forceinline__ float block_sum(float v, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (T == 32) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) s += buf[w];
    return s;
}

// Maximum of the bit patterns over the block (order-independent; as bits, a
// NaN is larger than an infinity and neither is dropped).
template <int T>
__device__ __forceinline__ uint32_t block_max_bits(uint32_t v, uint32_t* buf) {
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if constexpr (T == 32) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t t = 0;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) t = max(t, buf[w]);
    return t;
}

}  // namespace w4
