// Rows of bf16 worked on by a thread block, and reductions over the block.
#pragma once

#include "common.cuh"
#include "tma.cuh"

namespace w4 {

constexpr int kRowMaxC = 16384;   // 1024 threads x 2 groups of 8

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void cp_async_16_zfill(void* dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack_bf16x2(float2 v) { return bf162_bits(__floats2bfloat162_rn(v.x, v.y)); }
__device__ __forceinline__ uint16_t to_bf16_bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// A thread's columns of a row: G groups of 8 values, held as 4 words of
// bf16x2.  Columns outside the row read as 0, which is neutral in every sum
// and maximum here.
//
// VEC = 8: a group is 8 consecutive columns, groups of the block's threads
// side by side (rows of whole 16 bytes).
// VEC = 2: the other widths.  A word of a group is a whole word of memory, the
// words of the block's threads side by side: in a row that starts at an odd
// value (`shift` = 1) the pairs begin at column -1, whose half belongs to the
// row before.  A block's rows lie an even number of rows apart, so `shift` is
// the same for all of them and a thread keeps its columns.  (A sum over an odd
// row of odd width is thus added up in another order than over an even one.)
template <int T, int G, int VEC>
struct RowSpan {
    int shift;       // 1: the block's rows start in the middle of a word
    int c0;          // first column of this piece of a row (0 but in long rows)

    // the span of the rows of C values that start at m * C, m = first row's number
    __device__ __forceinline__ explicit RowSpan(long long m, int C, int c0_ = 0)
        : shift(VEC == 8 ? 0 : static_cast<int>(m & C & 1)), c0(c0_) {}
    __device__ __forceinline__ int col(int g, int i) const {     // column of value i of group g
        return c0 + (VEC == 8 ? (g * T + static_cast<int>(threadIdx.x)) * 8 + i
                              : ((g * 4 + (i >> 1)) * T + static_cast<int>(threadIdx.x)) * 2 + (i & 1) - shift);
    }
    // a row of the matrix
    __device__ __forceinline__ uint4 load(const uint16_t* row, int g, int C) const {
        if constexpr (VEC == 8) {
            const int c = col(g, 0);
            return c < C ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0u, 0u, 0u, 0u);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = col(g, 2 * i);
                w[i] = 0u;
                if (c >= 0 && c + 1 < C) w[i] = *reinterpret_cast<const uint32_t*>(row + c);
                else if (c >= 0 && c < C) w[i] = row[c];
                else if (c == -1 && C > 0) w[i] = static_cast<uint32_t>(row[0]) << 16;
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    // a vector over the columns (its words are not the matrix's when shift = 1)
    __device__ __forceinline__ uint4 load_vector(const uint16_t* v, int g, int C) const {
        if constexpr (VEC == 8) {
            return load(v, g, C);
        } else {
            if (shift == 0) return load(v, g, C);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = col(g, 2 * i);
                w[i] = (c >= 0 && c < C ? v[c] : 0u) | (c + 1 < C ? static_cast<uint32_t>(v[c + 1]) << 16 : 0u);
            }
            return make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    __device__ __forceinline__ void store(uint16_t* row, int g, int C, const uint32_t (&w)[4]) const {
        if constexpr (VEC == 8) {
            const int c = col(g, 0);
            if (c < C) *reinterpret_cast<uint4*>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = col(g, 2 * i);
                if (c >= 0 && c + 1 < C) *reinterpret_cast<uint32_t*>(row + c) = w[i];
                else if (c >= 0 && c < C) row[c] = static_cast<uint16_t>(w[i]);
                else if (c == -1 && C > 0) row[0] = static_cast<uint16_t>(w[i] >> 16);
            }
        }
    }
};

// Rows on their way from device memory: every thread copies its own groups of
// the next row ahead (cp.async) and later reads back what it copied itself, so
// the pipe needs no barriers, and no registers for what is in flight or must
// be read again after a reduction.  Two stages of `arrays` rows; without the
// pipe (PIPED = false) a read goes to memory.
template <int T, int G, int VEC, bool PIPED>
struct RowPipe {
    using S = RowSpan<T, G, VEC>;
    uint4* base;             // [2][arrays][G * T], or as many words [G * 4][T]
    int arrays;
    S span;
    __device__ __forceinline__ uint32_t* words(int stage, int array, int g) const {
        return reinterpret_cast<uint32_t*>(base + (stage * arrays + array) * (G * T)) + g * 4 * T + threadIdx.x;
    }
    __device__ __forceinline__ void fetch(int stage, int array, const uint16_t* row, int C) const {
#pragma unroll
        for (int g = 0; PIPED && g < G; ++g) {
            if constexpr (VEC == 8) {
                const int c = span.col(g, 0);
                cp_async_16_zfill(base + (stage * arrays + array) * (G * T) + g * T + threadIdx.x,
                                  row + (c < C ? c : 0), c < C);
            } else {
                // a word's bytes inside the row, but for the half at column -1 (read() drops it)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = span.col(g, 2 * i);
                    cp_async_4(words(stage, array, g) + i * T, row + (c < C ? c : -span.shift),
                               c + 1 < C ? 4u : c < C ? 2u : 0u);
                }
            }
        }
    }
    __device__ __forceinline__ void commit() const {
        if constexpr (PIPED) asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // all but the newest `newer` (0 or 1) groups have landed
    __device__ __forceinline__ void wait(bool newer) const {
        if constexpr (PIPED) {
            if (newer) asm volatile("cp.async.wait_group 1;" ::: "memory");
            else asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
    }
    __device__ __forceinline__ uint4 read(int stage, int array, const uint16_t* row, int g, int C) const {
        if constexpr (!PIPED) {
            return span.load(row, g, C);
        } else if constexpr (VEC == 8) {
            return base[(stage * arrays + array) * (G * T) + g * T + threadIdx.x];
        } else {
            const uint32_t* w = words(stage, array, g);
            uint4 v = make_uint4(w[0], w[T], w[2 * T], w[3 * T]);
            if (g == 0 && threadIdx.x == 0 && span.shift) v.x &= 0xFFFF0000u;
            return v;
        }
    }
};

// The row length, as a value that the compiler takes for new: without it the
// columns' comparisons are all hoisted out of a kernel's loop over rows and
// spilled.
__device__ __forceinline__ int fresh(int C) {
    asm volatile("" : "+r"(C));
    return C;
}

// Sum over the block's T threads in a fixed order, in every thread.  One
// barrier; `buf` (32 entries, 16-byte aligned) is not written again before another barrier has passed.
template <int T>
__device__ __forceinline__ float block_sum(float2 v2, float* buf) {
    float v = v2.x + v2.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < T / 32; w += 4) {
        const float4 u = *reinterpret_cast<const float4*>(buf + w);
        s += (u.x + u.y) + (u.z + u.w);
    }
    return s;
}

// Maximum of non-negative values as bit patterns (order-independent; a NaN is
// larger than an infinity and neither is dropped).
template <int T>
__device__ __forceinline__ uint32_t block_max_bits(uint32_t v, uint32_t* buf) {
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t t = 0;
#pragma unroll
    for (int w = 0; w < T / 32; w += 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(buf + w);
        t = max(t, max(max(u.x, u.y), max(u.z, u.w)));
    }
    return t;
}

// max(m, |v.x|, |v.y|), a NaN kept (the three-operand form of sm_100)
__device__ __forceinline__ float max_abs(float m, float2 v) {
    asm("{\n .reg .f32 a, b;\n abs.f32 a, %1;\n abs.f32 b, %2;\n max.NaN.f32 %0, %0, a, b;\n}\n"
        : "+f"(m)
        : "f"(v.x), "f"(v.y));
    return m;
}
// the larger magnitudes of two pairs of bf16, a NaN kept
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t m, uint32_t w) {
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&m), __habs2(*reinterpret_cast<__nv_bfloat162*>(&w)));
    return bf162_bits(r);
}

}  // namespace w4
