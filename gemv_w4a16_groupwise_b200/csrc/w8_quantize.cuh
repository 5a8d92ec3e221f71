// Rows of values as int8 codes with one fp32 scale per row:
//     s = max |v| / 127,   q = rint(127 v / max |v|)
// (symmetric, round half to even).  A row of zeros has s = 0 and q = 0; a row
// with an infinity or a NaN has s = NaN and q = 0, so all it takes part in is
// NaN.
//
// The quotient is not divided out per element: with inv = 127 / max |v|
// rounded up, the code is rint(v inv), one fma.  For bf16 v this is the exact
// quotient rounded half to even.  Write v = i 2^-d and max |v| = b in units of
// the maximum's last place, b in [128, 255], |i| <= 255: the quotient is
// 127 i 2^-d / b, and its distance from a rounding border h + 1/2 is a
// multiple of 1 / (2^(d+1) b), at least 2^-(d+9) when not zero, against an
// error of at most |q| 2^-23 < 2^(8-d) 2^-23 from inv.  Ties: 254 i = (2h+1) b
// 2^d needs 127 to divide b or 2h + 1; b = 254 makes inv a power of two, exact;
// 2h + 1 = 127 is |q| = 63.5, which goes to 64, the even code and the side
// that inv, rounded up, leans to.
#pragma once

#include "common.cuh"

namespace w4 {

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

struct RowScale {
    float scale;   // value of one code
    float inv;     // codes per unit of v pre
    float pre;     // a power of two that keeps inv finite for tiny rows
};

__device__ __forceinline__ RowScale row_scale(float top) {
    RowScale s;
    if (!(top < __uint_as_float(0x7F800000u))) {   // infinity or NaN
        s.scale = __uint_as_float(0x7FC00000u);
        s.inv = 0.0f;
        s.pre = 0.0f;
        return s;
    }
    s.scale = __fdiv_rn(top, 127.0f);
    s.pre = top < 1.2676506e-30f ? 18446744073709551616.0f : 1.0f;      // below 2^-99: times 2^64
    s.inv = top > 0.0f ? __fdiv_ru(127.0f, top * s.pre) : 0.0f;
    return s;
}

// rint(v inv) in the low byte: adding 1.5 * 2^23 leaves the integer, rounded
// half to even, in the low mantissa bits.  A poisoned row (pre = 0) gives 0:
// its values are replaced before the product, as 0 times an infinity is not 0.
__device__ __forceinline__ uint32_t code_bits(float v, const RowScale& s) {
    const float u = s.pre == 1.0f ? v : (s.pre == 0.0f ? 0.0f : v * s.pre);
    return __float_as_uint(fmaf(u, s.inv, 12582912.0f));
}
__device__ __forceinline__ int8_t code1(float v, const RowScale& s) {
    return static_cast<int8_t>(code_bits(v, s) & 0xFFu);
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, const RowScale& s) {
    const uint32_t lo = prmt(code_bits(a, s), code_bits(b, s), 0x0040u);
    const uint32_t hi = prmt(code_bits(c, s), code_bits(d, s), 0x0040u);
    return prmt(lo, hi, 0x5410u);
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const RowScale& s) {
    return make_uint2(codes4(v[0], v[1], v[2], v[3], s), codes4(v[4], v[5], v[6], v[7], s));
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

// One block per row: the largest magnitude, then the codes from a second read
// of the row (an L1 or L2 hit).  channel (fp32 [C], or null) multiplies the
// values first, rounded to fp32.
__global__ void __launch_bounds__(512) quantize_rows_kernel(const uint16_t* __restrict__ X, int C,
                                                            const float* __restrict__ channel,
                                                            int8_t* __restrict__ codes, long long ld,
                                                            float* __restrict__ scales) {
    __shared__ uint32_t buf[32];
    const long long m = blockIdx.x;
    const uint16_t* x = X + static_cast<size_t>(m) * C;
    pdl_launch_dependents();
    pdl_wait();
    auto value = [&](int c) {
        const float v = bf16_bits_to_float(x[c]);
        return channel ? v * channel[c] : v;
    };
    uint32_t top = 0;
    for (int c = threadIdx.x; c < C; c += 512) top = max(top, abs_bits(value(c)));
    top = block_max_bits<512>(top, buf);
    const RowScale sc = row_scale(__uint_as_float(top));
    if (threadIdx.x == 0) scales[m] = sc.scale;
    int8_t* q = codes + static_cast<size_t>(m) * ld;
    for (int c = threadIdx.x; c < C; c += 512) q[c] = code1(value(c), sc);
}

}  // namespace w4
