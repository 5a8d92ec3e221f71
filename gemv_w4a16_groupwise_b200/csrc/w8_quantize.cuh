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

#include "rows.cuh"

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

// The channel factors of a thread's columns, kept over its rows.
template <int T, int V, int VEC>
struct ChannelSpan {
    using S = RowSpan<T, V, VEC>;
    float f[S::E];
    __device__ __forceinline__ void load(const float* channel, int C) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = S::col(j);
            if constexpr (VEC == 8) {
                const bool in = c < C;
                const float4 lo = in ? *reinterpret_cast<const float4*>(channel + c) : make_float4(0.f, 0.f, 0.f, 0.f);
                const float4 hi = in ? *reinterpret_cast<const float4*>(channel + c + 4) : lo;
                f[8 * j] = lo.x, f[8 * j + 1] = lo.y, f[8 * j + 2] = lo.z, f[8 * j + 3] = lo.w;
                f[8 * j + 4] = hi.x, f[8 * j + 5] = hi.y, f[8 * j + 6] = hi.z, f[8 * j + 7] = hi.w;
            } else {
                f[j] = c < C ? channel[c] : 0.0f;
            }
        }
    }
};

// Rows of at most 16384: a block holds a row in registers between the maximum
// and the codes, so the row is read once.  Bound by device memory (3 bytes an
// element).  Blocks walk over the rows and keep the channel factors, which
// would otherwise be twice a row's own bytes from L2 every time.
template <int T, int V, int VEC, bool CHANNEL>
__global__ void __launch_bounds__(T) quantize_rows_kernel(const uint16_t* __restrict__ X, int R, int C,
                                                          const float* __restrict__ channel,
                                                          int8_t* __restrict__ codes, long long ld,
                                                          float* __restrict__ scales) {
    using S = RowSpan<T, V, VEC>;
    __shared__ uint32_t buf[2][32];
    pdl_wait();
    pdl_launch_dependents();
    ChannelSpan<T, V, VEC> ch;
    if constexpr (CHANNEL) ch.load(channel, C);
    int turn = 0;
    for (long long m = blockIdx.x; m < R; m += gridDim.x, turn ^= 1) {
        uint32_t p[S::W];
        S::load(p, X + static_cast<size_t>(m) * C, C);
        auto value = [&](int e) { return CHANNEL ? S::get(p, e) * ch.f[e] : S::get(p, e); };
        uint32_t top = 0;       // columns past C read as 0
#pragma unroll
        for (int e = 0; e < S::E; ++e) top = max(top, abs_bits(value(e)));
        top = block_max_bits<T>(top, buf[turn]);
        const RowScale sc = row_scale(__uint_as_float(top));
        if (threadIdx.x == 0) scales[m] = sc.scale;
        int8_t* q = codes + static_cast<size_t>(m) * ld;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = S::col(j);
            if (c < C) {
                if constexpr (VEC == 8) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = value(8 * j + i);
                    *reinterpret_cast<uint2*>(q + c) = codes8(v, sc);
                } else {
                    q[c] = code1(value(j), sc);
                }
            }
        }
    }
}

// Longer rows: the second pass reads the row again (from L2).
template <int VEC>
__global__ void __launch_bounds__(1024) quantize_long_rows_kernel(const uint16_t* __restrict__ X, int C,
                                                                  const float* __restrict__ channel,
                                                                  int8_t* __restrict__ codes, long long ld,
                                                                  float* __restrict__ scales) {
    __shared__ uint32_t buf[32];
    const size_t m = blockIdx.x;
    const uint16_t* x = X + m * C;
    pdl_wait();
    pdl_launch_dependents();
    auto load = [&](int c, float (&v)[VEC]) {
        if constexpr (VEC == 8) {
            const uint4 w = *reinterpret_cast<const uint4*>(x + c);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float((i & 1) ? u[i >> 1] & 0xFFFF0000u : u[i >> 1] << 16);
        } else {
            v[0] = bf16_bits_to_float(x[c]);
        }
        if (channel) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) v[i] *= channel[c + i];
        }
    };
    uint32_t top = 0;
#pragma unroll 2
    for (int c = threadIdx.x * VEC; c < C; c += 1024 * VEC) {
        float v[VEC];
        load(c, v);
#pragma unroll
        for (int i = 0; i < VEC; ++i) top = max(top, abs_bits(v[i]));
    }
    const RowScale sc = row_scale(__uint_as_float(block_max_bits<1024>(top, buf)));
    if (threadIdx.x == 0) scales[m] = sc.scale;
    int8_t* q = codes + m * ld;
#pragma unroll 2
    for (int c = threadIdx.x * VEC; c < C; c += 1024 * VEC) {
        float v[VEC];
        load(c, v);
        if constexpr (VEC == 8) *reinterpret_cast<uint2*>(q + c) = codes8(v, sc);
        else q[c] = code1(v[0], sc);
    }
}

}  // namespace w4
