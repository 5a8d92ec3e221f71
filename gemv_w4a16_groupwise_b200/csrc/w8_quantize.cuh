// Rows of values as int8 codes with one fp32 scale per row:
//     s = max |v| / 127,   q = rint(127 v / max |v|)
// (symmetric, round half to even).  A row of zeros has s = 0 and q = 0; a row
// with an infinity or a NaN has s = NaN and q = 0, so all it takes part in is
// NaN.
//
// No value is divided by the hardware's division: an IEEE division in every
// thread of a row's block, and the scale's, cost more issue slots than the row's
// own values.  How the quotient is had instead depends on the values.
//
// bf16 rows: the code is rint(v inv), one fma, with inv the least fp32 number
// that is not below 127 / max |v|, so above it by less than 2^-23 of it.  This
// is the exact quotient rounded half to even.  Write
// v = i 2^-d and max |v| = b in units of the maximum's last place, b in
// [128, 255], |i| <= 255: the quotient is 127 i 2^-d / b, and its distance from
// a rounding border h + 1/2 is a multiple of 1 / (2^(d+1) b), at least 2^-(d+9)
// when not zero, against less than 2^(8-d) 2^-23 from inv.  Ties: 254 i =
// (2h+1) b 2^d needs 127 to divide b or 2h + 1.  2h + 1 = 127 is |q| = 63.5,
// which goes to 64, the even code and the side that inv leans to; b = 254 makes
// 127 / max |v| a power of two, which inv then is.
// inv is a reciprocal of the hardware's (within 2^-23) times 127, corrected by
// what its product with the maximum leaves of 127 (one Newton step, which
// leaves the rounding alone), and moved up by one where that is still positive.
//
// fp32 rows (products with channel factors, normed rows): quotients lie as close
// to a border as one likes, and many lie on one but for a rounding: both kinds of
// row are products of two bf16 values but for a factor that cancels (the scales of
// quantized bf16 weights are bf16 values over 127), so ties are common.  The code
// is rint of the quotient that fp32 arithmetic gives, 127 v rounded, divided by
// max |v| and rounded.  The division is the product with the reciprocal and one
// correction by what that leaves (Markstein 1990: the quotient as it should be
// rounded).  rint(v inv) takes four operations less for a pair of values, 16.8
// instead of 17.4 us for 2048 x 11008 with factors and 14.0 instead of 14.7 for the
// norm's codes of 2048 x 4096, but puts half as many codes again beside the exact
// ones (3.1e-5 of dY times scales against 2.2e-5, 4.7e-6 of normed rows against
// 2.9e-6).
#pragma once

#include "rows.cuh"

namespace w4 {

// What turns a row's values into codes.
struct RowCodes {
    float inv;     // bf16 rows: codes per unit of v pre; fp32 rows: 1 / top
    float top;     // max |v| pre
    float pre;     // 1, a power of two that keeps inv normal for extreme rows, or 0 for a poisoned row
};

// BF16: the rows' values are bf16's.
template <bool BF16>
__device__ __forceinline__ RowCodes row_codes(float top) {
    RowCodes s;
    s.pre = 1.0f;
    if (!(top < __uint_as_float(0x7F800000u))) {       // infinity or NaN
        s.inv = s.top = s.pre = 0.0f;
        return s;
    }
    // below 2^-99 or from 2^100 on the row is taken times 2^64 or 2^-64, so that
    // the reciprocal stays a normal number
    if (top < 1.5777218e-30f) s.pre = 18446744073709551616.0f;
    if (top >= 1.2676506e30f) s.pre = 5.4210109e-20f;
    top *= s.pre;
    s.top = top;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(top));
    if constexpr (BF16) {
        float i = 127.0f * r;
        i = fmaf(fmaf(-i, top, 127.0f), r, i);
        // the sign of 127 - i top survives its rounding
        s.inv = fmaf(-i, top, 127.0f) > 0.0f ? __uint_as_float(__float_as_uint(i) + 1u) : i;
    } else {
        s.inv = fmaf(fmaf(-r, top, 1.0f), r, r);
    }
    if (!(top > 0.0f)) s.inv = 0.0f;
    return s;
}

// A row's scale, the value of one code.
__device__ __forceinline__ float row_scale(float top) {
    return top < __uint_as_float(0x7F800000u) ? __fdiv_rn(top, 127.0f) : __uint_as_float(0x7FC00000u);
}

// Eight values as codes: rint of the quotient is in the low byte after adding
// 1.5 * 2^23, which leaves the integer, rounded half to even, in the low
// mantissa bits.
template <bool BF16>
__device__ __forceinline__ uint2 codes8(float2 (&v)[4], const RowCodes& s) {
    if (s.pre != 1.0f) {       // the whole row: extreme, or poisoned (0 times an infinity is not 0)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = s.pre == 0.0f ? both(0.0f) : fmul2(v[i], both(s.pre));
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 f;
        if constexpr (BF16) {
            f = ffma2(v[i], both(s.inv), both(12582912.0f));
        } else {
            const float2 a = fmul2(v[i], both(127.0f)), q = fmul2(a, both(s.inv));
            f = fadd2(ffma2(ffma2(q, both(-s.top), a), both(s.inv), q), both(12582912.0f));
        }
        w[i] = prmt(__float_as_uint(f.x), __float_as_uint(f.y), 0x0040u);
    }
    return make_uint2(prmt(w[0], w[1], 0x5410u), prmt(w[2], w[3], 0x5410u));
}

// The codes of a thread's group to its row.
template <int VEC, class S>
__device__ __forceinline__ void store_codes(const S& span, int8_t* row, int g, int C, uint2 w) {
    if constexpr (VEC == 8) {
        const int c = span.col(g, 0);
        if (c < C) *reinterpret_cast<uint2*>(row + c) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t pair = (i < 2 ? w.x : w.y) >> (16 * (i & 1));
            const int c = span.col(g, 2 * i);
            if (span.shift == 0 && c + 1 < C) {
                *reinterpret_cast<uint16_t*>(row + c) = static_cast<uint16_t>(pair);
            } else {
                if (c >= 0 && c < C) row[c] = static_cast<int8_t>(pair & 0xFFu);
                if (c + 1 < C) row[c + 1] = static_cast<int8_t>((pair >> 8) & 0xFFu);
            }
        }
    }
}

// A group's channel factors from memory.
template <int VEC, class S>
__device__ __forceinline__ void channel_factors(const S& span, float2 (&f)[4], const float* __restrict__ channel, int g,
                                                int C) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = both(0.0f);
    if constexpr (VEC == 8) {
        const int c = span.col(g, 0);
        if (c < C) {
            const float4 lo = __ldg(reinterpret_cast<const float4*>(channel + c));
            const float4 hi = __ldg(reinterpret_cast<const float4*>(channel + c + 4));
            f[0] = make_float2(lo.x, lo.y);
            f[1] = make_float2(lo.z, lo.w);
            f[2] = make_float2(hi.x, hi.y);
            f[3] = make_float2(hi.z, hi.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = span.col(g, 2 * i);
            if (c >= 0 && c < C) f[i].x = __ldg(channel + c);
            if (c + 1 < C) f[i].y = __ldg(channel + c + 1);
        }
    }
}

__device__ __forceinline__ void unpack8(float2 (&v)[4], uint4 x) {
    v[0] = unpack_bf16x2(x.x);
    v[1] = unpack_bf16x2(x.y);
    v[2] = unpack_bf16x2(x.z);
    v[3] = unpack_bf16x2(x.w);
}

// Rows of at most 16384: a block holds a row in registers between the maximum
// and the codes, so the row is read once, and has the next row's loads under
// way meanwhile.  Bound by device memory (3 bytes an element): 4096 x 16384 in
// 31 us (6.4 TB/s), 28672 x 4096 in 53; 4096 x 4096 in 9.8 us, where launch and
// latency show.  Every thread
// keeps the channel factors of its columns (twice a row's bytes) in shared
// memory, 16 bytes of a thread beside its neighbours': from L1, 32 bytes apart,
// they took most of the time of a row.  THREADS: an SM's, 1024, or 1536 for some
// shapes with many rows.
template <int T, int G, int VEC, bool CHANNEL, int THREADS = 1024>
__global__ void __launch_bounds__(T, CHANNEL && G > 2 ? 1 : THREADS / T) quantize_rows_kernel(const uint16_t* __restrict__ X, int R, int C,
                                                                    const float* __restrict__ channel,
                                                                    int8_t* __restrict__ codes, long long ld,
                                                                    float* __restrict__ scales) {
    const RowSpan<T, G, VEC> span(blockIdx.x, C);
    extern __shared__ float4 factors[];      // CHANNEL: [2 G][T]
    __shared__ __align__(16) uint32_t buf[2][32];
    pdl_wait();
    pdl_launch_dependents();
    uint4 x[G], next[G];
#pragma unroll
    for (int g = 0; g < G; ++g) next[g] = span.load(X + static_cast<size_t>(blockIdx.x) * C, g, C);
    if constexpr (CHANNEL) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float2 f[4];
            channel_factors<VEC>(span, f, channel, g, C);
            factors[2 * g * T + threadIdx.x] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
            factors[(2 * g + 1) * T + threadIdx.x] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
        }
    }
    int turn = 0;
    for (long long m = blockIdx.x; m < R; m += gridDim.x, turn ^= 1) {
        const bool more = m + gridDim.x < R;
        if (VEC != 8) C = fresh(C);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            x[g] = next[g];
            if (more) next[g] = span.load(X + static_cast<size_t>(m + gridDim.x) * C, g, C);
        }
        uint32_t top;
        float2 v[CHANNEL ? G : 1][4];       // products with the factors are kept, plain values unpacked again
        if constexpr (CHANNEL) {
            float t = 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float4 lo = factors[2 * g * T + threadIdx.x], hi = factors[(2 * g + 1) * T + threadIdx.x];
                unpack8(v[g], x[g]);
                v[g][0] = fmul2(v[g][0], make_float2(lo.x, lo.y));
                v[g][1] = fmul2(v[g][1], make_float2(lo.z, lo.w));
                v[g][2] = fmul2(v[g][2], make_float2(hi.x, hi.y));
                v[g][3] = fmul2(v[g][3], make_float2(hi.z, hi.w));
#pragma unroll
                for (int i = 0; i < 4; ++i) t = max_abs(t, v[g][i]);
            }
            top = __float_as_uint(t);
        } else {
            uint32_t t = 0;
#pragma unroll
            for (int g = 0; g < G; ++g)
                t = max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(t, x[g].x), x[g].y), x[g].z), x[g].w);
            top = max(t << 16, t & 0xFFFF0000u);
        }
        top = block_max_bits<T>(top, buf[turn]);
        const RowCodes sc = row_codes<!CHANNEL>(__uint_as_float(top));
        if (threadIdx.x == 0) scales[m] = row_scale(__uint_as_float(top));
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float2(&u)[4] = v[CHANNEL ? g : 0];
            if constexpr (!CHANNEL) unpack8(u, x[g]);
            store_codes<VEC>(span, codes + static_cast<size_t>(m) * ld, g, C, codes8<!CHANNEL>(u, sc));
        }
    }
}

// Longer rows: a block takes a row 8192 values at a time, and the second pass
// reads it again (from L2).
template <int VEC>
__global__ void __launch_bounds__(1024) quantize_long_rows_kernel(const uint16_t* __restrict__ X, int C,
                                                                  const float* __restrict__ channel,
                                                                  int8_t* __restrict__ codes, long long ld,
                                                                  float* __restrict__ scales) {
    __shared__ __align__(16) uint32_t buf[32];
    const size_t m = blockIdx.x;
    const uint16_t* x = X + m * C;
    pdl_wait();
    pdl_launch_dependents();
    auto values = [&](const RowSpan<1024, 1, VEC>& span, float2 (&v)[4]) {
        unpack8(v, span.load(x, 0, C));
        if (channel) {
            float2 f[4];
            channel_factors<VEC>(span, f, channel, 0, C);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fmul2(v[i], f[i]);
        }
    };
    float t = 0.0f;
#pragma unroll 2
    for (int c0 = 0; c0 <= C; c0 += 8192) {       // a shifted row's last value may be in a piece of its own
        const RowSpan<1024, 1, VEC> span(m, C, c0);
        float2 v[4];
        values(span, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) t = max_abs(t, v[i]);
    }
    t = __uint_as_float(block_max_bits<1024>(__float_as_uint(t), buf));
    const RowCodes sc = channel ? row_codes<false>(t) : row_codes<true>(t);
    if (threadIdx.x == 0) scales[m] = row_scale(t);
#pragma unroll 2
    for (int c0 = 0; c0 <= C; c0 += 8192) {
        const RowSpan<1024, 1, VEC> span(m, C, c0);
        float2 v[4];
        values(span, v);
        store_codes<VEC>(span, codes + m * ld, 0, C, channel ? codes8<false>(v, sc) : codes8<true>(v, sc));
    }
}

}  // namespace w4
