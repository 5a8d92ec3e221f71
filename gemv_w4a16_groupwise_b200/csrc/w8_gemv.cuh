// Small-batch forward product (M <= 8): Y = A . W^T with int8 codes.
//
// Bound by the weights' bytes, so the kernel is a stream with little in its
// way: a block takes 16 weight rows at a time, its 8 warps interleaved 64-byte
// pieces of them, and every lane has 16 loads of 16 bytes under way (64 KB a
// block, at most two blocks an SM): the next ones are asked for as soon as the
// products have taken the last, before the sums of a finished 16 rows are
// added up.  The loads land where
// mma.sync.m16n8k32 wants them: lane (g, t) holds bytes 16 t .. 16 t + 15 of a
// piece of rows g and g + 8, and of token g; that the four words stand for
// other k than the instruction's own order is the same on both sides.  The
// integer sums of the warps are added in shared memory.  1 x 28672 x 4096 in
// 20.4 us (5.8 TB/s), 1 x 6144 x 4096 in 7.5 us; four blocks with half the loads
// each take 28 and 9.8.  Every block takes the same number of 16-row blocks, so
// the grid does not always fill the SMs: 28672 outputs are 256 blocks of 7 (40 of
// 148 SMs hold one), 6144 are 192 of 2 (104 hold one, with 64 KB in flight), and
// that is what bounds the second.
//
// MT > 0: bf16 tokens, quantized by every block for itself while its first
// weights are on their way (up to 16384 values a block, from L2): one launch
// for a decoding step's layer instead of two, and no codes through memory.
// MT = 0: the tokens' codes are copied to shared memory.
#pragma once

#include "w8_gemm.cuh"
#include "w8_quantize.cuh"

namespace w4 {

constexpr int kGvRows = 16, kGvWarps = 8, kGvUnroll = 8, kGvMaxTokens = 8;
// Bytes of the tokens' codes that a block takes into shared memory.  Past that
// (4 tokens of 14336) the copying in front of every block costs more than the
// tensor-core product's fixed time: 18.6 us against 17 at 4096 x 14336.
constexpr int kGvCodeBytes = 56 * 1024;
constexpr int kGvMaxSmem = 64 * 1024;
constexpr int kGvFusedValues = 16384;      // MT * K that a block may quantize for itself: 32 KB of bf16

// Bytes of a token's codes in shared memory: whole 512-byte steps of the
// block, and 64 more, so that two tokens' 64-byte pieces lie in distinct banks.
__host__ __device__ inline int w8_gemv_token_bytes(int K) { return (K + 511) / 512 * 512 + 64; }

struct W8GemvArgs {
    W8Args p;
    const uint16_t* X;     // MT > 0: bf16 tokens [M, K]
};

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg_stream_16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Bytes k .. k + 15 of a row of K, zero from K on.
__device__ __forceinline__ uint4 mask_tail(uint4 v, int k, int K) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int left = K - k - 4 * i;         // bytes of this word inside the row
        w[i] = left >= 4 ? w[i] : left <= 0 ? 0u : w[i] & (0xFFFFFFFFu >> (8 * (4 - left)));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int MT>
__global__ void __launch_bounds__(kGvWarps * 32, 2) w8_gemv_kernel(const W8GemvArgs a) {
    extern __shared__ __align__(16) uint8_t tokens[];      // rows of w8_gemv_token_bytes(K); MT > 0: then bf16
    __shared__ int red[2][kGvWarps][kGvMaxTokens][kGvRows];
    __shared__ uint32_t tops[kGvWarps];
    __shared__ float token_scale[kGvMaxTokens];
    const int K = a.p.K, N = a.p.N, M = a.p.M;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int blocks = (N + kGvRows - 1) / kGvRows;
    const int k_first = 64 * warp + 16 * t;                // then every 512
    pdl_launch_dependents();
    pdl_wait();

    const int tb = w8_gemv_token_bytes(K);
    // 256 / MT threads per token; their vectors of 8 values lie kT apart and
    // go through shared memory, as registers are full of weights
    constexpr int kT = kGvWarps * 32 / (MT > 0 ? MT : 1), kV = kGvFusedValues / (8 * kGvWarps * 32);
    uint4* raw = reinterpret_cast<uint4*>(tokens + MT * tb);
    if constexpr (MT > 0) {
        const int m = threadIdx.x / kT, i0 = threadIdx.x % kT;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int k = (v * kT + i0) * 8;
            cp_async_16_zfill(raw + v * kGvWarps * 32 + threadIdx.x,
                              a.X + (k < K && m < M ? static_cast<size_t>(m) * K + k : 0), k < K && m < M);
        }
    }

    uint4 lo[kGvUnroll], hi[kGvUnroll];
    auto load = [&](int b, int k0) {
        // rows past N repeat the last one; their sums are dropped
        const int8_t* w_lo = a.p.W + static_cast<size_t>(min(b * kGvRows + g, N - 1)) * a.p.ldw;
        const int8_t* w_hi = a.p.W + static_cast<size_t>(min(b * kGvRows + g + 8, N - 1)) * a.p.ldw;
#pragma unroll
        for (int i = 0; i < kGvUnroll; ++i) {
            const int k = k0 + 512 * i;
            lo[i] = hi[i] = make_uint4(0u, 0u, 0u, 0u);
            if (k < K) {
                lo[i] = ldg_stream_16(w_lo + k);
                hi[i] = ldg_stream_16(w_hi + k);
            }
        }
    };
    load(blockIdx.x, k_first);

    if constexpr (MT > 0) {
        asm volatile("cp.async.wait_all;" ::: "memory");   // every thread reads back what it copied
        const int m = threadIdx.x / kT, i0 = threadIdx.x % kT;
        uint32_t top = 0;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const uint4 x = raw[v * kGvWarps * 32 + threadIdx.x];
            top = max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(top, x.x), x.y), x.z), x.w);
        }
        top = max(top << 16, top & 0xFFFF0000u);
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if (lane == 0) tops[warp] = top;
        __syncthreads();
        top = 0;
#pragma unroll
        for (int w = 0; w < kT / 32; ++w) top = max(top, tops[m * (kT / 32) + w]);
        const RowCodes sc = row_codes<true>(__uint_as_float(top));
        if (i0 == 0) token_scale[m] = row_scale(__uint_as_float(top));
        // codes, and zeros up to the end of the block's last step
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int k = (v * kT + i0) * 8;
            if (k < tb - 64) {
                const uint4 x = raw[v * kGvWarps * 32 + threadIdx.x];
                float2 f[4] = {unpack_bf16x2(x.x), unpack_bf16x2(x.y), unpack_bf16x2(x.z), unpack_bf16x2(x.w)};
                *reinterpret_cast<uint2*>(tokens + m * tb + k) = codes8<true>(f, sc);
            }
        }
        __syncthreads();
    }

    if constexpr (MT == 0) {
        // the codes, and zeros up to the end of the block's last step
        for (int m = 0; m < M; ++m)
            for (int k = threadIdx.x * 16; k < tb - 64; k += kGvWarps * 32 * 16) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (k < K) x = *reinterpret_cast<const uint4*>(a.p.A + static_cast<size_t>(m) * a.p.lda + k);
                if (k + 16 > K) x = mask_tail(x, k, K);
                *reinterpret_cast<uint4*>(tokens + m * tb + k) = x;
            }
        __syncthreads();
    }
    const int held = MT > 0 ? MT : M;      // tokens in shared memory

    int c[4] = {0, 0, 0, 0};
    int turn = 0;
    int k0 = k_first;
    for (int b = blockIdx.x; b < blocks;) {
#pragma unroll
        for (int i = 0; i < kGvUnroll; ++i) {
            const int k = k0 + 512 * i;
            if (k - 16 * t >= K) break;                    // the warp's piece lies behind the row
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (g < held) x = *reinterpret_cast<const uint4*>(tokens + g * tb + k);
            mma_s8(c, lo[i].x, hi[i].x, lo[i].y, hi[i].y, x.x, x.y);
            mma_s8(c, lo[i].z, hi[i].z, lo[i].w, hi[i].w, x.z, x.w);
        }
        k0 += 512 * kGvUnroll;
        const bool done = k0 - k_first >= (K + 511) / 512 * 512;       // the same in every warp
        const int here = b;
        if (done) {
            b += gridDim.x;
            k0 = k_first;
        }
        if (b < blocks) load(b, k0);
        if (!done) continue;
        red[turn][warp][2 * t][g] = c[0];
        red[turn][warp][2 * t + 1][g] = c[1];
        red[turn][warp][2 * t][g + 8] = c[2];
        red[turn][warp][2 * t + 1][g + 8] = c[3];
        c[0] = c[1] = c[2] = c[3] = 0;
        __syncthreads();
        const int m = threadIdx.x / kGvRows, r = threadIdx.x % kGvRows, n = here * kGvRows + r;
        if (m < M && n < N) {
            int s = 0;
#pragma unroll
            for (int w = 0; w < kGvWarps; ++w) s += red[turn][w][m][r];
            const float as = MT > 0 ? token_scale[m] : a.p.a_scales[m];
            a.p.Y[static_cast<size_t>(m) * N + n] =
                w8_output(s, as * a.p.w_scales[n], a.p.bias ? bf16_bits_to_float(a.p.bias[n]) : 0.0f);
        }
        turn ^= 1;
    }
}

}  // namespace w4
