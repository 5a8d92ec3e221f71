// Matrix product in 8-bit integers with scales for each token and channel:
//     forward     Y[m, n]  = bf16(a_s[m] w_s[n] sum_k a[m, k] w[n, k] + bias[n])
//     transposed  dX[m, k] = bf16(a_s[m] sum_n a[m, n] w[n, k] + bias[k])
// The integer sums are exact (int32; the reduction length is limited so that
// no sum of products of any two codes overflows), so they do not depend on
// their order; scales and bias are applied in fp32 and rounded once.
#pragma once

#include "common.cuh"

namespace w4 {

// -128 * -128 * 131071 < 2^31
constexpr int kW8MaxReduction = 131071;

struct W8Args {
    const int8_t* A;       // tokens' codes [M, red], row stride lda
    const float* a_scales;
    const int8_t* W;       // weights' codes [N, K], row stride ldw
    const float* w_scales; // forward only
    const uint16_t* bias;
    uint16_t* Y;           // [M, out]
    long long lda, ldw;
    int M, N, K;
};

// acc a_s w_s + bias, rounded once
__device__ __forceinline__ uint16_t w8_output(int acc, float scale, float bias) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(fmaf(static_cast<float>(acc), scale, bias)));
}

// 64 tokens x 64 outputs per block, 64-long slices of the reduction in shared
// memory as words of four codes, dp4a.
template <bool TR>
__global__ void __launch_bounds__(256) w8_gemm_simple_kernel(const W8Args a) {
    __shared__ int8_t sa[64][68], sw[64][68];
    const int out = TR ? a.K : a.N, red = TR ? a.N : a.K;
    const int m0 = blockIdx.y * 64, o0 = blockIdx.x * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    pdl_launch_dependents();
    pdl_wait();
    int acc[4][4] = {};
    for (int k0 = 0; k0 < red; k0 += 64) {
        for (int i = threadIdx.x; i < 64 * 64; i += 256) {
            const int r = i >> 6, c = i & 63;
            sa[r][c] = (m0 + r < a.M && k0 + c < red) ? a.A[static_cast<size_t>(m0 + r) * a.lda + k0 + c] : 0;
            if (TR) sw[c][r] = (k0 + r < red && o0 + c < out) ? a.W[static_cast<size_t>(k0 + r) * a.ldw + o0 + c] : 0;
            else sw[r][c] = (o0 + r < out && k0 + c < red) ? a.W[static_cast<size_t>(o0 + r) * a.ldw + k0 + c] : 0;
        }
        __syncthreads();
        for (int k = 0; k < 64; k += 4) {
            int av[4], wv[4];
            for (int i = 0; i < 4; ++i) {
                av[i] = *reinterpret_cast<const int*>(&sa[ty + 16 * i][k]);
                wv[i] = *reinterpret_cast<const int*>(&sw[tx + 16 * i][k]);
            }
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(av[i], wv[j], acc[i][j]);
        }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty + 16 * i, o = o0 + tx + 16 * j;
            if (m < a.M && o < out)
                a.Y[static_cast<size_t>(m) * out + o] =
                    w8_output(acc[i][j], TR ? a.a_scales[m] : a.a_scales[m] * a.w_scales[o],
                              a.bias ? bf16_bits_to_float(a.bias[o]) : 0.0f);
        }
}

}  // namespace w4
