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

}  // namespace w4
