// C-ABI entry points of the 8-bit layer: validation, planning, dispatch.
// Included by w4a16.cu, whose host helpers it uses.
#pragma once

namespace {

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

w4_status check_w8(int M, int N, int K, long long ldw, int transposed, const void* W, const void* bias,
                   const void* Y) {
    if (M <= 0 || N <= 0 || K <= 0 || ldw < K || !W || !Y) return W4_ERR_INVALID_ARG;
    if ((transposed ? N : K) > w4::kW8MaxReduction) return W4_ERR_UNSUPPORTED;
    if (!aligned16(W) || !aligned16(Y) || (bias && !aligned16(bias)) || ldw % 16 != 0) return W4_ERR_ALIGNMENT;
    return W4_OK;
}

w4_status run_quantize_rows(const uint16_t* X, int R, int C, const float* channel, int8_t* codes, long long ld,
                            float* scales, cudaStream_t st) {
    launch_pdl(w4::quantize_rows_kernel, dim3(R), dim3(512), 0, st, X, C, channel, codes, ld, scales);
    return launch_status();
}

w4_status run_w8_gemm(const w4::W8Args& a, bool transposed, cudaStream_t st) {
    const int out = transposed ? a.K : a.N;
    const dim3 grid((out + 63) / 64, (a.M + 63) / 64);
    if (grid.y > 65535) return W4_ERR_UNSUPPORTED;
    if (transposed) launch_pdl(w4::w8_gemm_simple_kernel<true>, grid, dim3(256), 0, st, a);
    else launch_pdl(w4::w8_gemm_simple_kernel<false>, grid, dim3(256), 0, st, a);
    return launch_status();
}

}  // namespace

extern "C" {

w4_status w8_quantize_rows(const void* X, int R, int C, const float* channel_scales, int8_t* codes, long long ld,
                           float* scales, void* stream) {
    if (R <= 0 || C <= 0 || ld < C || !X || !codes || !scales) return W4_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(codes) || !aligned16(scales) || !aligned16(channel_scales) || ld % 16 != 0)
        return W4_ERR_ALIGNMENT;
    return run_quantize_rows(static_cast<const uint16_t*>(X), R, C, channel_scales, codes, ld, scales,
                             static_cast<cudaStream_t>(stream));
}

size_t w8a8_workspace_bytes(int M, int N, int K, int transposed) {
    (void)M;
    (void)N;
    (void)K;
    (void)transposed;
    return 0;
}

// the tokens' codes and scales lie in front of the product's own workspace
size_t w8a8_linear_workspace_bytes(int M, int N, int K, int transposed) {
    if (M <= 0 || N <= 0 || K <= 0) return 0;
    const size_t red = round16(static_cast<size_t>(transposed ? N : K));
    return M * red + round16(M * sizeof(float)) + w8a8_workspace_bytes(M, N, K, transposed);
}

w4_status w8a8_gemm(const int8_t* A, long long lda, const float* a_scales, int M, int N, int K, const int8_t* W,
                    long long ldw, const float* w_scales, const void* bias, int transposed, void* Y,
                    void* workspace, size_t workspace_bytes, void* stream) {
    const w4_status s = check_w8(M, N, K, ldw, transposed, W, bias, Y);
    if (s != W4_OK && s != W4_ERR_ALIGNMENT) return s;
    if (!A || !a_scales || lda < (transposed ? N : K) || (w_scales == nullptr) != (transposed != 0))
        return W4_ERR_INVALID_ARG;
    if (s != W4_OK || !aligned16(A) || !aligned16(a_scales) || !aligned16(w_scales) || lda % 16 != 0)
        return W4_ERR_ALIGNMENT;
    const size_t need = w8a8_workspace_bytes(M, N, K, transposed);
    if (workspace_bytes < need || (need > 0 && !workspace)) return W4_ERR_WORKSPACE;
    if (!aligned16(workspace)) return W4_ERR_ALIGNMENT;
    const w4::W8Args a = {A, a_scales, W, w_scales, static_cast<const uint16_t*>(bias),
                          static_cast<uint16_t*>(Y), lda, ldw, M, N, K};
    return run_w8_gemm(a, transposed != 0, static_cast<cudaStream_t>(stream));
}

w4_status w8a8_linear(const void* A, int M, int N, int K, const int8_t* W, long long ldw, const float* w_scales,
                      const void* bias, int transposed, void* Y, void* workspace, size_t workspace_bytes,
                      void* stream) {
    const w4_status s = check_w8(M, N, K, ldw, transposed, W, bias, Y);
    if (s != W4_OK && s != W4_ERR_ALIGNMENT) return s;
    if (!A || !w_scales) return W4_ERR_INVALID_ARG;
    if (s != W4_OK || !aligned16(A) || !aligned16(w_scales)) return W4_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < w8a8_linear_workspace_bytes(M, N, K, transposed)) return W4_ERR_WORKSPACE;
    if (!aligned16(workspace)) return W4_ERR_ALIGNMENT;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int red = transposed ? N : K;
    const size_t ld = round16(red);
    int8_t* codes = static_cast<int8_t*>(workspace);
    float* scales = reinterpret_cast<float*>(codes + M * ld);
    const w4_status q = run_quantize_rows(static_cast<const uint16_t*>(A), M, red, transposed ? w_scales : nullptr,
                                          codes, static_cast<long long>(ld), scales, st);
    if (q != W4_OK) return q;
    const w4::W8Args a = {codes, scales, W, transposed ? nullptr : w_scales, static_cast<const uint16_t*>(bias),
                          static_cast<uint16_t*>(Y), static_cast<long long>(ld), ldw, M, N, K};
    return run_w8_gemm(a, transposed != 0, st);
}

}  // extern "C"
