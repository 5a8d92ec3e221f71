// C-ABI entry points of the 8-bit layer: validation, planning, dispatch.
// Included by w4a16.cu, whose host helpers it uses.
#pragma once

namespace {

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

// Scales that the kernels read or write one at a time: part of a batch's or of the channels' may begin anywhere.
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

w4_status check_w8(int M, int N, int K, long long ldw, int transposed, const void* W, const void* bias,
                   const void* Y) {
    if (M <= 0 || N <= 0 || K <= 0 || ldw < K || !W || !Y) return W4_ERR_INVALID_ARG;
    if ((transposed ? N : K) > w4::kW8MaxReduction || std::max(M, std::max(N, K)) > (1 << 30))
        return W4_ERR_UNSUPPORTED;
    if (!aligned16(W) || !aligned16(Y) || (bias && !aligned16(bias)) || ldw % 16 != 0) return W4_ERR_ALIGNMENT;
    return W4_OK;
}

// The block of a row of C: threads T and groups of 8 values each.  One group
// as far as 2048; two from there, with half the threads.
template <template <int, int, int> class Launch, typename... Args>
auto dispatch_row(int C, Args... args) {
    const bool vec = C % 8 == 0;
    if (C <= 1024) return vec ? Launch<128, 1, 8>::run(args...) : Launch<128, 1, 2>::run(args...);
    if (C <= 2048) return vec ? Launch<256, 1, 8>::run(args...) : Launch<256, 1, 2>::run(args...);
    if (C <= 4096) return vec ? Launch<256, 2, 8>::run(args...) : Launch<256, 2, 2>::run(args...);
    if (C <= 8192) return vec ? Launch<512, 2, 8>::run(args...) : Launch<512, 2, 2>::run(args...);
    return vec ? Launch<1024, 2, 8>::run(args...) : Launch<1024, 2, 2>::run(args...);
}

// Blocks that walk over M rows: a row each, or an even number (see RowSpan).
int row_grid(int M, int blocks) { return M <= blocks ? M : std::max(2, blocks & ~1); }

template <int T, int G, int VEC>
struct QuantizeLaunch {
    static w4_status run(const uint16_t* X, int R, int C, const float* channel, int8_t* codes, long long ld,
                         float* scales, int sms, cudaStream_t st) {
        // many rows: 1536 threads an SM where a thread has two groups (28672 x 4096: 58 -> 53 us) or words
        // (8192 x 1001: 10.7 -> 9.3); one group of whole 16 bytes loses by it (8192 x 1024: 7.2 -> 7.9)
        constexpr bool kDenser = T <= 512 && (G == 2 || (G == 1 && VEC == 2));
        auto fn = channel ? w4::quantize_rows_kernel<T, G, VEC, true> : w4::quantize_rows_kernel<T, G, VEC, false>;
        int blocks = sms * (1024 / T);
        if (kDenser && !channel && R >= 2 * sms * (1536 / T)) {
            fn = w4::quantize_rows_kernel<T, G, VEC, false, kDenser ? 1536 : 1024>;
            blocks = sms * (1536 / T);
        }
        const size_t smem = channel ? static_cast<size_t>(G) * T * 32 : 0;
        if (smem > 40 * 1024 && ensure_smem(reinterpret_cast<const void*>(fn), smem) != cudaSuccess) return W4_ERR_CUDA;
        launch_pdl(fn, dim3(row_grid(R, blocks)), dim3(T), smem, st, X, R, C, channel, codes, ld, scales);
        return launch_status();
    }
};

// More than 8192 values in whole 16 bytes: three or four groups a thread waste fewer of them than 1024
// threads would.
template <>
struct QuantizeLaunch<1024, 2, 8> {
    template <typename... Args>
    static w4_status run(const uint16_t* X, int R, int C, Args... args) {
        return C <= 12288 ? QuantizeLaunch<512, 3, 8>::run(X, R, C, args...)
                          : QuantizeLaunch<512, 4, 8>::run(X, R, C, args...);
    }
};

w4_status run_quantize_rows(const uint16_t* X, int R, int C, const float* channel, int8_t* codes, long long ld,
                            float* scales, cudaStream_t st) {
    const int sms = device_info(current_device()).sms;
    if (C <= w4::kRowMaxC) return dispatch_row<QuantizeLaunch>(C, X, R, C, channel, codes, ld, scales, sms, st);
    if (C % 8 == 0)
        launch_pdl(w4::quantize_long_rows_kernel<8>, dim3(R), dim3(1024), 0, st, X, C, channel, codes, ld, scales);
    else
        launch_pdl(w4::quantize_long_rows_kernel<2>, dim3(R), dim3(1024), 0, st, X, C, channel, codes, ld, scales);
    return launch_status();
}

// The tensor-core product's plan: the token tile, whole tiles F and the pairs
// that share the others' reduction.
struct W8Plan {
    int TN = 32, tiles_m = 1, tiles = 1, F = 0, chunks = 1, cut_pairs = 1, grid_pairs = 1;
    size_t ws = 0;
    double us = 0.0;     // the estimate it was chosen by
};

// A plan's time by what was measured on 74 pairs: a call with one stage per
// tile takes `base`; every further stage of a pair adds `stage` (0.275 us for
// 256 tokens is the products' time, the others wait for the 16 KB of weights
// and their tokens from L2); a call is not faster than its weights through
// device memory; partial tiles, their sums and the second kernel add `cut`.
// (us)               TN =    32     64    128    256
constexpr double kW8Base[] = {4.6, 4.8, 5.5, 6.5};
constexpr double kW8Stage[] = {0.175, 0.18, 0.20, 0.275};
constexpr double kW8Cut[] = {4.2, 4.5, 9.0, 11.0};

W8Plan plan_w8_as(int M, int N, int K, bool transposed, int pairs, int size, bool cut) {
    W8Plan p;
    const int out = transposed ? K : N, red = transposed ? N : K;
    p.TN = 32 << size;
    p.tiles_m = (M + p.TN - 1) / p.TN;
    p.tiles = p.tiles_m * ((out + w4::kW8Rows - 1) / w4::kW8Rows);
    p.chunks = (red + w4::kW8Red - 1) / w4::kW8Red;
    p.F = cut ? p.tiles - p.tiles % pairs : p.tiles;
    const long long total = static_cast<long long>(p.tiles - p.F) * p.chunks;
    p.cut_pairs = static_cast<int>(std::max<long long>(1, std::min<long long>(pairs, total / 4)));
    p.grid_pairs = std::max(std::min(p.F, pairs), total > 0 ? p.cut_pairs : 1);
    // one pair leaves nothing to add up
    const bool partials = total > 0 && p.cut_pairs > 1;
    if (partials) p.ws = static_cast<size_t>(2) * p.cut_pairs * p.TN * w4::kW8Rows * sizeof(int32_t);
    const double stages = static_cast<double>((p.F + pairs - 1) / pairs) * p.chunks +
                          static_cast<double>(total) / p.cut_pairs;
    p.us = std::max(kW8Base[size] + stages * kW8Stage[size],
                    static_cast<double>(N) * K / 6.3e6 + 3.5) + (partials ? kW8Cut[size] : 0.0);
    return p;
}

W8Plan plan_w8(int M, int N, int K, bool transposed, int sms) {
    const int pairs = std::max(1, sms / 2);
    W8Plan best;
    best.us = 1e30;
    for (int size = 0; size < 4; ++size) {
        W8Plan p = plan_w8_as(M, N, K, transposed, pairs, size, false);
        const W8Plan cut = plan_w8_as(M, N, K, transposed, pairs, size, true);
        if (cut.us < p.us) p = cut;
        // Near ties go to the wider tile: the estimate flatters the narrower one. Of 80 sizes drawn
        // among the 4 % that this changes, 71 ran faster with the wider tile, by 13 % on the
        // geometric mean (1458 x 1287 x 468: 5.7 against 6.6 us; 59 x 29513 x 4185 transposed: 33
        // against 41), 9 slower (384 x 19008 x 6400 transposed: 59 against 45; the others by 3 to 10 %).
        if (p.us < 1.01 * best.us) best = p;
        if (M <= (32 << size)) break;    // a wider tile would only be emptier
    }
    return best;
}

// int8 rows, `ld` bytes apart, in boxes of 128 bytes x box_rows with the
// 128-byte swizzle; out-of-range bytes read as 0.
bool make_map_i8(CUtensorMap* map, const void* ptr, uint64_t rows, uint64_t cols, uint64_t ld, uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t gdim[2] = {cols, rows};
    cuuint64_t gstride[1] = {ld};
    cuuint32_t box[2] = {128, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), gdim, gstride, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool TR, int TN>
w4_status launch_w8_tc(const W8Plan& p, const w4::W8Args& g, int32_t* part, bool early, const DeviceInfo& di,
                       cudaStream_t st) {
    constexpr int kStage = w4::w8_stage_bytes(TN);
    const size_t fixed = 1024 + w4::kW8EpiBytes + 128;
    const int stages = std::min(10, static_cast<int>((di.max_smem_optin - fixed) / (kStage + 16)));
    if (di.max_smem_optin < 200 * 1024 || stages < 2) return W4_ERR_UNSUPPORTED;
    const size_t smem = fixed + static_cast<size_t>(stages) * (kStage + 16);
    CUtensorMap wmap, amap;
    const int red = TR ? g.N : g.K;
    if (!make_map_i8(&wmap, g.W, g.N, g.K, g.ldw, 128) || !make_map_i8(&amap, g.A, g.M, red, g.lda, TN / 2))
        return W4_ERR_CUDA;
    auto fn = w4::w8_gemm_tc_kernel<TR, TN>;
    if (ensure_smem(reinterpret_cast<const void*>(fn), smem) != cudaSuccess) return W4_ERR_CUDA;
    const w4::W8TcArgs a = {g, part, p.tiles_m, p.tiles, static_cast<uint32_t>((1ull << 32) / p.tiles_m + 1),
                            p.grid_pairs % p.tiles_m, p.grid_pairs / p.tiles_m, p.F, p.chunks, p.cut_pairs, stages,
                            early ? 1 : 0, withheld_stage(current_device()).load(std::memory_order_relaxed) - 1};
    launch_pdl(fn, dim3(2 * p.grid_pairs), dim3(w4::kW8Threads), smem, st, wmap, amap, a);
    const w4_status s = launch_status();
    if (s != W4_OK || p.ws == 0) return s;
    launch_pdl(w4::w8_finalize_kernel<TR>, dim3(TN * (w4::kW8Rows / 4) / 256, p.tiles - p.F), dim3(256), 0, st, a, TN);
    return launch_status();
}

// The stream kernel serves forward products of a few tokens whose codes it can
// hold (8 tokens as far as K = 6656).
bool w8_gemv_serves(int M, int K, bool transposed) {
    return !transposed && M <= w4::kGvMaxTokens &&
           static_cast<long long>(M) * w4::w8_gemv_token_bytes(K) <= w4::kGvCodeBytes;
}

// Whether w8_gemv_kernel quantizes the tokens itself, and for how many at
// once (1, 2 or 4; 0: it does not): rows of whole 16 bytes, at most
// kGvFusedValues values.
int w8_gemv_fused(int M, int K, bool transposed) {
    if (transposed || M > 4 || K % 8 != 0) return 0;
    const int MT = M > 2 ? 4 : M;
    return static_cast<long long>(MT) * K <= w4::kGvFusedValues ? MT : 0;
}

template <int MT>
w4_status launch_w8_gemv(const w4::W8Args& p, const uint16_t* X, cudaStream_t st) {
    const w4::W8GemvArgs a = {p, X};
    const size_t smem =
        static_cast<size_t>(MT > 0 ? MT : p.M) * w4::w8_gemv_token_bytes(p.K) + (MT > 0 ? 2 * w4::kGvFusedValues : 0);
    if (smem > 40 * 1024 &&
        ensure_smem(reinterpret_cast<const void*>(w4::w8_gemv_kernel<MT>), w4::kGvMaxSmem) != cudaSuccess)
        return W4_ERR_CUDA;
    // at most two blocks an SM, with equal shares of the 16-row blocks
    const int blocks = (p.N + w4::kGvRows - 1) / w4::kGvRows;
    const int slots = 2 * device_info(current_device()).sms;
    const int each = (blocks + slots - 1) / slots;
    launch_pdl(w4::w8_gemv_kernel<MT>, dim3((blocks + each - 1) / each), dim3(w4::kGvWarps * 32), smem, st, a);
    return launch_status();
}

// `early`: the kernel launched just before on the stream is run_quantize_rows,
// which does not write the weights and lets its dependents start only after
// all that came before it.
w4_status run_w8_gemm(const w4::W8Args& a, bool transposed, void* ws, bool early, cudaStream_t st) {
    if (w8_gemv_serves(a.M, a.K, transposed)) return launch_w8_gemv<0>(a, nullptr, st);
    const DeviceInfo di = device_info(current_device());
    const W8Plan p = plan_w8(a.M, a.N, a.K, transposed, di.sms);
    int32_t* part = static_cast<int32_t*>(ws);
    switch (p.TN) {
        case 32:
            return transposed ? launch_w8_tc<true, 32>(p, a, part, early, di, st)
                              : launch_w8_tc<false, 32>(p, a, part, early, di, st);
        case 64:
            return transposed ? launch_w8_tc<true, 64>(p, a, part, early, di, st)
                              : launch_w8_tc<false, 64>(p, a, part, early, di, st);
        case 128:
            return transposed ? launch_w8_tc<true, 128>(p, a, part, early, di, st)
                              : launch_w8_tc<false, 128>(p, a, part, early, di, st);
        default:
            return transposed ? launch_w8_tc<true, 256>(p, a, part, early, di, st)
                              : launch_w8_tc<false, 256>(p, a, part, early, di, st);
    }
}

}  // namespace

extern "C" {

w4_status w8_quantize_rows(const void* X, int R, int C, const float* channel_scales, int8_t* codes, long long ld,
                           float* scales, void* stream) {
    if (R <= 0 || C <= 0 || ld < C || !X || !codes || !scales) return W4_ERR_INVALID_ARG;
    if (std::max(R, C) > (1 << 30)) return W4_ERR_UNSUPPORTED;
    if (!aligned16(X) || !aligned16(codes) || !aligned4(scales) || !aligned16(channel_scales) || ld % 16 != 0)
        return W4_ERR_ALIGNMENT;
    return run_quantize_rows(static_cast<const uint16_t*>(X), R, C, channel_scales, codes, ld, scales,
                             static_cast<cudaStream_t>(stream));
}

size_t w8a8_workspace_bytes(int M, int N, int K, int transposed) {
    if (M <= 0 || N <= 0 || K <= 0 || w8_gemv_serves(M, K, transposed != 0)) return 0;
    return plan_w8(M, N, K, transposed != 0, device_info(current_device()).sms).ws;
}

// the tokens' codes and scales lie in front of the product's own workspace
size_t w8a8_linear_workspace_bytes(int M, int N, int K, int transposed) {
    if (M <= 0 || N <= 0 || K <= 0 || w8_gemv_fused(M, K, transposed != 0)) return 0;
    const size_t red = round16(static_cast<size_t>(transposed ? N : K));
    return round16(M * red) + round16(M * sizeof(float)) + w8a8_workspace_bytes(M, N, K, transposed);
}

w4_status w8a8_gemm(const int8_t* A, long long lda, const float* a_scales, int M, int N, int K, const int8_t* W,
                    long long ldw, const float* w_scales, const void* bias, int transposed, void* Y,
                    void* workspace, size_t workspace_bytes, void* stream) {
    const w4_status s = check_w8(M, N, K, ldw, transposed, W, bias, Y);
    if (s != W4_OK && s != W4_ERR_ALIGNMENT) return s;
    if (!A || !a_scales || lda < (transposed ? N : K) || (w_scales == nullptr) != (transposed != 0))
        return W4_ERR_INVALID_ARG;
    if (s != W4_OK || !aligned16(A) || !aligned4(a_scales) || !aligned4(w_scales) || lda % 16 != 0)
        return W4_ERR_ALIGNMENT;
    const size_t need = w8a8_workspace_bytes(M, N, K, transposed);
    if (workspace_bytes < need || (need > 0 && !workspace)) return W4_ERR_WORKSPACE;
    if (!aligned16(workspace)) return W4_ERR_ALIGNMENT;
    const w4::W8Args a = {A, a_scales, W, w_scales, static_cast<const uint16_t*>(bias),
                          static_cast<uint16_t*>(Y), lda, ldw, M, N, K};
    return run_w8_gemm(a, transposed != 0, workspace, false, static_cast<cudaStream_t>(stream));
}

w4_status w8a8_linear(const void* A, int M, int N, int K, const int8_t* W, long long ldw, const float* w_scales,
                      const void* bias, int transposed, void* Y, void* workspace, size_t workspace_bytes,
                      void* stream) {
    const w4_status s = check_w8(M, N, K, ldw, transposed, W, bias, Y);
    if (s != W4_OK && s != W4_ERR_ALIGNMENT) return s;
    if (!A || !w_scales) return W4_ERR_INVALID_ARG;
    if (s != W4_OK || !aligned16(A) || !aligned16(w_scales)) return W4_ERR_ALIGNMENT;
    const size_t need = w8a8_linear_workspace_bytes(M, N, K, transposed);
    if (workspace_bytes < need || (need > 0 && !workspace)) return W4_ERR_WORKSPACE;
    if (!aligned16(workspace)) return W4_ERR_ALIGNMENT;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (const int MT = w8_gemv_fused(M, K, transposed != 0)) {
        const w4::W8Args p = {nullptr, nullptr, W, w_scales, static_cast<const uint16_t*>(bias),
                              static_cast<uint16_t*>(Y), 0, ldw, M, N, K};
        const uint16_t* X = static_cast<const uint16_t*>(A);
        return MT == 1 ? launch_w8_gemv<1>(p, X, st) : MT == 2 ? launch_w8_gemv<2>(p, X, st) : launch_w8_gemv<4>(p, X, st);
    }
    const int red = transposed ? N : K;
    const size_t ld = round16(red);
    int8_t* codes = static_cast<int8_t*>(workspace);
    float* scales = reinterpret_cast<float*>(codes + M * ld);
    const w4_status q = run_quantize_rows(static_cast<const uint16_t*>(A), M, red, transposed ? w_scales : nullptr,
                                          codes, static_cast<long long>(ld), scales, st);
    if (q != W4_OK) return q;
    const w4::W8Args a = {codes, scales, W, transposed ? nullptr : w_scales, static_cast<const uint16_t*>(bias),
                          static_cast<uint16_t*>(Y), static_cast<long long>(ld), ldw, M, N, K};
    return run_w8_gemm(a, transposed != 0, reinterpret_cast<uint8_t*>(scales) + round16(M * sizeof(float)), true,
                       st);
}

}  // extern "C"
