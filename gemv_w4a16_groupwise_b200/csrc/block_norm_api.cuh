// C-ABI entry points of the block norms: validation and dispatch.  Included
// by w4a16.cu, whose host helpers it uses.
#pragma once

namespace {

// Bytes of a two-stage row pipe.
template <int T, int G, int VEC>
size_t pipe_bytes(int arrays) {
    return static_cast<size_t>(2) * arrays * G * T * 16;
}

template <int T, int G, int VEC>
struct NormLaunch {
    static w4_status run(const w4::NormArgs& a, int sms, cudaStream_t st) {
        const size_t smem = pipe_bytes<T, G, VEC>(1 + (a.y ? 1 : 0) + (a.gate_kind == w4::kGateToken ? 1 : 0));
        const int grid = row_grid(a.M, sms * (1024 / T));
        auto fn = a.scales ? w4::block_norm_kernel<T, G, VEC, true> : w4::block_norm_kernel<T, G, VEC, false>;
        if (smem > 40 * 1024 && ensure_smem(reinterpret_cast<const void*>(fn), smem) != cudaSuccess) return W4_ERR_CUDA;
        launch_pdl(fn, dim3(grid), dim3(T), smem, st, a);
        return launch_status();
    }
};

// Blocks of the backward pass; each leaves a partial row of the weights'
// gradients.  Fewer blocks of at least four rows write less of those and were
// slower all the same (513 x 2047: 15.7 -> 20.6 us): a row's latency counts.
template <int T, int G, int VEC>
struct NormGradBlocks {
    static int run(int M, int sms) {
        return row_grid(M, sms * w4::norm_grad_blocks_per_sm(T, G, VEC));
    }
};
int norm_grad_blocks(int M, int C, int sms) { return dispatch_row<NormGradBlocks>(C, M, sms); }

template <int T, int G, int VEC>
struct NormGradLaunch {
    static w4_status run(const w4::NormGradArgs& a, int blocks, int sums, cudaStream_t st) {
        constexpr bool kSmem = T == 1024;
        const int arrays = 2 + (a.dres ? 1 : 0) + (a.y ? 1 : 0) + (a.gate_kind == w4::kGateToken ? 1 : 0);
        const size_t smem = kSmem ? static_cast<size_t>(sums) * T * G * 8 * sizeof(float) : pipe_bytes<T, G, VEC>(arrays);
        auto fn = w4::block_norm_backward_kernel<T, G, VEC, kSmem>;
        if (smem > 40 * 1024 && ensure_smem(reinterpret_cast<const void*>(fn), smem) != cudaSuccess) return W4_ERR_CUDA;
        launch_pdl(fn, dim3(blocks), dim3(T), smem, st, a);
        return launch_status();
    }
};

bool gate_ok(int gate_kind, const void* gate, const void* y) {
    if (gate_kind < W4_GATE_NONE || gate_kind > W4_GATE_TOKEN) return false;
    return (gate != nullptr) == (gate_kind != W4_GATE_NONE) && (y || !gate);
}

}  // namespace

extern "C" {

w4_status w4_block_norm(const void* x, const void* y, int M, int C, const void* post_weight, const void* gate,
                        int gate_kind, float residual_scale, const void* pre_weight, float weight_offset, float eps,
                        void* residual, void* normed, long long ld, float* scales, float* rstd, void* stream) {
    if (M <= 0 || C <= 0) return W4_ERR_INVALID_ARG;
    if (C > w4::kRowMaxC || M > (1 << 30)) return W4_ERR_UNSUPPORTED;
    if (!gate_ok(gate_kind, gate, y) || !(eps > 0.0f) || !(eps < 3.4e38f)) return W4_ERR_INVALID_ARG;
    if (!x || !pre_weight || !normed || (post_weight && !y) || (residual != nullptr) != (y != nullptr))
        return W4_ERR_INVALID_ARG;
    if (scales && ld < C) return W4_ERR_INVALID_ARG;
    for (const void* p : {x, y, post_weight, gate, pre_weight, static_cast<const void*>(residual),
                          static_cast<const void*>(normed), static_cast<const void*>(scales),
                          static_cast<const void*>(rstd)})
        if (!aligned16(p)) return W4_ERR_ALIGNMENT;
    if (scales && ld % 16 != 0) return W4_ERR_ALIGNMENT;
    w4::NormArgs a;
    a.x = static_cast<const uint16_t*>(x);
    a.y = static_cast<const uint16_t*>(y);
    a.post = static_cast<const uint16_t*>(post_weight);
    a.gate = static_cast<const uint16_t*>(gate);
    a.pre = static_cast<const uint16_t*>(pre_weight);
    a.residual = static_cast<uint16_t*>(residual);
    a.normed = normed;
    a.scales = scales;
    a.rstd = rstd;
    a.M = M;
    a.C = C;
    a.gate_kind = gate_kind;
    a.ld = ld;
    a.alpha = residual_scale;
    a.off = weight_offset;
    a.eps = eps;
    return dispatch_row<NormLaunch>(C, a, device_info(current_device()).sms, static_cast<cudaStream_t>(stream));
}

size_t w4_block_norm_workspace_bytes(int M, int C) {
    if (M <= 0 || C <= 0 || C > w4::kRowMaxC || M > (1 << 30)) return 0;
    const int blocks = norm_grad_blocks(M, C, device_info(current_device()).sms);
    return static_cast<size_t>(3) * blocks * w4::partial_stride(C) * sizeof(float);
}

w4_status w4_block_norm_backward(const void* d_normed, const void* d_residual, const void* residual,
                                 const float* rstd, const void* y, int M, int C, const void* post_weight,
                                 const void* gate, int gate_kind, float residual_scale, const void* pre_weight,
                                 float weight_offset, void* d_x, void* d_y, void* d_pre_weight, void* d_post_weight,
                                 void* d_gate, void* workspace, size_t workspace_bytes, void* stream) {
    if (M <= 0 || C <= 0) return W4_ERR_INVALID_ARG;
    if (C > w4::kRowMaxC || M > (1 << 30)) return W4_ERR_UNSUPPORTED;
    if (!gate_ok(gate_kind, gate, y)) return W4_ERR_INVALID_ARG;
    if (!d_normed || !residual || !rstd || !pre_weight || !d_x || !d_pre_weight || (post_weight && !y))
        return W4_ERR_INVALID_ARG;
    if ((d_y != nullptr) != (y != nullptr) || (d_post_weight != nullptr) != (post_weight != nullptr) ||
        (d_gate != nullptr) != (gate != nullptr))
        return W4_ERR_INVALID_ARG;
    for (const void* p : {d_normed, d_residual, residual, static_cast<const void*>(rstd), y, post_weight, gate,
                          pre_weight, static_cast<const void*>(d_x), static_cast<const void*>(d_y),
                          static_cast<const void*>(d_pre_weight), static_cast<const void*>(d_post_weight),
                          static_cast<const void*>(d_gate), static_cast<const void*>(workspace)})
        if (!aligned16(p)) return W4_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < w4_block_norm_workspace_bytes(M, C)) return W4_ERR_WORKSPACE;
    const bool chan = gate_kind == W4_GATE_CHANNEL;
    w4::NormGradArgs a;
    a.dn = static_cast<const uint16_t*>(d_normed);
    a.dres = static_cast<const uint16_t*>(d_residual);
    a.r = static_cast<const uint16_t*>(residual);
    a.rstd = rstd;
    a.y = static_cast<const uint16_t*>(y);
    a.post = static_cast<const uint16_t*>(post_weight);
    a.gate = static_cast<const uint16_t*>(gate);
    a.pre = static_cast<const uint16_t*>(pre_weight);
    a.dx = static_cast<uint16_t*>(d_x);
    a.dy = static_cast<uint16_t*>(d_y);
    a.dgate_token = chan ? nullptr : static_cast<uint16_t*>(d_gate);
    a.part = static_cast<float*>(workspace);
    a.M = M;
    a.C = C;
    a.gate_kind = gate_kind;
    a.alpha = residual_scale;
    a.off = weight_offset;
    const int blocks = norm_grad_blocks(M, C, device_info(current_device()).sms);
    const int sums = 1 + (post_weight ? 1 : 0) + (chan ? 1 : 0);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const w4_status s = dispatch_row<NormGradLaunch>(C, a, blocks, sums, st);
    if (s != W4_OK) return s;
    // the slabs in order: pre, post, gate
    uint16_t* o[3] = {static_cast<uint16_t*>(d_pre_weight), nullptr, nullptr};
    int k = 1;
    if (post_weight) o[k++] = static_cast<uint16_t*>(d_post_weight);
    if (chan) o[k++] = static_cast<uint16_t*>(d_gate);
    const dim3 grid((C + 31) / 32, sums);
    const float* part = a.part;
    if (blocks > 128)
        launch_pdl(w4::column_sums_kernel<16>, grid, dim3(512), 0, st, part, blocks, C, o[0], o[1], o[2]);
    else
        launch_pdl(w4::column_sums_kernel<8>, grid, dim3(256), 0, st, part, blocks, C, o[0], o[1], o[2]);
    return launch_status();
}

}  // extern "C"
