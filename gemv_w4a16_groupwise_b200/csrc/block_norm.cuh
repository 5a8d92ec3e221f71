// Norms around a transformer block fused with the residual add between them:
//     t = y;  t = norm(y) (post + off);  t = t gate        (each where given)
//     r = bf16(x + alpha t)                                the residual stream
//     n = norm(r) (pre + off)                              the next block's input
// norm(v) = v / sqrt(mean(v^2) + eps).  n leaves as bf16 (for the w4a16
// products) or as int8 codes with one scale per row (for the 8-bit ones).
// The second norm reads r as it is stored, so the fused call is the add
// followed by a norm of the stored residual, and the backward pass, which
// sees only the stored values, differentiates what was computed.
//
// Backward, with xh = r rstd_r, yh = y rstd_y (or y), dh = dn (pre + off):
//     dr     = d_res + rstd_r (dh - xh mean(dh xh))        = d_x
//     dt     = alpha dr;  d_gate = dt u,  u = yh (post + off) or y;  dt *= gate
//     d_post = sum_m dt yh;  dt *= (post + off)
//     d_y    = rstd_y (dt - yh mean(dt yh))                (dt without a post norm)
//     d_pre  = sum_m dn xh
//
// Both kernels are bound by device memory: a row is read once and held in
// registers as bf16 (half the registers of fp32) between the reductions.
// Sums and statistics are fp32 in a fixed order.
#pragma once

#include "rows.cuh"
#include "w8_quantize.cuh"

namespace w4 {

enum GateKind { kGateNone = 0, kGateChannel = 1, kGateToken = 2 };

struct NormArgs {
    const uint16_t* x;
    const uint16_t* y;           // null: r = x
    const uint16_t* post;        // null: no norm after the block
    const uint16_t* gate;
    const uint16_t* pre;
    uint16_t* residual;          // unused when y is null
    void* normed;                // bf16 [M, C], or int8 codes with row stride ld
    float* scales;               // of the codes
    float* rstd;                 // [2, M]: post norm (0 without one), pre norm; or null
    int M, C, gate_kind;
    long long ld;
    float alpha, off, eps;
};

template <int T, int V, int VEC, bool CODES>
__global__ void __launch_bounds__(T) block_norm_kernel(const NormArgs a) {
    using S = RowSpan<T, V, VEC>;
    __shared__ float buf[2][32];
    __shared__ uint32_t ubuf[32];
    const float inv_c = 1.0f / static_cast<float>(a.C);
    const long long m = blockIdx.x;
    const size_t at = static_cast<size_t>(m) * a.C;
    pdl_launch_dependents();
    pdl_wait();
    uint32_t r[S::W];
    S::load(r, a.x + at, a.C);
    float rstd_y = 0.0f;
    if (a.y) {
        uint32_t y[S::W], w[S::W], g[S::W];
        S::load(y, a.y + at, a.C);
        if (a.post) {
            S::load(w, a.post, a.C);
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < S::E; ++e) ss = fmaf(S::get(y, e), S::get(y, e), ss);
            rstd_y = 1.0f / sqrtf(block_sum<T>(ss, buf[0]) * inv_c + a.eps);
        }
        if (a.gate_kind != kGateNone) S::load(g, a.gate + (a.gate_kind == kGateToken ? at : 0), a.C);
#pragma unroll
        for (int e = 0; e < S::E; ++e) {
            float t = S::get(y, e);
            if (a.post) t = t * rstd_y * (S::get(w, e) + a.off);
            if (a.gate_kind != kGateNone) t *= S::get(g, e);
            S::put(r, e, to_bf16_bits(fmaf(a.alpha, t, S::get(r, e))));
        }
        S::store(r, a.residual + at, a.C);
    }
    uint32_t w[S::W];
    S::load(w, a.pre, a.C);
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < S::E; ++e)
        if (S::col(e / VEC) < a.C) ss = fmaf(S::get(r, e), S::get(r, e), ss);
    const float rstd = 1.0f / sqrtf(block_sum<T>(ss, buf[1]) * inv_c + a.eps);
    if (a.rstd && threadIdx.x == 0) {
        a.rstd[m] = rstd_y;
        a.rstd[a.M + m] = rstd;
    }
    auto normed = [&](int e) { return S::get(r, e) * rstd * (S::get(w, e) + a.off); };
    if constexpr (!CODES) {
#pragma unroll
        for (int e = 0; e < S::E; ++e) S::put(r, e, to_bf16_bits(normed(e)));
        S::store(r, static_cast<uint16_t*>(a.normed) + at, a.C);
    } else {
        // columns past C hold zeros in r, so they are neutral here
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < S::E; ++e)
            if (S::col(e / VEC) < a.C) top = max(top, abs_bits(normed(e)));
        top = block_max_bits<T>(top, ubuf);
        const RowScale sc = row_scale(__uint_as_float(top));
        if (threadIdx.x == 0) a.scales[m] = sc.scale;
        int8_t* q = static_cast<int8_t*>(a.normed) + static_cast<size_t>(m) * a.ld;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = S::col(j);
            if (c < a.C) {
                if constexpr (VEC == 8) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = normed(8 * j + i);
                    *reinterpret_cast<uint2*>(q + c) = codes8(v, sc);
                } else {
                    q[c] = code1(normed(j), sc);
                }
            }
        }
    }
}

struct NormGradArgs {
    const uint16_t* dn;
    const uint16_t* dres;        // null: no gradient into the residual itself
    const uint16_t* r;
    const float* rstd;           // [2, M]
    const uint16_t* y;           // null: d_x and d_pre only
    const uint16_t* post;
    const uint16_t* gate;
    const uint16_t* pre;
    uint16_t* dx;
    uint16_t* dy;
    uint16_t* dgate_token;       // gate of its own for every token: its gradient
    float* part;                 // [sums][gridDim.x][C]: pre, post, gate per channel
    int M, C, gate_kind;
    float alpha, off;
};

// One block takes rows blockIdx.x, + gridDim.x, ...; a thread keeps the same
// columns throughout and with them the column sums of the weight gradients,
// in registers, or in shared memory (ACC_SMEM) where 1024 threads leave no
// room for them.
template <int T, int V, int VEC, bool ACC_SMEM>
__global__ void __launch_bounds__(T) block_norm_backward_kernel(const NormGradArgs a) {
    using S = RowSpan<T, V, VEC>;
    extern __shared__ float acc_smem[];     // [sums][E][T] with ACC_SMEM
    __shared__ float buf[4][32];
    const float inv_c = 1.0f / static_cast<float>(a.C);
    pdl_launch_dependents();
    pdl_wait();
    float acc_pre[ACC_SMEM ? 1 : S::E], acc_post[ACC_SMEM ? 1 : S::E], acc_gate[ACC_SMEM ? 1 : S::E];
    const bool post = a.post != nullptr, chan = a.gate_kind == kGateChannel;
#pragma unroll
    for (int e = 0; e < S::E; ++e) {
        if constexpr (ACC_SMEM) {
            acc_smem[e * T + threadIdx.x] = 0.0f;
            if (post) acc_smem[(S::E + e) * T + threadIdx.x] = 0.0f;
            if (chan) acc_smem[((post ? 2 : 1) * S::E + e) * T + threadIdx.x] = 0.0f;
        } else {
            acc_pre[e] = acc_post[e] = acc_gate[e] = 0.0f;
        }
    }
    auto add = [&](float (&reg)[ACC_SMEM ? 1 : S::E], int slot, int e, float v) {
        if constexpr (ACC_SMEM) acc_smem[(slot * S::E + e) * T + threadIdx.x] += v;
        else reg[e] += v;
    };
    uint32_t wpre[S::W];
    S::load(wpre, a.pre, a.C);
    int turn = 0;
    for (long long m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
        const size_t at = static_cast<size_t>(m) * a.C;
        uint32_t dn[S::W], r[S::W], y[S::W], ds[S::W];
        S::load(dn, a.dn + at, a.C);
        S::load(r, a.r + at, a.C);
        if (a.dres) S::load(ds, a.dres + at, a.C);
        if (a.y) S::load(y, a.y + at, a.C);
        const float rr = a.rstd[a.M + m];
        float s1 = 0.0f;
#pragma unroll
        for (int e = 0; e < S::E; ++e) {
            if (S::col(e / VEC) >= a.C) continue;
            const float xh = S::get(r, e) * rr, d = S::get(dn, e);
            add(acc_pre, 0, e, d * xh);
            s1 = fmaf(d * (S::get(wpre, e) + a.off), xh, s1);
        }
        s1 = block_sum<T>(s1, buf[2 * turn]) * inv_c;
        float dt[S::E];
#pragma unroll
        for (int e = 0; e < S::E; ++e) {
            const float xh = S::get(r, e) * rr, dh = S::get(dn, e) * (S::get(wpre, e) + a.off);
            float d = rr * (dh - xh * s1);
            if (a.dres) d += S::get(ds, e);
            S::put(r, e, to_bf16_bits(d));
            dt[e] = a.alpha * d;
        }
        S::store(r, a.dx + at, a.C);
        if (!a.y) continue;
        uint32_t wpost[S::W];
        const float ry = post ? a.rstd[m] : 1.0f;
        if (post) S::load(wpost, a.post, a.C);
        if (a.gate_kind != kGateNone) {
            uint32_t g[S::W];
            S::load(g, a.gate + (chan ? 0 : at), a.C);
            uint32_t dg[S::W];
#pragma unroll
            for (int e = 0; e < S::E; ++e) {
                float u = S::get(y, e);
                if (post) u = u * ry * (S::get(wpost, e) + a.off);
                if (chan) {
                    if (S::col(e / VEC) < a.C) add(acc_gate, post ? 2 : 1, e, dt[e] * u);
                } else {
                    S::put(dg, e, to_bf16_bits(dt[e] * u));
                }
                dt[e] *= S::get(g, e);
            }
            if (!chan) S::store(dg, a.dgate_token + at, a.C);
        }
        if (post) {
            float s2 = 0.0f;
#pragma unroll
            for (int e = 0; e < S::E; ++e) {
                if (S::col(e / VEC) >= a.C) continue;
                const float yh = S::get(y, e) * ry;
                add(acc_post, 1, e, dt[e] * yh);
                dt[e] *= S::get(wpost, e) + a.off;
                s2 = fmaf(dt[e], yh, s2);
            }
            s2 = block_sum<T>(s2, buf[2 * turn + 1]) * inv_c;
#pragma unroll
            for (int e = 0; e < S::E; ++e) dt[e] = ry * (dt[e] - S::get(y, e) * ry * s2);
        }
#pragma unroll
        for (int e = 0; e < S::E; ++e) S::put(y, e, to_bf16_bits(dt[e]));
        S::store(y, a.dy + at, a.C);
    }
    const size_t slab = static_cast<size_t>(gridDim.x) * a.C;
    float* p = a.part + static_cast<size_t>(blockIdx.x) * a.C;
#pragma unroll
    for (int e = 0; e < S::E; ++e) {
        const int c = S::col(e / VEC) + e % VEC;
        if (c < a.C) {
            if constexpr (ACC_SMEM) {
                p[c] = acc_smem[e * T + threadIdx.x];
                if (post) p[slab + c] = acc_smem[(S::E + e) * T + threadIdx.x];
                if (chan) p[(post ? 2 : 1) * slab + c] = acc_smem[((post ? 2 : 1) * S::E + e) * T + threadIdx.x];
            } else {
                p[c] = acc_pre[e];
                if (post) p[slab + c] = acc_post[e];
                if (chan) p[(post ? 2 : 1) * slab + c] = acc_gate[e];
            }
        }
    }
}

// out_k[c] = bf16(sum over the G partial rows of slab k), in a fixed order:
// warp w of a block takes rows w, w + 8, ... of 32 columns, then the warps'
// sums are added in order.
__global__ void __launch_bounds__(256) column_sums_kernel(const float* __restrict__ part, int G, int C,
                                                          uint16_t* o0, uint16_t* o1, uint16_t* o2) {
    __shared__ float s[8][32];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const float* p = part + static_cast<size_t>(blockIdx.y) * G * C;
    float v = 0.0f;
    if (c < C) {
#pragma unroll 8
        for (int g = warp; g < G; g += 8) v += p[static_cast<size_t>(g) * C + c];
    }
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < C) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += s[w][lane];
        uint16_t* o = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
        o[c] = to_bf16_bits(t);
    }
}

}  // namespace w4
