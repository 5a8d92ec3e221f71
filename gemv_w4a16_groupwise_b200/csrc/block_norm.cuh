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
// A row is read from device memory once; what a reduction separates stays in
// registers as bf16 or is read again from shared memory.  Sums and statistics
// are fp32 in a fixed order.  Measured on 4096 x 4096 with a post norm and a
// gate per token: forward 28.5 us (5.9 TB/s, bound by memory), backward with its
// column sums 56.5 us (4.8 TB/s, bound by issue slots and the latency of a row's
// reductions; 53.0 and 7.5 when the second kernel starts after the first).
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

// A block walks over rows blockIdx.x, + gridDim.x, ... with the next row's
// loads under way while it works on one.  The values are worked on in pairs
// (f32x2): with scalar arithmetic and predicated sums the kernel was bound by
// the instructions it issued, not by memory.  rsqrtf is within 2 ulp, less than
// the sum under it is.
template <int T, int G, int VEC, bool CODES>
__global__ void __launch_bounds__(T, 1024 / T) block_norm_kernel(const NormArgs a) {
    using S = RowSpan<T, G, VEC>;
    extern __shared__ uint4 ring[];
    __shared__ __align__(16) float buf[2][2][32];      // [row's parity][reduction]
    __shared__ __align__(16) uint32_t ubuf[2][32];
    const float inv_c = 1.0f / static_cast<float>(a.C);
    const bool post = a.post != nullptr, token = a.gate_kind == kGateToken, gated = a.gate_kind != kGateNone;
    const S span(blockIdx.x, a.C);
    const RowPipe<T, G, VEC, true> pipe = {ring, 1 + (a.y ? 1 : 0) + (token ? 1 : 0), span};
    pdl_launch_dependents();
    pdl_wait();
    auto fetch = [&](int stage, long long m) {
        const int C = fresh(a.C);
        const size_t at = static_cast<size_t>(m) * C;
        pipe.fetch(stage, 0, a.x + at, C);
        if (a.y) pipe.fetch(stage, 1, a.y + at, C);
        if (token) pipe.fetch(stage, 2, a.gate + at, C);
        pipe.commit();
    };
    fetch(0, blockIdx.x);
    const float2 off = both(a.off);
    uint4 wpre[G];
#pragma unroll
    for (int g = 0; g < G; ++g) wpre[g] = span.load_vector(a.pre, g, a.C);
    int turn = 0;
    for (long long m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
        const int C = VEC == 8 ? a.C : fresh(a.C);
        const size_t at = static_cast<size_t>(m) * C;
        const bool more = m + gridDim.x < a.M;
        if (more) fetch(turn ^ 1, m + gridDim.x);
        pipe.wait(more);
        float rstd_y = 0.0f;
        if (post) {
            float2 ss = both(0.0f);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint4 y = pipe.read(turn, 1, a.y + at, g, C);
                for (uint32_t w : {y.x, y.y, y.z, y.w}) {
                    const float2 v = unpack_bf16x2(w);
                    ss = ffma2(v, v, ss);
                }
            }
            rstd_y = rsqrtf(block_sum<T>(ss, buf[turn][0]) * inv_c + a.eps);
        }
        uint32_t r[G][4];
        float2 ss = both(0.0f);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const uint4 x = pipe.read(turn, 0, a.x + at, g, C);
            r[g][0] = x.x, r[g][1] = x.y, r[g][2] = x.z, r[g][3] = x.w;
            if (a.y) {
                const uint4 y = pipe.read(turn, 1, a.y + at, g, C);
                float2 t[4] = {unpack_bf16x2(y.x), unpack_bf16x2(y.y), unpack_bf16x2(y.z), unpack_bf16x2(y.w)};
                if (post) {
                    const uint4 p = span.load_vector(a.post, g, C);
                    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        t[i] = fmul2(fmul2(t[i], both(rstd_y)), fadd2(unpack_bf16x2(w[i]), off));
                }
                if (gated) {
                    const uint4 p = token ? pipe.read(turn, 2, a.gate + at, g, C) : span.load_vector(a.gate, g, C);
                    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) t[i] = fmul2(t[i], unpack_bf16x2(w[i]));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) r[g][i] = pack_bf16x2(ffma2(both(a.alpha), t[i], unpack_bf16x2(r[g][i])));
                span.store(a.residual + at, g, C, r[g]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = unpack_bf16x2(r[g][i]);
                ss = ffma2(v, v, ss);
            }
        }
        const float rstd = rsqrtf(block_sum<T>(ss, buf[turn][1]) * inv_c + a.eps);
        if (a.rstd && threadIdx.x == 0) {
            a.rstd[m] = rstd_y;
            a.rstd[a.M + m] = rstd;
        }
        float2 n[G][4];
        float top = 0.0f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const uint32_t w[4] = {wpre[g].x, wpre[g].y, wpre[g].z, wpre[g].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                n[g][i] = fmul2(fmul2(unpack_bf16x2(r[g][i]), both(rstd)), fadd2(unpack_bf16x2(w[i]), off));
                if constexpr (CODES) top = max_abs(top, n[g][i]);
                else r[g][i] = pack_bf16x2(n[g][i]);
            }
            if constexpr (!CODES) span.store(static_cast<uint16_t*>(a.normed) + at, g, C, r[g]);
        }
        if constexpr (CODES) {
            top = __uint_as_float(block_max_bits<T>(__float_as_uint(top), ubuf[turn]));
            const RowCodes sc = row_codes<false>(top);
            if (threadIdx.x == 0) a.scales[m] = row_scale(top);
#pragma unroll
            for (int g = 0; g < G; ++g)
                store_codes<VEC>(span, static_cast<int8_t*>(a.normed) + static_cast<size_t>(m) * a.ld, g, C,
                                    codes8<false>(n[g], sc));
        }
    }
}

// Floats from one block's partial sums to the next: whole 16 bytes.
__host__ __device__ constexpr int partial_stride(int C) { return (C + 3) & ~3; }

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
    float* part;                 // [sums][gridDim.x][partial_stride(C)]: pre, post, gate per channel
    int M, C, gate_kind;
    float alpha, off;
};

// Blocks an SM holds: 512 threads' worth at two groups (128 registers each)
// and in rows of words, 1024 at one group of whole 16 bytes (64; with 768 of 80,
// 8192 x 1024 took 44 us instead of 39).  Words need more registers for their
// columns: with 1024 threads they spilled 136 bytes each way (513 x 2047 13.7 us
// against 12.2, 300 x 1001 11.2 against 7.9, 4096 x 2047 with token gates 64.5
// against 57.3); with 768 they spill 24, which is better for some (8192 x 2047
// 97.9 against 105.7) and worse for others (4096 x 2047 73.2, 513 x 2047 13.9).
__host__ __device__ constexpr int norm_grad_blocks_per_sm(int T, int G, int VEC) {
    return T == 1024 ? 1 : G == 2 || VEC == 2 ? 512 / T : 1024 / T;
}

// One block takes rows blockIdx.x, + gridDim.x, ...; a thread keeps the same
// columns throughout and with them the column sums of the weight gradients,
// in registers, or in shared memory (ACC_SMEM, then without the row pipe)
// where 1024 threads leave no room for them.  What a reduction separates is
// read again from the pipe instead of being held.
template <int T, int G, int VEC, bool ACC_SMEM>
__global__ void __launch_bounds__(T, norm_grad_blocks_per_sm(T, G, VEC)) block_norm_backward_kernel(const NormGradArgs a) {
    using S = RowSpan<T, G, VEC>;
    constexpr bool PIPED = !ACC_SMEM;
    constexpr int kRegs = ACC_SMEM ? 1 : G;
    extern __shared__ uint4 dyn_smem[];     // the row pipe; with ACC_SMEM the sums, [sums][G][4][T]
    float2* acc_smem = reinterpret_cast<float2*>(dyn_smem);
    __shared__ __align__(16) float buf[2][2][32];
    const float inv_c = 1.0f / static_cast<float>(a.C);
    const bool post = a.post != nullptr, chan = a.gate_kind == kGateChannel, token = a.gate_kind == kGateToken;
    pdl_launch_dependents();
    pdl_wait();
    float2 acc_pre[kRegs][4], acc_post[kRegs][4], acc_gate[kRegs][4];
    const int sums = 1 + (post ? 1 : 0) + (chan ? 1 : 0);
    if constexpr (ACC_SMEM) {
        for (int e = 0; e < sums * G * 4; ++e) acc_smem[e * T + threadIdx.x] = both(0.0f);
    } else {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc_pre[g][i] = acc_post[g][i] = acc_gate[g][i] = both(0.0f);
    }
    auto add = [&](float2 (&reg)[kRegs][4], int slab, int g, int i, float2 x, float2 y) {
        if constexpr (ACC_SMEM) {
            float2& s = acc_smem[((slab * G + g) * 4 + i) * T + threadIdx.x];
            s = ffma2(x, y, s);
        } else {
            reg[g][i] = ffma2(x, y, reg[g][i]);
        }
    };
    const int dres_at = 2, y_at = 2 + (a.dres ? 1 : 0), gate_at = y_at + (a.y ? 1 : 0);
    const S span(blockIdx.x, a.C);
    const RowPipe<T, G, VEC, PIPED> pipe = {dyn_smem, gate_at + (token ? 1 : 0), span};
    auto fetch = [&](int stage, long long m) {
        const int C = fresh(a.C);
        const size_t at = static_cast<size_t>(m) * C;
        pipe.fetch(stage, 0, a.dn + at, C);
        pipe.fetch(stage, 1, a.r + at, C);
        if (a.dres) pipe.fetch(stage, dres_at, a.dres + at, C);
        if (a.y) pipe.fetch(stage, y_at, a.y + at, C);
        if (token) pipe.fetch(stage, gate_at, a.gate + at, C);
        pipe.commit();
    };
    auto words = [](uint4 v, uint32_t (&w)[4]) { w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w; };
    fetch(0, blockIdx.x);
    float next_rr = a.rstd[a.M + blockIdx.x], next_ry = post ? a.rstd[blockIdx.x] : 1.0f;
    const float2 off = both(a.off);
    int turn = 0;
    for (long long m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
        const int C = VEC == 8 ? a.C : fresh(a.C);
        const size_t at = static_cast<size_t>(m) * C;
        const bool more = m + gridDim.x < a.M;
        const float2 rr = both(next_rr), ry = both(next_ry);
        if (more) {
            fetch(turn ^ 1, m + gridDim.x);
            next_rr = a.rstd[a.M + m + gridDim.x];
            if (post) next_ry = a.rstd[m + gridDim.x];
        }
        pipe.wait(more);
        float2 s = both(0.0f);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            uint32_t dn[4], r[4], w[4];
            words(pipe.read(turn, 0, a.dn + at, g, C), dn);
            words(pipe.read(turn, 1, a.r + at, g, C), r);
            words(span.load_vector(a.pre, g, C), w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 xh = fmul2(unpack_bf16x2(r[i]), rr), d = unpack_bf16x2(dn[i]);
                add(acc_pre, 0, g, i, d, xh);
                s = ffma2(fmul2(d, fadd2(unpack_bf16x2(w[i]), off)), xh, s);
            }
        }
        // mean(dh xh) rstd, negated: d_r = rstd (dh - xh mean) is fma(xh, it, dh rstd)
        const float2 c1 = both(-block_sum<T>(s, buf[turn][0]) * inv_c * rr.x);
        float2 dt[G][4];
        s = both(0.0f);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            uint32_t dn[4], r[4], w[4], dx[4];
            words(pipe.read(turn, 0, a.dn + at, g, C), dn);
            words(pipe.read(turn, 1, a.r + at, g, C), r);
            words(span.load_vector(a.pre, g, C), w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 xh = fmul2(unpack_bf16x2(r[i]), rr);
                const float2 dh = fmul2(unpack_bf16x2(dn[i]), fadd2(unpack_bf16x2(w[i]), off));
                dt[g][i] = ffma2(xh, c1, fmul2(dh, rr));
            }
            if (a.dres) {
                words(pipe.read(turn, dres_at, a.dres + at, g, C), w);
#pragma unroll
                for (int i = 0; i < 4; ++i) dt[g][i] = fadd2(dt[g][i], unpack_bf16x2(w[i]));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) dx[i] = pack_bf16x2(dt[g][i]);
            span.store(a.dx + at, g, C, dx);
            if (!a.y) continue;
            uint32_t y[4], p[4];
            words(pipe.read(turn, y_at, a.y + at, g, C), y);
            if (post) words(span.load_vector(a.post, g, C), p);
#pragma unroll
            for (int i = 0; i < 4; ++i) dt[g][i] = fmul2(dt[g][i], both(a.alpha));
            if (chan || token) {
                words(token ? pipe.read(turn, gate_at, a.gate + at, g, C) : span.load_vector(a.gate, g, C), w);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float2 u = unpack_bf16x2(y[i]);
                    if (post) u = fmul2(fmul2(u, ry), fadd2(unpack_bf16x2(p[i]), off));
                    if (chan) add(acc_gate, post ? 2 : 1, g, i, dt[g][i], u);
                    else dx[i] = pack_bf16x2(fmul2(dt[g][i], u));
                    dt[g][i] = fmul2(dt[g][i], unpack_bf16x2(w[i]));
                }
                if (token) span.store(a.dgate_token + at, g, C, dx);
            }
            if (post) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 yh = fmul2(unpack_bf16x2(y[i]), ry);
                    add(acc_post, 1, g, i, dt[g][i], yh);
                    dt[g][i] = fmul2(dt[g][i], fadd2(unpack_bf16x2(p[i]), off));
                    s = ffma2(dt[g][i], yh, s);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) dx[i] = pack_bf16x2(dt[g][i]);
                span.store(a.dy + at, g, C, dx);
            }
        }
        if (!post) continue;
        const float2 c2 = both(-block_sum<T>(s, buf[turn][1]) * inv_c * ry.x);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            uint32_t y[4];
            words(pipe.read(turn, y_at, a.y + at, g, C), y);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[i] = pack_bf16x2(ffma2(fmul2(unpack_bf16x2(y[i]), ry), c2, fmul2(dt[g][i], ry)));
            span.store(a.dy + at, g, C, y);
        }
    }
    const size_t slab = static_cast<size_t>(gridDim.x) * partial_stride(a.C);
    float* p = a.part + static_cast<size_t>(blockIdx.x) * partial_stride(a.C);
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 v[3];
            if constexpr (ACC_SMEM) {
                for (int k = 0; k < sums; ++k) v[k] = acc_smem[((k * G + g) * 4 + i) * T + threadIdx.x];
            } else {
                v[0] = acc_pre[g][i];
                v[1] = post ? acc_post[g][i] : acc_gate[g][i];
                v[2] = acc_gate[g][i];
            }
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (k < sums) {
                    const int c = span.col(g, 2 * i);
                    if (VEC == 8) {      // c < C says the whole group is inside
                        if (c < a.C) *reinterpret_cast<float2*>(p + k * slab + c) = v[k];
                    } else {
                        if (c >= 0 && c < a.C) p[k * slab + c] = v[k].x;
                        if (c + 1 < a.C) p[k * slab + c + 1] = v[k].y;
                    }
                }
        }
}

// out_k[c] = bf16(sum over the rows of slab k of the blocks' partial sums), in
// a fixed order: a block takes 32 columns, its WARPS warps 4 rows each at a time
// (8 lanes x 4 columns a row); a warp adds its 4 rows by shuffles, then the
// warps' sums are added in order.  Bound by latency: 16 warps halve the loads
// that a thread makes one after the other (8192 x 1024 backward: 39 -> 34 us);
// for a few dozen rows 8 are enough, and quicker to start (64 x 1024: 5.5
// against 7.4 us).
template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS) column_sums_kernel(const float* __restrict__ part, int rows, int C,
                                                                uint16_t* o0, uint16_t* o1, uint16_t* o2) {
    __shared__ float4 s[WARPS][8];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const size_t stride = partial_stride(C);
    const float* p = part + static_cast<size_t>(blockIdx.y) * rows * stride;
    const int quad = blockIdx.x * 32 + (lane & 7) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (quad < C) {                   // columns behind C are read and dropped
#pragma unroll 8
        for (int r = warp * 4 + (lane >> 3); r < rows; r += 4 * WARPS) {
            const float4 u = *reinterpret_cast<const float4*>(p + r * stride + quad);
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
        }
    }
#pragma unroll
    for (int o = 8; o <= 16; o <<= 1) {
        v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
        v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
        v.z += __shfl_xor_sync(0xFFFFFFFFu, v.z, o);
        v.w += __shfl_xor_sync(0xFFFFFFFFu, v.w, o);
    }
    if (lane < 8) s[warp][lane] = v;
    __syncthreads();
    const int c = blockIdx.x * 32 + lane;
    if (warp == 0 && c < C) {
        const float* sums = reinterpret_cast<const float*>(s);
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) t += sums[w * 32 + lane];
        uint16_t* o = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
        o[c] = to_bf16_bits(t);
    }
}

}  // namespace w4
