// 8-bit product on the tensor cores: TMA -> tcgen05.mma kind::i8 by CTA pairs
// -> int32 in tensor memory -> scales, bias, bf16.
//
//     forward     D[n, m] = sum_k w[n, k] a[m, k]      weights K-major
//     transposed  D[k, m] = sum_n w[n, k] a[m, n]      weights MN-major, as they lie
//
// The weights take the MMA's 256-row side (128 rows in each CTA of the pair)
// and the tokens its column side, TN in {32, 64, 128, 256}: one kernel serves
// a few dozen tokens and thousands.  A stage holds 128 of the reduction: the
// CTA's 16 KB of weights and its half of the token tile (TN / 2 rows); with
// pairs an SM fetches 32 KB for 256 x 256 x 128 / 2 products instead of the 48
// of a 128 x 256 tile of its own, and it is the fetch from L2 that a wider
// tile on one SM would wait for.
//
// Persistent: pair p takes whole tiles p, p + P, ... below F, then a share of
// the remaining tiles' reduction slices, cut evenly over the pairs across tile
// borders.  A tile cut that way leaves int32 partials (exact, so their order
// does not matter) which w8_finalize_kernel adds, scales and rounds.
//
// Warps: 0 TMA producer, 1 MMA issuer (in the pair's first CTA), 2..9
// epilogue.  Accumulators are double buffered, so a tile's epilogue runs
// beside the next tile's products.  Full barriers live in the first CTA and
// count both CTAs' bytes; the stage's release and the accumulator's
// completion are committed to both.
//
// Measured: 2048 x 28672 x 4096 in 151 us (3.2 PFLOP/s, tensor pipe busy 93 %
// of the SMs' active cycles, 83 % of the launch), bound by the products; 33 x 28672 x 4096 in 22.3 us
// (5.3 TB/s), bound by the weights' bytes; a call with one stage per tile in
// 4.6 to 6.5 us, bound by its own latency.
#pragma once

#include "gemm_tc.cuh"
#include "tma.cuh"
#include "w8_gemm.cuh"

namespace w4 {

constexpr int kW8Rows = 256;          // outputs of a pair's tile
constexpr int kW8Red = 128;           // reduction of a stage
constexpr int kW8ABytes = 128 * kW8Red;
constexpr int kW8EpiWarps = 8;
constexpr int kW8Threads = 64 + 32 * kW8EpiWarps;
// An epilogue warp stages 32 outputs of 16 token pairs, the pairs 36 words
// apart (two pairs' 16-byte reads then meet no bank twice), and its tokens' scales.
constexpr int kW8PairStride = 36;
constexpr int kW8EpiWarpBytes = 16 * kW8PairStride * 4 + 128 * 4;
constexpr int kW8EpiBytes = kW8EpiWarps * kW8EpiWarpBytes;
__host__ __device__ constexpr int w8_stage_bytes(int TN) { return kW8ABytes + TN / 2 * kW8Red; }

struct W8TcArgs {
    W8Args p;
    int32_t* part;       // [2 pairs][TN][256] partial tiles
    int tiles_m, tiles;  // token tiles, tiles in all (token tiles fastest)
    uint32_t inv_tiles_m;     // floor(2^32 / tiles_m) + 1 (tiles_m > 1): exact quotients of pair numbers
    int step_m, step_o;  // from a tile to the one `pairs` on
    int F;               // tiles below F are whole units
    int chunks;          // stages of one tile
    int cut_pairs;       // pairs that share the tiles from F on
    int stages;
    int early;           // the kernel before does not write the weights
    int withhold;        // a test's tile before which the producers stop, or -1 (a test for every stage
                         // took 0.9 us of 33 x 28672 x 4096)
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t first_cta_addr(const void* p) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}
// The form without .aligned counts threads, so it holds for a warp whose lanes
// arrive apart.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
// The producer and the MMA issuer run as whole warps whose lanes hold the same
// operands, with one elected lane issuing: the operands then sit in uniform
// registers, where these instructions take them from.  Issued from a branch of
// one lane, moving them there took 320 cycles for a stage's four MMAs and as
// much for its two copies, and a stage 600 cycles whatever its tile.

// One 2-D load into this CTA's shared memory that completes on the barrier
// `bar` of the pair's first CTA; with `expect` that CTA's barrier (its own, at
// local_bar) is armed first for that many bytes.
__device__ __forceinline__ void tma_pair_elected(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar,
                                                 uint32_t local_bar, uint32_t expect) {
    asm volatile(
        "{\n .reg .pred P, L;\n elect.sync _|P, 0xffffffff;\n setp.ne.and.u32 L, %6, 0, P;\n"
        " @L mbarrier.arrive.expect_tx.shared::cta.b64 _, [%5], %6;\n"
        " @P cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "r"(local_bar), "r"(expect)
        : "memory");
}
// The four MMAs of a stage (128 of the reduction), with descriptors `astep`
// and 2 sixteen-byte units apart, and the release of the stage (`empty`) in
// both CTAs once they are done.  `accumulate` = 0: the first overwrites.
__device__ __forceinline__ void umma_i8_stage_elected(uint32_t d, uint64_t adesc, uint64_t bdesc, uint64_t astep,
                                                      uint32_t idesc, uint32_t accumulate, uint32_t empty) {
    asm volatile(
        "{\n .reg .pred P, p;\n .reg .b64 a, b;\n .reg .b16 m;\n"
        " elect.sync _|P, 0xffffffff;\n setp.ne.b32 p, %5, 0;\n mov.b16 m, 3;\n"
        " @P tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %4, p;\n"
        " setp.eq.b32 p, 0, 0;\n"
        " add.s64 a, %1, %3;\n add.s64 b, %2, 2;\n"
        " @P tcgen05.mma.cta_group::2.kind::i8 [%0], a, b, %4, p;\n"
        " add.s64 a, a, %3;\n add.s64 b, b, 2;\n"
        " @P tcgen05.mma.cta_group::2.kind::i8 [%0], a, b, %4, p;\n"
        " add.s64 a, a, %3;\n add.s64 b, b, 2;\n"
        " @P tcgen05.mma.cta_group::2.kind::i8 [%0], a, b, %4, p;\n"
        " @P tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%6], m;\n}\n" ::"r"(
            d),
        "l"(adesc), "l"(bdesc), "l"(astep), "r"(idesc), "r"(accumulate), "r"(empty)
        : "memory");
}
// Arrive on the barrier at this offset in both CTAs once the MMAs before are done.
__device__ __forceinline__ void umma_commit_pair_elected(uint32_t bar) {
    asm volatile(
        "{\n .reg .pred P;\n .reg .b16 m;\n elect.sync _|P, 0xffffffff;\n mov.b16 m, 3;\n"
        " @P tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}\n" ::"r"(
            bar)
        : "memory");
}
// mbar_wait_bounded by a whole warp, with one answer.
__device__ __forceinline__ bool warp_wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort,
                                                  unsigned int err) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, abort, err));
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Instruction descriptor: s8 x s8 -> s32, M = 256 over the pair, N = TN.
__host__ __device__ constexpr uint32_t umma_idesc_i8(int TN, bool a_mn_major) {
    return (2u << 4)                              // D format s32
           | (1u << 7)                            // A format s8
           | (1u << 10)                           // B format s8
           | ((a_mn_major ? 1u : 0u) << 15)       // A major
           | (static_cast<uint32_t>(TN >> 3) << 17)
           | (static_cast<uint32_t>(kW8Rows >> 4) << 24);
}

// The units of pair p of P, in order (no division on the way to the first one:
// 1 % of a short call).
struct W8Unit {
    int mt, ot;          // token tile, output tile
    int kb0, kb1;        // its stages
    int part;            // slot of the partial tile, or -1 for a whole tile
};
struct W8Walk {
    int t, mt, ot;       // the next whole tile
    uint32_t c, c1;      // the pair's share of the cut tiles' stages (pairs^2 x at most 2^10 stages: 32 bits up to 2047 pairs)
    int cut_units;
    __device__ __forceinline__ W8Walk(const W8TcArgs& a, int pair) {
        t = pair;
        ot = a.tiles_m == 1 ? pair : static_cast<int>(__umulhi(pair, a.inv_tiles_m));
        mt = pair - ot * a.tiles_m;
        c = c1 = 0;
        cut_units = 0;
        if (a.F < a.tiles && pair < a.cut_pairs) {
            const uint32_t total = static_cast<uint32_t>(a.tiles - a.F) * a.chunks;
            c = total * pair / a.cut_pairs;
            c1 = total * (pair + 1) / a.cut_pairs;
        }
    }
    __device__ __forceinline__ bool next(const W8TcArgs& a, int pair, int pairs, W8Unit* u) {
        if (t < a.F) {
            *u = W8Unit{mt, ot, 0, a.chunks, -1};
            t += pairs;
            mt += a.step_m;
            ot += a.step_o;
            if (mt >= a.tiles_m) {
                mt -= a.tiles_m;
                ++ot;
            }
            return true;
        }
        if (c >= c1) return false;
        const int tile = static_cast<int>(c / a.chunks);
        u->mt = (a.F + tile) % a.tiles_m;
        u->ot = (a.F + tile) / a.tiles_m;
        u->kb0 = static_cast<int>(c) - tile * a.chunks;
        u->kb1 = min(a.chunks, u->kb0 + static_cast<int>(c1 - c));
        u->part = (u->kb0 == 0 && u->kb1 == a.chunks) ? -1 : 2 * pair + (cut_units > 0 ? 1 : 0);
        ++cut_units;
        c += u->kb1 - u->kb0;
        return true;
    }
};

template <bool TR, int TN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kW8Threads, 1)
    w8_gemm_tc_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap,
                      const W8TcArgs a) {
    static_assert(TN == 32 || TN == 64 || TN == 128 || TN == 256, "TN");
    constexpr int kStageBytes = w8_stage_bytes(TN);
    constexpr uint32_t kTmemCols = 2 * TN;
    constexpr uint32_t kIdesc = umma_idesc_i8(TN, TR);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int NS = a.stages;
    uint8_t* epi = base + NS * kStageBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(epi + kW8EpiBytes);
    uint64_t* empty = full + NS;
    uint64_t* acc_full = empty + NS;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int out = TR ? a.p.K : a.p.N;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&wmap);
        tma_prefetch_desc(&amap);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * kW8EpiWarps);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    __syncwarp();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();        // both CTAs' barriers stand before either uses them
    tc_fence_after();
    const uint32_t tmem_d = *tmem_slot;
    pdl_launch_dependents();

    W8Walk walk(a, pair);
    W8Unit u;
    const uint32_t stage0 = smem_u32(base), full0 = smem_u32(full), empty0 = smem_u32(empty);
    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        const uint32_t full_first = first_cta_addr(full);
        const uint32_t expect = rank == 0 ? 2 * kStageBytes : 0;
        auto load_weights = [&](int s, int kb, int o0) {
            tma_pair_elected(stage0 + s * kStageBytes, &wmap, TR ? o0 : kb * kW8Red, TR ? kb * kW8Red : o0,
                             full_first + 8 * s, full0 + 8 * s, expect);
        };
        int s = 0;
        uint32_t round = 0;
        bool ok = true;
        // Weights that no kernel still running writes (a.early) are asked for
        // before the tokens' codes are waited for: the first NS stages.
        int early = 0;
        if (a.early) {
            W8Walk ahead(a, pair);
            while (early < NS && ahead.next(a, pair, pairs, &u)) {
                const int o0 = u.ot * kW8Rows + static_cast<int>(rank) * 128;
                for (int kb = u.kb0; kb < u.kb1 && early < NS; ++kb, ++early) load_weights(early, kb, o0);
            }
        }
        pdl_wait();
        int n = 0, units = 0;
        while (ok && walk.next(a, pair, pairs, &u) && units++ != a.withhold) {
            const int m0 = u.mt * TN + static_cast<int>(rank) * (TN / 2);
            const int o0 = u.ot * kW8Rows + static_cast<int>(rank) * 128;
            for (int kb = u.kb0; kb < u.kb1; ++kb, ++n) {
                if (round > 0 && !warp_wait_bounded(&empty[s], (round - 1) & 1u, abort_flag, kErrTimeoutEmpty)) {
                    ok = false;
                    break;
                }
                if (n >= early) load_weights(s, kb, o0);
                tma_pair_elected(stage0 + s * kStageBytes + kW8ABytes, &amap, kb * kW8Red, m0, full_first + 8 * s,
                                 full0 + 8 * s, 0);
                if (++s == NS) {
                    s = 0;
                    ++round;
                }
            }
        }
        // the releases of the stages still in use come from the other CTA:
        // see them in before this one may leave
        for (int j = 0; j < NS && ok; ++j) {
            if (round > 0) ok = warp_wait_bounded(&empty[s], (round - 1) & 1u, abort_flag, kErrTimeoutEmpty);
            if (++s == NS) {
                s = 0;
                ++round;
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        if (rank == 0) {
            // MN-major: 32 reduction rows are four groups of 8 rows, 1024 bytes each
            const uint64_t adesc0 = TR ? umma_desc_sw128(stage0, kW8ABytes, 1024) : umma_desc_sw128(stage0, 16, 1024);
            const uint64_t bdesc0 = umma_desc_sw128(stage0 + kW8ABytes, 16, 1024);
            bool ok = true;
            int s = 0, i = 0;
            uint32_t phase = 0;
            while (ok && walk.next(a, pair, pairs, &u)) {
                const int buf = i & 1;
                if (i >= 2) ok = warp_wait_bounded(&acc_empty[buf], ((i >> 1) - 1) & 1u, abort_flag, kErrTimeoutAccum);
                if (!ok) break;
                tc_fence_after();
                for (int kb = u.kb0; kb < u.kb1; ++kb) {
                    ok = warp_wait_bounded(&full[s], phase, abort_flag, kErrTimeoutTmaFull);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t at = static_cast<uint64_t>(s * (kStageBytes >> 4));
                    umma_i8_stage_elected(tmem_d + static_cast<uint32_t>(buf) * TN, adesc0 + at, bdesc0 + at,
                                          TR ? 4096 >> 4 : 32 >> 4, kIdesc, kb != u.kb0 ? 1u : 0u, empty0 + 8 * s);
                    if (++s == NS) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
                // An unfinished tile is not handed on: the other CTA's epilogue does not see
                // this one's abort flag and would store it.  Its wait runs out as this one did.
                if (!ok) break;
                umma_commit_pair_elected(smem_u32(&acc_full[buf]));
                ++i;
            }
        }
    } else {
        // ------------------------------------------------ epilogue
        // Two warps per quadrant of 32 TMEM lanes (outputs), each on half of
        // the tile's tokens, 32 at a time.
        const int q = warp & 3;                 // TMEM lanes 32 q .. 32 q + 31
        const int half = (warp - 2) >> 2;
        constexpr int kBlocks = TN >= 64 ? TN / 64 : 1;
        const int cbase = half * kBlocks * 32;  // TN = 32: the second half has nothing
        uint32_t* stage = reinterpret_cast<uint32_t*>(epi) + (warp - 2) * 16 * kW8PairStride;
        float* scales = reinterpret_cast<float*>(epi + kW8EpiWarps * 16 * kW8PairStride * 4) + (warp - 2) * 128;
        int i = 0;
        pdl_wait();
        while (walk.next(a, pair, pairs, &u)) {
            const int buf = i & 1;
            const int m0 = u.mt * TN + cbase;
            const int row = static_cast<int>(rank) * 128 + 32 * q + lane;      // in the tile
            const int o0 = u.ot * kW8Rows;
            const int o = o0 + row;
            const bool ov = o < out;
            // scales and bias come in while the products still run
            const float ws = (!TR && ov) ? a.p.w_scales[o] : 1.0f;
            const float bias = (a.p.bias && ov) ? bf16_bits_to_float(a.p.bias[o]) : 0.0f;
            const int tokens = cbase < TN ? min(kBlocks * 32, a.p.M - m0) : 0;
            __syncwarp();
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
                scales[32 * b + lane] = 32 * b + lane < tokens ? a.p.a_scales[m0 + 32 * b + lane] : 0.0f;
            const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&acc_full[buf], (i >> 1) & 1u, abort_flag,
                                                                      kErrTimeoutAccum));
            if (__any_sync(0xFFFFFFFFu, !ok || *abort_flag)) break;
            tc_fence_after();
            const uint32_t acc =
                tmem_d + static_cast<uint32_t>(buf * TN + cbase) + (static_cast<uint32_t>(32 * q) << 16);
#pragma unroll 1
            for (int b = 0; 32 * b < tokens; ++b) {
                uint32_t r[32];
                __syncwarp();
                tmem_ld_x32(acc + static_cast<uint32_t>(32 * b), r);
                if (u.part >= 0) {
                    int32_t* pt = a.part + (static_cast<size_t>(u.part) * TN + cbase + 32 * b) * kW8Rows + row;
#pragma unroll
                    for (int e = 0; e < 32; ++e) pt[e * kW8Rows] = static_cast<int32_t>(r[e]);
                    continue;
                }
                // pairs of tokens as bf16x2
                uint32_t y[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float2 sc = *reinterpret_cast<const float2*>(scales + 32 * b + 2 * e);
                    y[e] = bf162_bits(__floats2bfloat162_rn(
                        fmaf(static_cast<float>(static_cast<int>(r[2 * e])), sc.x * ws, bias),
                        fmaf(static_cast<float>(static_cast<int>(r[2 * e + 1])), sc.y * ws, bias)));
                }
                const int mb = m0 + 32 * b;
                if ((out & 7) == 0) {
                    // through shared memory: [token pair][output], then 8 outputs of two tokens a lane
#pragma unroll
                    for (int e = 0; e < 16; ++e) stage[e * kW8PairStride + lane] = y[e];
                    __syncwarp();
                    const int ol = o0 + static_cast<int>(rank) * 128 + 32 * q + (lane & 3) * 8;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const int pr = g * 8 + (lane >> 2), m = mb + 2 * pr;
                        const uint32_t* src = stage + pr * kW8PairStride + (lane & 3) * 8;
                        const uint4 v0 = *reinterpret_cast<const uint4*>(src);
                        const uint4 v1 = *reinterpret_cast<const uint4*>(src + 4);
                        uint16_t* dst = a.p.Y + static_cast<size_t>(m) * out + ol;
                        if (m < a.p.M && ol < out)
                            *reinterpret_cast<uint4*>(dst) =
                                make_uint4(prmt(v0.x, v0.y, 0x5410u), prmt(v0.z, v0.w, 0x5410u),
                                           prmt(v1.x, v1.y, 0x5410u), prmt(v1.z, v1.w, 0x5410u));
                        if (m + 1 < a.p.M && ol < out)
                            *reinterpret_cast<uint4*>(dst + out) =
                                make_uint4(prmt(v0.x, v0.y, 0x7632u), prmt(v0.z, v0.w, 0x7632u),
                                           prmt(v1.x, v1.y, 0x7632u), prmt(v1.z, v1.w, 0x7632u));
                    }
                } else {
                    // rows of Y that are not whole 16 bytes: 32 outputs of a token, 2 bytes a lane (put
                    // together to 16-byte stores by four warps, 777 x 4099 x 1001 took 13.0 us instead of 10.2)
                    uint16_t* dst = a.p.Y + static_cast<size_t>(mb) * out + o;
                    const int left = ov ? a.p.M - mb : 0;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        if (2 * e < left) *dst = static_cast<uint16_t>(y[e]);
                        dst += out;
                        if (2 * e + 1 < left) *dst = static_cast<uint16_t>(y[e] >> 16);
                        dst += out;
                    }
                }
            }
            // this warp's reads of the buffer are complete
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(first_cta_addr(&acc_empty[buf]));
            ++i;
        }
    }

    // The collective instructions below take whole warps: a deallocation that
    // each part of a split warp issued would free the tensor memory of whatever
    // runs on the SM next.
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {
        // a role gave up: let copies and mma already issued land (bounded)
        // before the tensor memory and the CTAs' shared memory are released
        const unsigned long long t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {
        }
    }
    cluster_sync();        // neither CTA leaves while the other may still reach into it
    __syncwarp();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_d), "r"(kTmemCols) : "memory");
    }
}

// The cut tiles: Y = bf16(sum of the partials * scales + bias).  One thread per
// token and four outputs, blocks (x, y): 256 threads of tile F + y; a tile that
// one pair computed whole is already stored.  The pair whose share
// [total p / P, total (p + 1) / P) holds stage c is ((c + 1) P - 1) / total.
// Bound by its reads from L2; with the share's arithmetic in 64 bits and per
// thread it took 10 us more for 44 tiles of 256 x 256.
template <bool TR>
__global__ void __launch_bounds__(256) w8_finalize_kernel(const W8TcArgs a, int TN) {
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t pairs = a.cut_pairs;
    const int out = TR ? a.p.K : a.p.N;
    const int tt = blockIdx.y, t = a.F + tt;
    const int e = blockIdx.x * 256 + threadIdx.x;
    const int tok = e / (kW8Rows / 4), rl = (e % (kW8Rows / 4)) * 4;
    const int m = (t % a.tiles_m) * TN + tok, o = (t / a.tiles_m) * kW8Rows + rl;
    if (m >= a.p.M || o >= out) return;
    const uint32_t total = static_cast<uint32_t>(a.tiles - a.F) * a.chunks;
    const uint32_t first = static_cast<uint32_t>(tt) * a.chunks;
    const uint32_t p0 = ((first + 1) * pairs - 1) / total;
    const uint32_t p1 = ((first + a.chunks) * pairs - 1) / total;
    if (p0 == p1) return;
    int4 s = make_int4(0, 0, 0, 0);
#pragma unroll 4
    for (uint32_t p = p0; p <= p1; ++p) {
        // only the first of the pairs can have begun in an earlier tile
        const uint32_t slot = 2 * p + (p == p0 && total * p / pairs < first ? 1 : 0);
        const int4 v = *reinterpret_cast<const int4*>(a.part + (static_cast<size_t>(slot) * TN + tok) * kW8Rows + rl);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    const int v[4] = {s.x, s.y, s.z, s.w};
    const float as = a.p.a_scales[m];
    uint16_t y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool ok = o + i < out;
        const float ws = (!TR && ok) ? a.p.w_scales[o + i] : 1.0f;
        y[i] = w8_output(v[i], as * ws, (a.p.bias && ok) ? bf16_bits_to_float(a.p.bias[o + i]) : 0.0f);
    }
    uint16_t* dst = a.p.Y + static_cast<size_t>(m) * out + o;
    if ((out & 3) == 0) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(y[0] | (static_cast<uint32_t>(y[1]) << 16),
                                                    y[2] | (static_cast<uint32_t>(y[3]) << 16));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (o + i < out) dst[i] = y[i];
    }
}

}  // namespace w4
