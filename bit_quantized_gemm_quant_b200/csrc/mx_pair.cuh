// mx_pair.cuh -- the product of microscaled activations and weights on the block-scaled
// tensor cores, on pairs of SMs (cta_group::2).
//
//   D[n][m] = sum_k W[n][k] x[m][k],  each a code times its block's power of two
//
// The tensor cores read the codes and the E8M0 scales as they are (block_scale, one scale
// per 32 elements of either operand), so nothing is dequantized and weights cost 4.25 bits
// from memory to the multiplier:
//   x in E2M1: kind::mxf4, both operands packed, K = 64 per instruction;
//   x in E4M3: kind::mxf8f6f4, K = 32; its 4-bit operand lies in shared memory in 8-byte
//     groups of 16 codes with 8-byte gaps, which the copy makes (16U4_ALIGN16B; it wants rows of whole
//     128 codes and 32-byte aligned).
// Either way a stage is one 128-byte swizzle atom per row: 256 elements (4 bits) or 128.
//
// Tiles, pairs, units of work and the epilogue are tc_pair.cuh's: 256 rows of W x bn tokens
// per pair, two accumulators (bn columns each, bn <= 192), so that 512 - 2 bn columns of
// tensor memory are left for scales.  These live there as the instruction wants them: row r
// of an operand in lane r % 32, column r / 32, a 32-bit word of the scales of 128
// consecutive k (the same in all four lane quarters).  Per stage, one warp each for W's
// 128 rows, tokens 0 .. 127 and tokens 128 .. reads 16 scale bytes of a row at a time (512
// k), and writes a stage's words, four rows' per lane, as the 16 bytes that tcgen05.cp.32x128b.warpx4
// takes to the four lane quarters.  Each CTA holds the scales of its own 128 rows and of all of
// the pair's tokens.
//
// Each pipeline stage has its own columns of scales, freed with it, so a copy never
// overwrites scales that an earlier product may still read.
//
// Barriers of a stage: full (the leader's: both CTAs' copies, and an arrival per scale warp of
// both), empty (each CTA's own; the MMA's commit arrives on both).
#pragma once

#include "mx.cuh"
#include "tc_pair.cuh"

namespace bq {

constexpr int kMxEpiWarps = 8;
constexpr int kMxTmaWarp = kMxEpiWarps, kMxMmaWarp = kMxEpiWarps + 1, kMxScaleWarp0 = kMxEpiWarps + 2;
constexpr int kMxThreads = 32 * (kMxScaleWarp0 + 3);
constexpr int kMxMaxStages = 8;
constexpr int kMxMaxBn = 192;

// Elements of a stage, its 128-element chunks, shared bytes and tensor-memory columns of its scales
// (a chunk: 512 bytes and 4 columns for W, twice that for the tokens).
__host__ __device__ constexpr int mx_stage_k(int xbits) { return xbits == 4 ? 256 : 128; }
__host__ __device__ constexpr int mx_chunks(int xbits) { return mx_stage_k(xbits) / 128; }
__host__ __device__ constexpr uint32_t mx_scale_bytes(int xbits) { return 1536u * (uint32_t)mx_chunks(xbits); }
__host__ __device__ constexpr int mx_scale_cols(int xbits) { return 12 * mx_chunks(xbits); }

struct MxParams {
    PairParams q;
    const uint8_t* xs;         // [M][blocks]
    const uint8_t* ws;         // [N][blocks]
    int blocks;                // K / 32
    int vec;                   // scale bytes of one load: 16, 4 or 1 (what rows are a multiple of)
};

// One product of the pair, D += A B with the scales at sfa and sfb (tensor memory).
template <int XB>
BQ_DEVINL void umma_mx_pair(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                            uint32_t accumulate)
{
    if constexpr (XB == 4)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %7, 0;\n\t"
            "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %4, [%5], [%6], p;\n\t}"
            ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %7, 0;\n\t"
            "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], da, db, %4, [%5], [%6], p;\n\t}"
            ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
}

// 512 bytes of scales (32 rows of 16 bytes, without swizzle) to 4 columns of every lane
// quarter, in both CTAs, each from its own shared memory.
BQ_DEVINL void scales_to_tmem_pair(uint32_t taddr, uint32_t smem)
{
    const uint64_t desc = (uint64_t)((smem >> 4) & 0x3FFFu) | (uint64_t)1u << 16 | (uint64_t)(128u >> 4) << 32 | (uint64_t)1u << 46;
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Instruction descriptor of the block-scaled kinds: D fp32.
//   bits 4-5 B scale byte   bits 7-9 A format   bits 10-12 B format   bits 17-22 N >> 3
//   bit 23 scales E8M0   bits 27-28 M >> 7   bits 29-30 A scale byte
// A is W (E2M1), B the tokens.  Formats: kind::mxf4 E2M1 1; kind::mxf8f6f4 E4M3 0, E2M1 5.
template <int XB>
__host__ __device__ constexpr uint32_t umma_idesc_mx(int M, int N)
{
    return (XB == 4 ? (1u << 7) | (1u << 10) : 5u << 7) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27);
}

// Bytes 16 g .. 16 g + 15 of a row of `blocks` scale bytes, zero past its end.
BQ_DEVINL uint4 load_scales16(const uint8_t* row, int g, int blocks, int vec)
{
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    const int b0 = 16 * g;
    if (vec == 16) {
        if (b0 < blocks) v = __ldg(reinterpret_cast<const uint4*>(row + b0));
        return v;
    }
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (vec == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (b0 + 4 * i < blocks) w[i] = __ldg(reinterpret_cast<const uint32_t*>(row + b0 + 4 * i));
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (b0 + i < blocks) w[i >> 2] |= (uint32_t)__ldg(row + b0 + i) << (8 * (i & 3));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

BQ_DEVINL uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// tm_a: codes of W, boxes of a stage x 128 rows; tm_b: codes of the tokens, boxes of a
// stage x bn / 2 tokens.
template <int XB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMxThreads, 1)
mx_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
               const __grid_constant__ MxParams mp)
{
    constexpr int kChunks = mx_chunks(XB), kGroup = 4 / kChunks;       // stages of one 16-byte scale load
    constexpr uint32_t kSfBytes = mx_scale_bytes(XB);
    const PairParams& p = mp.q;
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int S = p.stages;
    const uint32_t b_bytes = (uint32_t)p.bn * 64u;             // this CTA's half of the token tile
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t a_base = base, b_base = base + (uint32_t)S * kPairABytes, sf_base = b_base + (uint32_t)S * b_bytes;
    const uint32_t bar_base = sf_base + (uint32_t)S * kSfBytes;
    auto full_bar = [&](int s) { return bar_base + 8u * (uint32_t)s; };
    auto empty_bar = [&](int s) { return bar_base + 8u * (uint32_t)(S + s); };
    auto tfull_bar = [&](int b) { return bar_base + 8u * (uint32_t)(2 * S + b); };
    auto tempty_bar = [&](int b) { return bar_base + 8u * (uint32_t)(2 * S + 2 + b); };
    const uint32_t done_bar = bar_base + 8u * (uint32_t)(2 * S + 4);
    const uint32_t tmem_slot = done_bar + 8u;
    volatile uint32_t* tmem_slot_ptr =
        reinterpret_cast<volatile uint32_t*>(smem_raw + (base - smem_u32(smem_raw)) + (tmem_slot - base));
    const int scale_warps = p.bn > 128 ? 3 : 2;

    auto tile_r0 = [&](int t) { return (t / p.m_tiles) * 256 + (int)rank * 128; };   // this CTA's first row of W
    auto tile_m0 = [&](int t) { return (t % p.m_tiles) * p.bn; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1 + 2 * (uint32_t)scale_warps);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 2 * kMxEpiWarps);
        }
        mbar_init(done_bar, 1);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == kMxMmaWarp) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot_ptr;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == kMxTmaWarp) {
        // ---------------- codes (each CTA: its own halves) ----------------
        int s = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (PairUnits u(p); ok && u.next();) {
            const int r0 = tile_r0(u.tile), m0 = tile_m0(u.tile) + (int)rank * (p.bn / 2);
            for (int it = u.kb0; it < u.kb1; ++it) {
                if (!mbar_wait_warp(empty_bar(s), ph ^ 1u)) { ok = false; break; }
                const uint32_t bar = map_to_cta(full_bar(s), 0);
                if (elect_one()) {
                    // 16U4_ALIGN16B copies count the packed bytes
                    if (rank == 0) mbar_arrive_expect_tx(full_bar(s), 2u * ((XB == 4 ? kPairABytes : kPairABytes / 2) + b_bytes));
                    tma_load_2d_pair(a_base + (uint32_t)s * kPairABytes, &tm_a, bar, it * 128, r0);
                    tma_load_2d_pair(b_base + (uint32_t)s * b_bytes, &tm_b, bar, it * 128, m0);
                }
                __syncwarp();
                ++issued;
                if (++s == S) { s = 0; ph ^= 1u; }
            }
        }
        // Neither CTA leaves before its last stages are freed (see tc_pair.cuh).
        for (int q = 0; q < S && q < issued; ++q) {
            if (--s < 0) { s = S - 1; ph ^= 1u; }
            if (rank == 0 && !mbar_wait_warp(full_bar(s), ph)) ok = false;
            if (ok) ok = mbar_wait_warp(empty_bar(s), ph);
        }
    } else if (warp == kMxMmaWarp) {
        // ---------------- MMA issuer (the leader's; one elected lane issues) ----------------
        if (rank == 0) {                                 // the whole warp, as in tc_pair.cuh
            const uint32_t idesc = umma_idesc_mx<XB>(256, p.bn);
            const uint64_t bd0 = umma_desc_k_sw128(b_base);
            const uint32_t desc_hi = (uint32_t)(bd0 >> 32), b_lo0 = (uint32_t)bd0, a_lo0 = (uint32_t)umma_desc_k_sw128(a_base);
            const uint32_t sf_tmem0 = tmem_base + 2u * (uint32_t)p.bn;
            int s = 0, lt = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (PairUnits u(p); ok && u.next(); ++lt) {
                const int acc = lt & 1;
                const int kb0 = u.kb0, kb1 = u.kb1;
                if (!mbar_wait_warp(tempty_bar(acc), ((uint32_t)(lt >> 1) & 1u) ^ 1u)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * p.bn);
                for (int it = kb0; it < kb1; ++it) {
                    if (!mbar_wait_warp(full_bar(s), ph)) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t sfa = sf_tmem0 + (uint32_t)(s * mx_scale_cols(XB)), sfb = sfa + 4u * kChunks;
                        const uint32_t sm = sf_base + (uint32_t)s * kSfBytes;
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) {
                            scales_to_tmem_pair(sfa + 4u * c, sm + 512u * c);
                            scales_to_tmem_pair(sfb + 8u * c, sm + 512u * kChunks + 1024u * c);
                            if (p.bn > 128) scales_to_tmem_pair(sfb + 8u * c + 4u, sm + 512u * kChunks + 1024u * c + 512u);
                        }
                        const uint32_t al = a_lo0 + (uint32_t)s * (kPairABytes >> 4), bl = b_lo0 + (uint32_t)s * (b_bytes >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int c = XB == 4 ? k >> 1 : 0;
                            const uint32_t sf = XB == 4 ? 2u * (k & 1) : (uint32_t)k;        // the first scale byte of its word
                            umma_mx_pair<XB>(d_tmem, al + 2u * k, bl + 2u * k, desc_hi, idesc | sf << 4 | sf << 29, sfa + 4u * c,
                                             sfb + 8u * c, it > kb0 || k > 0);
                        }
                        umma_commit_pair(empty_bar(s));
                    }
                    __syncwarp();
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
                if (elect_one()) umma_commit_pair(tfull_bar(acc));
                __syncwarp();
            }
            if (elect_one()) umma_commit_leader(done_bar);   // nothing stays in flight past this point
            __syncwarp();
            mbar_wait_warp(done_bar, 0);
        }
    } else if (warp >= kMxScaleWarp0) {
        // ---------------- scales ----------------
        const int which = warp - kMxScaleWarp0;              // W's rows, tokens 0 .. 127, tokens 128 ..
        if (which < scale_warps) {
            const uint8_t* src = which == 0 ? mp.ws : mp.xs;
            const int limit = which == 0 ? p.N : p.M;
            const uint32_t dst0 = sf_base + (which == 0 ? 0u : 512u * kChunks + 512u * (uint32_t)(which - 1)) + 16u * (uint32_t)lane;
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (PairUnits u(p); ok && u.next();) {
                const int row0 = which == 0 ? tile_r0(u.tile) : tile_m0(u.tile) + 128 * (which - 1);
                const uint8_t* row[4];
                bool in[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = row0 + 32 * j + lane;
                    in[j] = r < limit && (which == 0 || 128 * (which - 1) + 32 * j < p.bn);
                    row[j] = src + (int64_t)(in[j] ? r : 0) * mp.blocks;
                }
                uint4 cur[4], next[4];
                auto load = [&](uint4 (&v)[4], int g) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = in[j] ? load_scales16(row[j], g, mp.blocks, mp.vec) : make_uint4(0u, 0u, 0u, 0u);
                };
                load(next, u.kb0 / kGroup);
                for (int it = u.kb0; it < u.kb1; ++it) {
                    const int sub = it & (kGroup - 1);
                    if (it == u.kb0 || sub == 0) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) cur[j] = next[j];
                        load(next, it / kGroup + 1);
                    }
                    if (!mbar_wait_warp(empty_bar(s), ph ^ 1u)) { ok = false; break; }
                    const uint32_t dst = dst0 + (uint32_t)s * kSfBytes;
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        const int w = sub * kChunks + c;
                        st_shared_v4(dst + (which == 0 ? 512u : 1024u) * c, word_of(cur[0], w), word_of(cur[1], w),
                                     word_of(cur[2], w), word_of(cur[3], w));
                    }
                    fence_proxy_async_smem();                // the copy to tensor memory reads through the async proxy
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(map_to_cta(full_bar(s), 0));
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
        }
    } else {
        // ---------------- epilogue ----------------
        const int q4 = warp & 3, half = warp >> 2;
        const uint32_t lane_addr0 = tmem_base + ((uint32_t)(32 * q4) << 16);
        int lt = 0;
        for (PairUnits u(p); u.next(); ++lt) {
            const int t = u.tile, acc = lt & 1;
            const int r = 32 * q4 + lane;                    // row of this CTA's half of the tile
            float* part = u.slot < 0 ? nullptr : p.ws + (int64_t)u.slot * ((int64_t)p.bn * 256) + (int)rank * 128 + r;
            if (!mbar_wait_warp(tfull_bar(acc), (uint32_t)(lt >> 1) & 1u)) break;
            tc_fence_after();
            pair_drain<kEpiPlain>(p, lane_addr0 + (uint32_t)(acc * p.bn), tile_m0(t), tile_r0(t) + r, part, half, 2);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_cta(tempty_bar(acc), 0));
        }
    }
    __syncwarp();

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == kMxMmaWarp) tmem_dealloc_pair(tmem_base, 512);
}

}  // namespace bq
