// tc_pair.cuh -- bf16 tensor-core product of dequantized weights with an epilogue,
// on pairs of SMs (cta_group::2), and the dequantizer that feeds it.
//
//   forward:   D[n][m] = sum_k W[n][k] x[m][k]          (W rows K-major)
//   gradient:  D[k][m] = sum_n W[n][k] dz[m][n]         (W rows MN-major: the same
//              row-major bf16 W, read with n as the reduction; up to two matrices
//              summed, for the gated form)
//
// The weights are the MMA's M side: a pair of CTAs owns a tile of 256 output rows
// (128 per CTA, its 128 tensor-memory lanes) x bn tokens (the MMA's N, up to 256).
// Each CTA loads its own 128 rows of the weight tile and half of the tokens; the
// pair's MMA reads both halves, so a token tile costs each SM half the shared
// memory and L2 traffic that it costs alone.  The reduction advances 64 elements
// (one 128-byte swizzle atom) per pipeline stage.
//
// Persistent: one pair per two SMs walks a static schedule of (tile, reduction
// range) units.  Two accumulators of 256 columns: the epilogue drains one while the
// MMA fills the other.  Roles per CTA: 8 epilogue warps (4 lane quarters x 2 column
// halves), one TMA producer warp, one MMA warp (one lane of the pair's leader CTA
// issues).  Barriers of a stage: full (the leader's; both CTAs' copies complete on
// it), empty (each CTA's own; the MMA's commit arrives on both).  Every wait is
// bounded as in tc_gemm.cuh.
#pragma once

#include "epilogue.cuh"
#include "tcgen05.cuh"

namespace bq {

// ------------------------------------------------------------------ pair primitives
BQ_DEVINL uint32_t cluster_ctarank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

BQ_DEVINL void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// This CTA's shared address `a` as seen in CTA `rank` of the cluster.
BQ_DEVINL uint32_t map_to_cta(uint32_t a, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}

// Arrive on a barrier of either CTA.
BQ_DEVINL void mbar_arrive_cluster(uint32_t bar_cluster)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

// Tiled load into this CTA, completing on a barrier of either CTA of the pair.
BQ_DEVINL void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar_cluster, int32_t x, int32_t y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];"
        ::"r"(dst), "l"(map), "r"(bar_cluster), "r"(x), "r"(y) : "memory");
}

BQ_DEVINL void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
                 : "memory");
}

BQ_DEVINL void tmem_relinquish_pair()
{
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

BQ_DEVINL void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// True in one lane of the (converged) warp.
BQ_DEVINL bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// Arrive on `bar` (the same offset in both CTAs) when this thread's earlier tcgen05
// operations complete.
BQ_DEVINL void umma_commit_pair(uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}"
        ::"r"(bar) : "memory");
}

BQ_DEVINL void umma_commit_leader(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// One 64-element block of the reduction: four K = 16 MMAs.  The start address of A's
// descriptor advances by A_STEP 16-byte units per MMA (K-major 2; MN-major 16 rows
// of 128 bytes = 128), B's by 2.
template <int A_STEP>
BQ_DEVINL void umma_kblock_pair(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 l1, l2, l3, m1, m2, m3;\n\t.reg .b64 a0, a1, a2, a3, d0, d1, d2, d3;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 q, %5, %5;\n\t"
        "add.u32 l1, %2, 2;\n\tadd.u32 l2, %2, 4;\n\tadd.u32 l3, %2, 6;\n\t"
        "add.u32 m1, %1, %6;\n\tadd.u32 m2, %1, %7;\n\tadd.u32 m3, %1, %8;\n\t"
        "mov.b64 d0, {%2, %3};\n\tmov.b64 d1, {l1, %3};\n\tmov.b64 d2, {l2, %3};\n\tmov.b64 d3, {l3, %3};\n\t"
        "mov.b64 a0, {%1, %3};\n\tmov.b64 a1, {m1, %3};\n\tmov.b64 a2, {m2, %3};\n\tmov.b64 a3, {m3, %3};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a0, d0, %4, p;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a1, d1, %4, q;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a2, d2, %4, q;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a3, d3, %4, q;\n\t}"
        ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "n"(A_STEP), "n"(2 * A_STEP),
          "n"(3 * A_STEP) : "memory");
}

// ------------------------------------------------------------------ the product
constexpr int kPairEpiWarps = 8;
constexpr int kPairThreads = 32 * (kPairEpiWarps + 2);
constexpr int kPairAccCols = 256;
constexpr uint32_t kPairABytes = 128 * 128;                  // 128 rows x 64 bf16 per CTA and stage

// Shared memory that a CTA of a pair asks for at least: all of tensor memory is its own, and beside it
// no CTA may be resident that holds tensor memory while it waits for another SM's CTA.  (Such a CTA on
// one SM, waiting for one that this CTA keeps from its columns on another, and this CTA's partner waiting
// for the first one's columns, would wait for each other for good.)  More than half of an SM's keeps two
// pairs apart; this much also a pair and a cluster of mx_decode_kernel (kMdMinSmem).
constexpr uint32_t kPairMinSmem = 156 * 1024;

__host__ __device__ constexpr uint32_t pair_stage_bytes(int bn) { return kPairABytes + (uint32_t)bn * 64u; }

struct PairParams {
    EpiParams e;
    int M;                    // tokens
    int N;                    // outputs (D rows; glu: of each of gate and up)
    int bn;                   // token tile, a multiple of 32 in [32, 256]
    int stages;
    int m_tiles, tiles;
    int seg_blocks;           // 64-element blocks of the reduction per matrix
    int segs;                 // matrices summed (1 or 2)
    TailSplit split;          // tiles from split.dp_tiles on are split over the reduction
    float* ws;                // their partial tiles
};

// The units of work of one pair, in order: whole tiles, then its range of the tail.
struct PairUnits {
    const PairParams& p;
    int pair, pairs, nk, next_tile, seg;
    int64_t pos, end;
    int tile, kb0, kb1, slot;                      // the current unit; slot -1: a whole tile

    BQ_DEVINL explicit PairUnits(const PairParams& prm)
        : p(prm), pair((int)blockIdx.x >> 1), pairs((int)gridDim.x >> 1), nk(prm.seg_blocks * prm.segs), next_tile(pair),
          seg(0), pos(0), end(0)
    {
        if (pair < p.split.tail_pairs) {
            pos = p.split.range_begin(pair);
            end = p.split.range_begin(pair + 1);
        }
    }
    BQ_DEVINL bool next()
    {
        if (next_tile < p.split.dp_tiles) {
            tile = next_tile;
            next_tile += pairs;
            kb0 = 0;
            kb1 = nk;
            slot = -1;
            return true;
        }
        if (pos >= end) return false;
        const int j = (int)(pos / nk);
        tile = p.split.dp_tiles + j;
        kb0 = (int)(pos - (int64_t)j * nk);
        kb1 = (int)(end - (int64_t)j * nk < nk ? end - (int64_t)j * nk : nk);
        pos += kb1 - kb0;
        slot = 2 * pair + seg++;
        return true;
    }
};

// Chunks idx, idx + parts, ... of a unit's tokens, of one warp's lane quarter of an
// accumulator (lane_addr), to the outputs, or to the unit's partial tile (part: this
// thread's row of its first token).
template <int EPI>
BQ_DEVINL void pair_drain(const PairParams& p, uint32_t lane_addr, int m0, int n, float* part, int idx, int parts)
{
    constexpr int T = kEpiTokens<EPI>;
    const EpiRow<EPI> row = epi_row<EPI>(p.e, n, p.N);
#pragma unroll 1
    for (int c = T * idx; c < p.bn && m0 + c < p.M; c += T * parts) {
        uint32_t v[T];
        if constexpr (T == 16) tmem_ld_32x32b_x16(lane_addr + (uint32_t)c, v);
        else tmem_ld_32x32b_x8(lane_addr + (uint32_t)c, v);
        tmem_wait_ld();
        if (part) {
#pragma unroll
            for (int j = 0; j < T; ++j) part[(int64_t)(c + j) * 256] = __uint_as_float(v[j]);
        } else {
            epi_store<EPI, T>(p.e, row, v, m0 + c, p.M, p.N);
        }
    }
}

// Tensor maps: A of matrix 0 and 1 (K-major: box 64 x 128 rows; MN-major: box 64 x
// 64 rows, two boxes side by side per stage), B likewise (box 64 x bn / 2 tokens).
template <bool MN, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
tc_pair_kernel(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_a1,
               const __grid_constant__ CUtensorMap tm_b0, const __grid_constant__ CUtensorMap tm_b1,
               const __grid_constant__ PairParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int S = p.stages;
    const uint32_t b_bytes = (uint32_t)p.bn * 64u;             // this CTA's half of the token tile
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t a_base = base, b_base = base + (uint32_t)S * kPairABytes;
    const uint32_t bar_base = b_base + (uint32_t)S * b_bytes;
    auto full_bar = [&](int s) { return bar_base + 8u * (uint32_t)s; };
    auto empty_bar = [&](int s) { return bar_base + 8u * (uint32_t)(S + s); };
    auto tfull_bar = [&](int b) { return bar_base + 8u * (uint32_t)(2 * S + b); };
    auto tempty_bar = [&](int b) { return bar_base + 8u * (uint32_t)(2 * S + 2 + b); };
    const uint32_t done_bar = bar_base + 8u * (uint32_t)(2 * S + 4);
    const uint32_t tmem_slot = done_bar + 8u;
    volatile uint32_t* tmem_slot_ptr =
        reinterpret_cast<volatile uint32_t*>(smem_raw + (base - smem_u32(smem_raw)) + (tmem_slot - base));

    auto tile_r0 = [&](int t) { return (t / p.m_tiles) * 256 + (int)rank * 128; };   // this CTA's first D row
    auto tile_m0 = [&](int t) { return (t % p.m_tiles) * p.bn; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 2 * kPairEpiWarps);
        }
        mbar_init(done_bar, 1);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == kPairEpiWarps + 1) {
        tmem_alloc_pair(tmem_slot, 2 * kPairAccCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot_ptr;

    if (warp == kPairEpiWarps) {
        // ---------------- producer (each CTA: its own halves) ----------------
        if (lane == 0) {
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (PairUnits u(p); ok && u.next();) {
                const int r0 = tile_r0(u.tile), m0 = tile_m0(u.tile) + (int)rank * (p.bn / 2);
                for (int it = u.kb0; it < u.kb1; ++it) {
                    if (!mbar_wait(empty_bar(s), ph ^ 1u)) { ok = false; break; }
                    const bool second = it >= p.seg_blocks;
                    const int k0 = (second ? it - p.seg_blocks : it) * 64;
                    const CUtensorMap* ta = second ? &tm_a1 : &tm_a0;
                    const CUtensorMap* tb = second ? &tm_b1 : &tm_b0;
                    const uint32_t bar = map_to_cta(full_bar(s), 0);
                    const uint32_t a_dst = a_base + (uint32_t)s * kPairABytes;
                    if (rank == 0) mbar_arrive_expect_tx(full_bar(s), 2u * (kPairABytes + b_bytes));
                    if constexpr (MN) {
                        tma_load_2d_pair(a_dst, ta, bar, r0, k0);
                        tma_load_2d_pair(a_dst + kPairABytes / 2, ta, bar, r0 + 64, k0);
                    } else {
                        tma_load_2d_pair(a_dst, ta, bar, k0, r0);
                    }
                    tma_load_2d_pair(b_base + (uint32_t)s * b_bytes, tb, bar, k0, m0);
                    ++issued;
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
            }
            // Neither CTA leaves before its last stages are freed: then every copy has
            // landed and every arrival on this CTA's barriers has been made.  (After a
            // timeout the leader waits for the copies alone.)
            for (int q = 0; q < S && q < issued; ++q) {
                if (--s < 0) { s = S - 1; ph ^= 1u; }
                if (rank == 0 && !mbar_wait(full_bar(s), ph)) ok = false;
                if (ok) ok = mbar_wait(empty_bar(s), ph);
            }
        }
        __syncwarp();
    } else if (warp == kPairEpiWarps + 1) {
        // ---------------- MMA issuer (the leader's; one elected lane issues) ----------------
        // The whole warp runs the loop, so that descriptors and addresses stay in uniform
        // registers: with the loop in one lane every operand of an MMA is moved there
        // first, and a block took 630 clocks with nothing else on the SM.
        if (rank == 0) {
            const uint32_t idesc = umma_idesc_bf16_f32(256, p.bn) | (MN ? 1u << 15 : 0u);
            const uint64_t bd0 = umma_desc_k_sw128(b_base);
            const uint32_t desc_hi = (uint32_t)(bd0 >> 32);
            // MN-major: rows of the reduction 128 bytes apart, 8-row groups 1024 bytes
            // apart (the stride offset, as for K-major), the second 64 of the 128 outputs
            // half a tile further on (the leading offset).
            const uint32_t a_lo0 = MN ? (((a_base >> 4) & 0x3FFFu) | ((kPairABytes / 2) >> 4 << 16))
                                      : (uint32_t)umma_desc_k_sw128(a_base);
            const uint32_t b_lo0 = (uint32_t)bd0;
            int s = 0, lt = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (PairUnits u(p); ok && u.next(); ++lt) {
                const int acc = lt & 1;
                const int kb0 = u.kb0, kb1 = u.kb1;
                if (!mbar_wait_warp(tempty_bar(acc), ((uint32_t)(lt >> 1) & 1u) ^ 1u)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kPairAccCols);
                for (int it = kb0; it < kb1; ++it) {
                    if (!mbar_wait_warp(full_bar(s), ph)) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        umma_kblock_pair<MN ? 128 : 2>(d_tmem, a_lo0 + (uint32_t)s * (kPairABytes >> 4),
                                                       b_lo0 + (uint32_t)s * (b_bytes >> 4), desc_hi, idesc, it > kb0);
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
        __syncwarp();
    } else {
        // ---------------- epilogue ----------------
        const int q4 = warp & 3, half = warp >> 2;
        const uint32_t lane_addr0 = tmem_base + ((uint32_t)(32 * q4) << 16);
        int lt = 0;
        for (PairUnits u(p); u.next(); ++lt) {
            const int t = u.tile, acc = lt & 1;
            const int r = 32 * q4 + lane;                      // row of this CTA's half of the tile
            const int m0 = tile_m0(t);
            const int n = epi_tile_rows<EPI>(tile_r0(t)) + epi_out_row<EPI>(r);
            float* part = u.slot < 0 ? nullptr : p.ws + (int64_t)u.slot * ((int64_t)p.bn * 256) + (int)rank * 128 + r;
            if (!mbar_wait_warp(tfull_bar(acc), (uint32_t)(lt >> 1) & 1u)) break;
            tc_fence_after();
            pair_drain<EPI>(p, lane_addr0 + (uint32_t)(acc * kPairAccCols), m0, n, part, half, 2);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_cta(tempty_bar(acc), 0));
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == kPairEpiWarps + 1) tmem_dealloc_pair(tmem_base, 2 * kPairAccCols);
}

// ------------------------------------------------------------------ dequantized weights for it
// One or two matrices [N][K] to bf16 rows, the bits of q4_0_dequantize and
// affine_dequantize.  Forward glu interleaves the two in blocks of 16 rows (see
// epi_out_row), into a matrix of 32 ceil(N / 16) rows; otherwise matrix i starts at
// out + i N K.
//
// Bound by HBM: codes and scales in, 2 N K bytes out per matrix.  A thread makes 8
// consecutive weights, so that a warp's stores are 512 consecutive bytes and its code
// loads (8 BITS bits per thread) are consecutive too.
struct DequantMat {
    const uint32_t* wq;
    const uint16_t* scales;
    const uint16_t* biases;
};

// BITS 0: Q4_0.
template <int BITS>
BQ_DEVINL uint4 dequant8(const DequantMat& w, int64_t row, int c, int chunks, int gs_shift)
{
    const int64_t gi = row * ((chunks * 8) >> gs_shift) + ((c * 8) >> gs_shift);
    float v[8];
    if constexpr (BITS == 0) {
        // 8 weights of a block: the low or high nibbles of 8 of its 16 bytes
        const uint2 b = __ldg(reinterpret_cast<const uint2*>(w.wq) + (row * chunks + c) / 4 * 2 + (c & 1));
        const float d = f16_bits_to_f32(__ldg(w.scales + gi));
        const int sh = (c & 2) * 2;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __fmul_rn(d, (float)((int)(((i < 4 ? b.x : b.y) >> (8 * (i & 3) + sh)) & 15u) - 8));
    } else {
        const int64_t bit = (row * chunks + c) * (8 * BITS);
        const uint32_t* p = w.wq + (bit >> 5);
        const int sh = (int)(bit & 31);
        uint64_t q = __ldg(p);
        if (8 * BITS > 32 || (32 % (8 * BITS) != 0 && sh + 8 * BITS > 32)) q |= (uint64_t)__ldg(p + 1) << 32;
        q >>= sh;
        const float s = bf16_bits_to_f32(__ldg(w.scales + gi)), z = bf16_bits_to_f32(__ldg(w.biases + gi));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __fmaf_rn(s, (float)(uint32_t)((q >> (BITS * i)) & ((1u << BITS) - 1u)), z);
    }
    return make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]), pack_bf16x2_rn(v[4], v[5]),
                      pack_bf16x2_rn(v[6], v[7]));
}

template <int BITS>
__global__ void __launch_bounds__(256)
dequant_rows_kernel(DequantMat w0, DequantMat w1, uint16_t* __restrict__ out, int N, int chunks, int gs_shift,
                    int interleave)
{
    const DequantMat& w = blockIdx.y ? w1 : w0;
    const int64_t total = (int64_t)N * chunks;
    uint4* o = reinterpret_cast<uint4*>(out);
    for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / chunks;
        const int c = (int)(i - row * chunks);
        const int64_t to = interleave ? 32 * (row >> 4) + (row & 15) + 16 * blockIdx.y : row + (int64_t)blockIdx.y * N;
        o[to * chunks + c] = dequant8<BITS>(w, row, c, chunks, gs_shift);
    }
}

}  // namespace bq
