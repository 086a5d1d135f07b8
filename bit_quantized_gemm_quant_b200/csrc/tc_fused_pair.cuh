// tc_fused_pair.cuh -- prompt and training sizes of the products with an epilogue: the
// packed weights are dequantized inside the tensor-core product, on pairs of SMs.
//
//   forward:   D[n][m] = sum_k W[n][k] x[m][k]       (weight tile K-major)
//   gradient:  D[k][m] = sum_n W[n][k] dz[m][n]      (weight tile MN-major; up to two
//              matrices summed, for the gated form)
//
// Tiles, pairs, accumulators and units of work are tc_pair.cuh's: 256 D rows x bn
// tokens per pair (cta_group::2), two accumulators of 256 columns; a block of the
// reduction is 128 elements here, two halves of one swizzle atom each.  The weight tile
// arrives as codes: a block's 128 x 128 weights per CTA are 8 KB (8-bit: 16 KB) and 2 KB of
// scales where their bf16 form is 32 KB, so at 256 tokens a block moves 42 KB per SM
// through L2 instead of 64, and no bf16 copy of W is written to or read from memory.  16
// dequant warps, in four groups of four, two groups per block, expand the codes to bf16 in
// shared memory in the layout that the MMA reads: 64 weights of one row per thread, either
// 64 consecutive k of an output row (forward) or 64 consecutive outputs of a reduction row
// (gradient).  The codes land swizzled, so that the code reads and the tile writes of a
// warp cover all banks evenly.
//
// What set the pace on the way (gated 12288 x 4096 affine 4-bit, 2048 tokens, us):
//  - scales: a thread needs two of one row, and rows are far apart in memory, so every load
//    of a warp touches 32 lines; with the loads the dequantization alone took 318, without
//    198.  scale_pack_kernel now lays them out by block first (32 weights: one word of two
//    16-bit values, scale and bias, or Q4_0's d split in two), and they come with the codes;
//  - one ring for codes, tokens and tiles held each through a copy's round trip, the wait
//    for a group and the product: now three rings, each at its own depth;
//  - the MMA warp and the producers beside 16 busy dequant warps: 150 clocks for each wait
//    on a barrier, and an operand move for everything that is not in a uniform register.
//    So blocks are 128 elements (two waits and one commit each), and these warps run their
//    loops whole with one elected lane issuing (forward: 355 with one lane and blocks of
//    64, 277 now);
//  - the epilogue: eight warps, and for the last unit, which no product overlaps, the
//    dequant warps as well.
// Forward, large products are bound by the tensor cores and the power they may draw (1.49
// PFLOP/s in isolation, cuBLAS bf16 reaches 1.64); below 192 tokens a tile the 1050 to 1300 clocks
// that a block's dequantization takes exceed the MMA's.  No pipe is full then (12288 x 4096
// affine 4-bit with gelu, 512 tokens: issue slots 53%, ALU 41%, shared-memory banks 17% + 17%):
// by the decode kernel's loop the arithmetic is about 440 of them, and the rest is the chain
// of a group's block, wait, load, convert, wait for the tile, store, fence and arrive, which
// nothing of the same group overlaps.  Gradients, whose epilogue is a
// plain store and whose reductions are long, may take two token tiles per unit (H = 2): both
// accumulators work on one weight tile, so that a block's dequantization serves up to 512
// tokens (8-bit 12288 x 4096, 2048 tokens, gelu and bias: 199 us with one tile, 172 with
// two).  The price is that the next unit's first products wait for the epilogue.
//
// Barriers: cfull / cempty (codes, each CTA's own), bfull (tokens of both CTAs, the
// leader's), ready (a block's tile, the leader's; 8 dequant warps of each CTA arrive),
// consumed (one per product of a block and a token tile, each CTA's own; the MMA's commit
// arrives on both and thereby frees the token tile and, the last of a block, the weight tile).
#pragma once

#include "scale_pack.cuh"
#include "tc_gemm.cuh"
#include "tc_pair.cuh"

namespace bq {

constexpr int kFpDeqWarps = 16;                 // four groups of 4
constexpr int kFpEpiWarp0 = kFpDeqWarps;        // lane quarter = warp % 4
constexpr int kFpEpiWarps = 8;                  // two per lane quarter (with 4, affine 8-bit 4096 x 4096, 1999 tokens,
                                                // residual and z took 75 us against 69)
constexpr int kFpTokWarp = kFpEpiWarp0 + kFpEpiWarps;   // producer of token tiles
constexpr int kFpCodeWarp = kFpTokWarp + 1;     // producer of codes
constexpr int kFpMmaWarp = kFpCodeWarp + 1;
constexpr int kFpThreads = 32 * (kFpMmaWarp + 1);
constexpr uint32_t kFpScaleBytes = 2048;        // packed scales of a block
// Code stages (a block each), an even number, so that a stage always serves the same two
// dequant groups: a barrier's phases are told apart by parity alone, and a group that had
// not waited for the stage's last fill (made for other groups, and possibly landing after
// later ones) could take the fill before it for its own.
constexpr int kFpMaxCodes = 4;
static_assert(kFpMaxCodes % 2 == 0, "a code stage serves two dequant groups");
constexpr int kFpMaxTiles = 3;
constexpr int kFpConsumed = 16;                 // consumed barriers, at least the depth of each ring
constexpr int kFpMaxTok = 8;                    // token tiles of a block

__host__ __device__ constexpr uint32_t fp_code_bytes(int mode) { return mode == kModeAff8 ? 16384u : 8192u; }   // of a block
// Shared memory beside the token tiles: `tiles` bf16 weight tiles of a block and the codes
__host__ __device__ constexpr uint32_t fp_fixed_bytes(int mode, int tiles, int codes)
{
    return (uint32_t)tiles * 2u * kPairABytes + (uint32_t)codes * (fp_code_bytes(mode) + kFpScaleBytes);
}

struct FpParams {
    PairParams q;
    int codes;                     // code stages: 2 or 4
    const uint32_t* scales;        // packed (scale_pack_kernel)
    int64_t pack_rows;             // its rows per column block
    int64_t pack_mat;              // gradient: its words per matrix
};

// The dequant warps' part: group grp (4 warps) takes half (grp & 1) of the blocks grp >> 1,
// grp >> 1 + 2, ... of the CTA's `left` ones.  A thread expands 64 weights: forward, row r of the tile;
// gradient, row r of the half-block, outputs 64 hk .. of the tile.  (A function of its own:
// inlined, the code that follows it for these warps slowed this loop by 13%.)
template <int MODE, bool MN, int EPI, int H, int kTiles>
__device__ __noinline__ void fp_dequantize(int left, int codes_ring, uint32_t a_base, uint32_t c_base, uint32_t cfull0, uint32_t cempty0,
                                           uint32_t ready0, uint32_t consumed0)
{
    constexpr uint32_t kCBytes = fp_code_bytes(MODE), kCStage = kCBytes + kFpScaleBytes;
    constexpr int kBits = MODE == kModeAff8 ? 8 : 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = warp >> 2, w4 = warp & 3;
    const int half = grp & 1;                       // of the block, always the same for a group
    const int r = MN ? 32 * (w4 & 1) + lane : 32 * w4 + lane;
    const int hk = MN ? w4 >> 1 : 0;
    // row among the block's codes: forward 128 rows (glu: 64 of gate, 64 of up) of 128
    // columns, of which this group takes 64; gradient 128 rows, of which it takes 64
    const int crow = MN ? 64 * half + r : EPI == kEpiGlu ? epi_out_row<EPI>(r) + (lane & 16 ? 64 : 0) : r;
    constexpr int kRowBytes = 128 * kBits / 8;      // 64 or 128
    constexpr int kUnits = kBits / 2;               // 16-byte units of codes per thread
    const int unit0 = (MN ? hk : half) * kUnits;
    const int sw = kRowBytes == 64 ? (crow >> 1) & 3 : crow & 7;     // the units of a row, as the copy swizzles them
    const uint32_t code_row = c_base + (uint32_t)(crow * kRowBytes);
    const uint32_t tile_row = a_base + (uint32_t)(half * (int)kPairABytes + hk * (int)(kPairABytes / 2) + r * 128);
    const uint32_t scale_row = c_base + kCBytes + (uint32_t)(MN ? crow * 16 + hk * 8 : r * 16 + half * 8);
    int a = grp >> 1, c = grp >> 1, block = grp >> 1;   // tile, code stage and block
    uint32_t ph = 0;
    bool ok = true;
    for (; block < left; block += 2) {
        ok = mbar_wait_warp(cfull0 + 8u * (uint32_t)c, ph);
        if (!ok) break;
        const uint32_t codes = code_row + (uint32_t)c * kCStage;
        const uint2 sc = ld_shared_v2(scale_row + (uint32_t)c * kCStage);
        uint4 raw[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i) raw[i] = ld_shared_v4(codes + (uint32_t)(((unit0 + i) ^ sw) << 4));
        __syncwarp();
        if (lane == 0) mbar_arrive(cempty0 + 8u * (uint32_t)c);
        const uint32_t tile = tile_row + (uint32_t)a * (2u * kPairABytes);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t wv[16];
            const uint32_t w = h ? sc.y : sc.x;
            if constexpr (MODE == kModeQ4_0)
                deq_q4_0_half(raw[h], prmt(w, w, 0x1010u), prmt(w, w, 0x3232u), wv);
            else if constexpr (MODE == kModeAff4)
                deq_aff4_half(raw[h], prmt(w, w, 0x1010u), prmt(w, w, 0x3232u), wv);
            else
                deq_aff8_half(raw[2 * h], raw[2 * h + 1], __uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u), wv);
            if (h == 0 && block >= kTiles) {           // the tile's last block is consumed
                const int q = (block - kTiles + 1) * H - 1;
                ok = mbar_wait(consumed0 + 8u * (uint32_t)(q & (kFpConsumed - 1)), (uint32_t)(q / kFpConsumed) & 1u);
                __syncwarp();
            }
            if (!ok) break;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                st_shared_v4(tile + (uint32_t)(((4 * h + j) ^ (r & 7)) << 4), wv[4 * j], wv[4 * j + 1], wv[4 * j + 2],
                             wv[4 * j + 3]);
        }
        if (!ok) break;
        fence_proxy_async_smem();                    // the MMA reads the tile through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(ready0 + 8u * (uint32_t)a);
        if ((c += 2) >= codes_ring) { c -= codes_ring; ph ^= 1u; }
        a = (a + 2) % kTiles;
    }
}

// tm_a0, tm_a1: codes of matrix 0 and 1 as bytes, boxes of 128 columns x 128 rows (glu
// forward: 64 rows of gate and of up).
// tm_b0, tm_b1: tokens, boxes of 64 elements x bn / 2 tokens.
// H: token tiles per unit, 1 (the two accumulators take units in turn) or 2 (both work on
// one unit, which reads each weight tile twice).  kTiles: weight tiles, 2 or 3.
template <int MODE, bool MN, int EPI, int H, int kTiles>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFpThreads, 1)
tc_fused_pair_kernel(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_a1,
                     const __grid_constant__ CUtensorMap tm_b0, const __grid_constant__ CUtensorMap tm_b1,
                     const __grid_constant__ FpParams fp)
{
    constexpr uint32_t kCBytes = fp_code_bytes(MODE), kCStage = kCBytes + kFpScaleBytes;
    constexpr int kBits = MODE == kModeAff8 ? 8 : 4;
    const PairParams& p = fp.q;
    extern __shared__ uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int NC = fp.codes;
    const int NB = p.stages;                       // token tiles (of a block) in the ring
    const uint32_t b_bytes = (uint32_t)p.bn * 64u;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t a_base = base, c_base = a_base + kTiles * 2u * kPairABytes, b_base = c_base + (uint32_t)NC * kCStage;
    const uint32_t bar_base = b_base + (uint32_t)NB * 2u * b_bytes;
    auto cfull_bar = [&](int i) { return bar_base + 8u * (uint32_t)i; };
    auto cempty_bar = [&](int i) { return bar_base + 8u * (uint32_t)(kFpMaxCodes + i); };
    auto ready_bar = [&](int i) { return bar_base + 8u * (uint32_t)(2 * kFpMaxCodes + i); };
    auto bfull_bar = [&](int i) { return bar_base + 8u * (uint32_t)(2 * kFpMaxCodes + kFpMaxTiles + i); };
    auto consumed_bar = [&](int i) { return bar_base + 8u * (uint32_t)(2 * kFpMaxCodes + kFpMaxTiles + kFpMaxTok + i); };
    constexpr int kBars = 2 * kFpMaxCodes + kFpMaxTiles + kFpMaxTok + kFpConsumed;
    auto tfull_bar = [&](int b) { return bar_base + 8u * (uint32_t)(kBars + b); };
    auto tempty_bar = [&](int b) { return bar_base + 8u * (uint32_t)(kBars + 2 + b); };
    const uint32_t done_bar = bar_base + 8u * (uint32_t)(kBars + 4);
    const uint32_t tmem_slot = done_bar + 8u;
    static_assert(8 * (kBars + 6) <= 512, "barriers fit the space the host reserves");
    volatile uint32_t* tmem_slot_ptr =
        reinterpret_cast<volatile uint32_t*>(smem_raw + (base - smem_u32(smem_raw)) + (tmem_slot - base));
    // wait until the pos-th product (of a block and a token tile, >= 0) is done
    auto wait_consumed = [&](int pos) {
        return mbar_wait(consumed_bar(pos & (kFpConsumed - 1)), (uint32_t)(pos / kFpConsumed) & 1u);
    };

    auto tile_r0 = [&](int t) { return (t / p.m_tiles) * 256 + (int)rank * 128; };
    auto tile_m0 = [&](int t) { return (t % p.m_tiles) * (p.bn * H); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < NC; ++i) {
            mbar_init(cfull_bar(i), 1);
            mbar_init(cempty_bar(i), 8);
        }
        for (int i = 0; i < kTiles; ++i) mbar_init(ready_bar(i), 16);
        for (int i = 0; i < NB; ++i) mbar_init(bfull_bar(i), 1);
        for (int i = 0; i < kFpConsumed; ++i) mbar_init(consumed_bar(i), 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull_bar(b), 1);
            mbar_init(tempty_bar(b), 2 * kFpEpiWarps);
        }
        mbar_init(done_bar, 1);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == kFpMmaWarp) {
        tmem_alloc_pair(tmem_slot, 2 * kPairAccCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot_ptr;
    grid_dependency_wait();
    grid_dependents_launch();

    // Chunks idx, idx + parts, ... of the h-th token tile of a unit, in accumulator acc, in
    // the lane quarter of this warp.
    auto drain = [&](int t, int slot, int acc, int h, int idx, int parts) {
        const int q4 = warp & 3, r = 32 * q4 + lane;
        tc_fence_after();
        pair_drain<EPI>(p, tmem_base + ((uint32_t)(32 * q4) << 16) + (uint32_t)(acc * kPairAccCols), tile_m0(t) + h * p.bn,
                        epi_tile_rows<EPI>(tile_r0(t)) + epi_out_row<EPI>(r),
                        slot < 0 ? nullptr : p.ws + ((int64_t)slot * H + h) * ((int64_t)p.bn * 256) + (int)rank * 128 + r, idx,
                        parts);
        tc_fence_before();
    };

    if (warp == kFpTokWarp) {
        // ---------------- token tiles (each CTA: its own half) ----------------
        // (whole warp, one elected lane issues: see the MMA warp)
        int b = 0, pos = 0;
        bool ok = true;
        for (PairUnits u(p); ok && u.next();) {
            const int m0 = tile_m0(u.tile) + (int)rank * (p.bn / 2);
            for (int it = u.kb0; ok && it < u.kb1; ++it) {
                const bool second = it >= p.seg_blocks;
                const CUtensorMap* map = second ? &tm_b1 : &tm_b0;
                const int k0 = (second ? it - p.seg_blocks : it) * 128;
#pragma unroll
                for (int h = 0; h < H; ++h, ++pos) {
                    if (pos >= NB) {
                        ok = wait_consumed(pos - NB);
                        __syncwarp();
                        if (!ok) break;
                    }
                    const uint32_t dst = b_base + (uint32_t)b * 2u * b_bytes, bar = map_to_cta(bfull_bar(b), 0);
                    if (elect_one()) {
                        if (rank == 0) mbar_arrive_expect_tx(bfull_bar(b), 4u * b_bytes);
                        tma_load_2d_pair(dst, map, bar, k0, m0 + h * p.bn);
                        tma_load_2d_pair(dst + b_bytes, map, bar, k0 + 64, m0 + h * p.bn);
                    }
                    __syncwarp();
                    if (++b == NB) b = 0;
                }
            }
        }
        // Leave only when the last products are done: every copy of the pair has then
        // landed and every arrival on this CTA's barriers has been made.  (After a timeout
        // the leader still waits for the copies.)
        for (int q = max(pos - NB, 0); q < pos; ++q) {
            if (rank == 0 && !mbar_wait_warp(bfull_bar(q % NB), (uint32_t)(q / NB) & 1u)) ok = false;
            if (ok) ok = wait_consumed(q);
        }
        __syncwarp();
    } else if (warp == kFpCodeWarp) {
        // ---------------- codes and scales (each CTA: its own rows) ----------------
        int c = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (PairUnits u(p); ok && u.next();) {
            const int r0 = tile_r0(u.tile);
            for (int it = u.kb0; it < u.kb1; ++it, ++issued) {
                if (!mbar_wait_warp(cempty_bar(c), ph ^ 1u)) { ok = false; break; }
                const uint32_t dst = c_base + (uint32_t)c * kCStage, bar = cfull_bar(c);
                const bool second = MN && it >= p.seg_blocks;
                const int kb = second ? it - p.seg_blocks : it;
                // forward: column block kb, rows r0 ..; gradient: column block r0 / 128, rows 128 kb ..
                const uint32_t* sc = fp.scales + (second ? fp.pack_mat : 0) +
                                     (MN ? (int64_t)(r0 / 128) * fp.pack_rows + kb * 128
                                         : (int64_t)kb * fp.pack_rows + r0) * 4;
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar, kCStage);
                    bulk_load(dst + kCBytes, sc, kFpScaleBytes, bar);
                    if constexpr (MN) {
                        tma_load_2d(dst, second ? &tm_a1 : &tm_a0, bar, r0 * kBits / 8, kb * 128);
                    } else if constexpr (EPI == kEpiGlu) {
                        tma_load_2d(dst, &tm_a0, bar, kb * (128 * kBits / 8), r0 / 2);
                        tma_load_2d(dst + kCBytes / 2, &tm_a1, bar, kb * (128 * kBits / 8), r0 / 2);
                    } else {
                        tma_load_2d(dst, &tm_a0, bar, kb * (128 * kBits / 8), r0);
                    }
                }
                __syncwarp();
                if (++c == NC) { c = 0; ph ^= 1u; }
            }
        }
        for (int q = 0; q < NC && q < issued; ++q) {            // every copy has landed
            if (--c < 0) { c = NC - 1; ph ^= 1u; }
            mbar_wait_warp(cfull_bar(c), ph);
        }
        __syncwarp();
    } else if (warp == kFpMmaWarp) {
        // ---------------- MMA issuer (the leader's; one elected lane issues) ----------------
        if (rank == 0) {                                 // the whole warp, as in tc_pair.cuh
            const uint32_t idesc = umma_idesc_bf16_f32(256, p.bn) | (MN ? 1u << 15 : 0u);
            const uint64_t bd0 = umma_desc_k_sw128(b_base);
            const uint32_t desc_hi = (uint32_t)(bd0 >> 32);
            const uint32_t a_lo0 = MN ? (((a_base >> 4) & 0x3FFFu) | ((kPairABytes / 2) >> 4 << 16))   // as in tc_pair.cuh
                                      : (uint32_t)umma_desc_k_sw128(a_base);
            const uint32_t b_lo0 = (uint32_t)bd0;
            int a = 0, b = 0, c = 0, lt = 0;
            uint32_t pha = 0, phb = 0;
            bool ok = true;
            for (PairUnits u(p); ok && u.next(); ++lt) {
                const int kb0 = u.kb0, kb1 = u.kb1;
                const int acc = H == 1 ? lt & 1 : 0;             // the unit's first accumulator, and its uses before
                const uint32_t use = H == 1 ? (uint32_t)(lt >> 1) : (uint32_t)lt;
                if (!mbar_wait_warp(tempty_bar(acc), (use & 1u) ^ 1u)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kPairAccCols);
                for (int it = kb0; ok && it < kb1; ++it) {
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        if (!mbar_wait_warp(bfull_bar(b), phb) || (h == 0 && !mbar_wait_warp(ready_bar(a), pha)) ||
                            (h > 0 && it == kb0 && !mbar_wait_warp(tempty_bar(h), (use & 1u) ^ 1u))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t al = a_lo0 + (uint32_t)a * (kPairABytes >> 3), bl = b_lo0 + (uint32_t)b * (b_bytes >> 3);
                            const uint32_t d = d_tmem + (uint32_t)(h * kPairAccCols);
                            umma_kblock_pair<MN ? 128 : 2>(d, al, bl, desc_hi, idesc, it > kb0);
                            umma_kblock_pair<MN ? 128 : 2>(d, al + (kPairABytes >> 4), bl + (b_bytes >> 4), desc_hi, idesc, 1u);
                            umma_commit_pair(consumed_bar(c));
                        }
                        __syncwarp();
                        c = (c + 1) & (kFpConsumed - 1);
                        if (++b == NB) { b = 0; phb ^= 1u; }
                    }
                    if (++a == kTiles) { a = 0; pha ^= 1u; }
                }
                if (elect_one()) {
#pragma unroll
                    for (int h = 0; h < H; ++h) umma_commit_pair(tfull_bar(acc + h));
                }
                __syncwarp();
            }
            if (elect_one()) umma_commit_pair(done_bar);     // nothing stays in flight past this point
            __syncwarp();
            mbar_wait_warp(done_bar, 0);
        }
        // (the other CTA's MMA warp has nothing to wait for: the pair leaves together, after
        // the leader; its wait here would last as long as the kernel, past any limit)
    } else if (warp >= kFpEpiWarp0) {
        // ---------------- epilogue: all units but the last ----------------
        int lt = 0;
        PairUnits u(p);
        for (bool more = u.next(); more; ++lt) {
            const int tile = u.tile, slot = u.slot;
            more = u.next();
            if (!more) break;
            for (int h = 0; h < H; ++h) {
                const int acc = H == 1 ? lt & 1 : h, use = H == 1 ? lt >> 1 : lt;
                more = more && mbar_wait_warp(tfull_bar(acc), (uint32_t)use & 1u);
                if (!more) break;
                drain(tile, slot, acc, h, (warp - kFpEpiWarp0) >> 2, kFpEpiWarps / 4);
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_to_cta(tempty_bar(acc), 0));
            }
        }
    } else {
        // ---------------- dequantization ----------------
        int left = 0;                                    // blocks of this CTA's sequence
        for (PairUnits u(p); u.next();) left += u.kb1 - u.kb0;
        fp_dequantize<MODE, MN, EPI, H, kTiles>(left, NC, a_base, c_base, cfull_bar(0), cempty_bar(0), map_to_cta(ready_bar(0), 0),
                                     consumed_bar(0));
    }
    __syncwarp();

    // ---------------- the last unit's epilogue: dequant and epilogue warps together ----------------
    // No product overlaps it.  (It waits on done, which has one phase: the dequant warps
    // have not followed tfull's.)
    if (warp < kFpTokWarp) {
        int lt = -1, tile = 0, slot = 0;
        for (PairUnits u(p); u.next(); ++lt) {
            tile = u.tile;
            slot = u.slot;
        }
        if (lt >= 0 && mbar_wait_warp(done_bar, 0))
            for (int h = 0; h < H; ++h) drain(tile, slot, H == 1 ? lt & 1 : h, h, warp >> 2, kFpTokWarp / 4);
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == kFpMmaWarp) tmem_dealloc_pair(tmem_base, 2 * kPairAccCols);
}

}  // namespace bq
