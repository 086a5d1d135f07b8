// gemv_ring.cuh -- decode sizes (up to 16 tokens) of the products with an epilogue:
// packed weights stream once through a shared-memory ring, are dequantized in
// registers to bf16 (Q4_0 and 8 bits: the dequantizers' bits; the others round scale q + bias
// once, see gemv.cuh) and multiplied by warp MMAs with fp32 accumulators; bias, activation, residual or gate follow in the same
// kernel.
//
// A tile is 16 rows of the MMA's M side: 16 outputs, or with a gate 8 gate rows and
// the 8 up rows of the same outputs, so that a thread's accumulators of rows g and
// g + 8 are the two factors of one output.  A CTA takes tiles b, b + grid, ...; its
// reduction columns come in chunks of 2048 (one ring stage: 16 rows of codes, scales
// and biases, each one tensor copy; copies of single rows were limited by their
// number: glu, 8 tokens, 12288 x 4096 affine 4-bit took 48 us with them).  8 compute
// warps split a chunk, two steps of 128 columns each (16 warps with one step each spend
// more on waits: 22.6 against 20.3 us; fetching the next chunk ahead into registers costs
// more issue slots than it hides, 22.4): the four threads of a quad take 32 consecutive
// columns each of rows g and g + 8.  So every warp sees the same columns
// of every tile, and its activations (the MMA's B fragments, 16 registers per 8 tokens
// and step) are loaded once for Q4_0, 4 and 8 bits: up to K = 8192 with 8 tokens, up to 4096
// with 9 to 16 (64 registers).  The compiler keeps part of them in local memory where all 64 are in
// use: 40 to 96 bytes a thread for Q4_0, 88 to 128 for 4 bits, 176 to 288 for 8.  Longer
// reductions and the other widths load them from L2 again for every tile.
//
// The floor is HBM (the packed weights, read once), but neither it nor a pipe is what binds:
// in the profile of glu, 8 tokens, 12288 x 4096 affine 4-bit, HBM runs at 29% and issue slots
// are half busy while the kernel is active (39% of its time), with waits for loads and barriers
// as the first stall.  The two compute warps of a scheduler each wait for a stage, load,
// dequantize (2 to 2.5 instructions per weight) and multiply in order, so that one other warp
// at most covers a wait: a chunk takes about 1500 clocks, where a loop of its dequantization
// and MMAs alone takes 880 (Q4_0: 1050; the MMAs 420).  About 4 us of a call are launch, first
// copy and last output.  The ring keeps about 150 KB per SM in flight.  Measured, graph-timed
// over rotating weights: 8192 x 2048 Q4_0 gated, one token, 10.2 us (18.9 MB); 12288 x 4096
// affine 4-bit gated, 8 tokens, 20.3 us (57 MB), one matrix 13.0; 2048 x 8192 Q4_0, one token
// with residual, 6.7 us (9.4 MB); 256 x 512, 16 tokens, 3.8 us; 12288 x 4096 with 2, 3 and 6 bits,
// one token, 15.5, 16.4 and 17.8 us; 4096 x 14336 affine 4-bit, one token, 17.1 us.
//
// Rows of a stage are padded so that the quads' loads of 8 rows fall in different
// banks (ring_code_pitch).  The warps' partial sums of a tile meet in shared memory, two
// buffers in turn; two epilogue warps add them in warp order and write the outputs
// while the compute warps go on with the next tile.
#pragma once

#include "dequant.cuh"
#include "epilogue.cuh"
#include "gemv.cuh"
#include "gemv_stream.cuh"

namespace bq {

constexpr int kRingWarps = 8;
constexpr int kRingSteps = 2;                     // 128-column steps of a chunk per warp
constexpr int kRingEpiWarps = 2;
constexpr int kRingThreads = 32 * (kRingWarps + 1 + kRingEpiWarps);
constexpr int kRingCols = 128 * kRingSteps * kRingWarps;   // reduction columns per stage (2048)
constexpr int kRingMaxStages = 8;

// BITS 0 is Q4_0 (4 bits).
__host__ __device__ constexpr int ring_bits(int BITS) { return BITS == 0 ? 4 : BITS; }

// A stage's codes of one row: kRingCols columns in panels of at most 1024 bytes (8-bit:
// two), each with bytes of padding that make 8 rows x 4 quads of (4 BITS)-byte chunks,
// read 4, 8 or 16 bytes at a time, cover all banks once.  The copy's box is as wide as
// the padded row (the padding holds the next columns), so one tensor copy writes it.
__host__ __device__ constexpr int ring_panels(int bits) { return bits == 8 ? 2 : 1; }
__host__ __device__ constexpr int ring_code_pitch(int bits)
{
    return kRingCols * bits / 8 / ring_panels(bits) +
           (bits == 2 ? 32 : bits == 3 ? 48 : bits == 4 ? 64 : bits == 6 ? 96 : 16);
}
// Scales: 16 bytes of padding spread 8 rows over the banks for every group size.
__host__ __device__ constexpr int ring_scale_pitch(int gs_shift) { return (kRingCols >> gs_shift) * 2 + 16; }

// Codes first, then 16 rows of scales and of biases (space for groups of 32).
__host__ __device__ constexpr int ring_code_bytes(int bits) { return 16 * ring_panels(bits) * ring_code_pitch(bits); }
__host__ __device__ constexpr int ring_stage_bytes(int BITS)
{
    return ring_code_bytes(ring_bits(BITS)) + (BITS == 0 ? 1 : 2) * 16 * ring_scale_pitch(5);
}

struct RingMat {
    const uint16_t* scales;
    const uint16_t* biases;
};

// Tensor maps of gate and up (act: [0] only): codes as 8-byte words, box = a panel's
// padded rows; scales and biases as 16-bit values.
struct RingMaps {
    CUtensorMap codes[2], scales[2], biases[2];
};

struct RingParams {
    RingMat w[2];
    const uint16_t* x;
    EpiParams e;
    int M, N, K;
    int gs_shift;
    int tiles, stages, nchunks;
    int scale_bulk;            // scale rows start on 16 bytes and go through the ring
};

// 32 codes of one row to 16 bf16x2 weights; MMA i of the chunk's 8 takes pairs 2i (its
// k slots 2t, 2t + 1) and 2i + 1 (2t + 8, 2t + 9).  ring_x gives x in the same order.
template <int BITS>
BQ_DEVINL void ring_dequant(const uint32_t (&w)[ring_bits(BITS)], uint32_t s_raw, uint32_t b_raw, uint32_t (&p)[16])
{
    if constexpr (BITS == 0 || BITS == 4) {
        const ChunkScale cs = expand_scale<BITS == 0 ? Fmt::Q4_0 : Fmt::AFF4>(s_raw, b_raw);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t q[4];
            dequant_word<BITS == 0 ? Fmt::Q4_0 : Fmt::AFF4>(w[i], cs, q);
#pragma unroll
            for (int k = 0; k < 4; ++k) p[4 * i + k] = q[k];
        }
    } else if constexpr (BITS == 8) {
        const uint64_t s2 = f32x2_splat(bf16_bits_to_f32(s_raw)), b2 = f32x2_splat(bf16_bits_to_f32(b_raw));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[2 * i] = deq_aff8_pair<0>(w[i], s2, b2);
            p[2 * i + 1] = deq_aff8_pair<2>(w[i], s2, b2);
        }
    } else {
        const uint32_t s2 = s_raw | (s_raw << 16), b2 = b_raw | (b_raw << 16);
        if constexpr (BITS == 2) {
            // codes n and n + 8 of a word side by side, 128 + q as bf16, minus 128 (exact)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                p[i] = hfma2_bf16(hsub2_bf16_i<0x43004300u>(and_or_i<0x00030003u, 0x43004300u>(w[i >> 3] >> (2 * (i & 7)))),
                                  s2, b2);
        } else {
            constexpr uint32_t mask = (1u << BITS) - 1u;
#pragma unroll
            for (int i = 0; i < 16; ++i) {                       // codes 2i and 2i + 1
                const int bit = 2 * BITS * i, j = bit >> 5, sh = bit & 31;
                const uint32_t v = sh + 2 * BITS > 32 ? __funnelshift_r(w[j], w[j + 1], sh) : w[j] >> sh;
                const uint32_t q = and_or_i<mask, 0x43004300u>(v) | ((v << (16 - BITS)) & (mask << 16));
                p[i] = hfma2_bf16(hsub2_bf16_i<0x43004300u>(q), s2, b2);
            }
        }
    }
}

// The 32 activations xw (pairs in column order) as B fragments, in ring_dequant's order.
template <int BITS>
BQ_DEVINL void ring_x(const uint32_t (&xw)[16], uint32_t (&b)[16])
{
    if constexpr (BITS == 0 || BITS == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t q[4];
            x_word_pairs<BITS == 0 ? Fmt::Q4_0 : Fmt::AFF4>(xw, i, q);
#pragma unroll
            for (int k = 0; k < 4; ++k) b[4 * i + k] = q[k];
        }
    } else if constexpr (BITS == 2) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {                           // columns 16 w + n, 16 w + n + 8
            const int w = i >> 3, n = i & 7;
            b[i] = prmt(xw[8 * w + n / 2], xw[8 * w + 4 + n / 2], n & 1 ? 0x7632u : 0x5410u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) b[i] = xw[i];
    }
}

// The B fragments of step (columns 128 step + 32 t ...) for tokens 8n + g.
template <int BITS, int NT>
BQ_DEVINL void ring_load_x(const RingParams& p, int step, int g, int t, uint32_t (&b)[NT][16])
{
    const int k0 = 128 * step + 32 * t;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        uint32_t xw[16];
        if (k0 < p.K && 8 * n + g < p.M) {
            const uint16_t* xp = p.x + (int64_t)(8 * n + g) * p.K + k0;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const uint4 q = ldg_cached(xp + 8 * v);
                xw[4 * v] = q.x; xw[4 * v + 1] = q.y; xw[4 * v + 2] = q.z; xw[4 * v + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int v = 0; v < 16; ++v) xw[v] = 0u;
        }
        ring_x<BITS>(xw, b[n]);
    }
}

// 4 BITS bytes of shared memory (one chunk of 32 codes).
template <int BITS>
BQ_DEVINL void ring_load_codes(const uint8_t* s, uint32_t (&w)[ring_bits(BITS)])
{
    constexpr int B = ring_bits(BITS);
    if constexpr (B % 4 == 0) {
#pragma unroll
        for (int i = 0; i < B / 4; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(s + 16 * i);
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
    } else if constexpr (B % 2 == 0) {
#pragma unroll
        for (int i = 0; i < B / 2; ++i) {
            const uint2 v = *reinterpret_cast<const uint2*>(s + 8 * i);
            w[2 * i] = v.x; w[2 * i + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < B; ++i) w[i] = *reinterpret_cast<const uint32_t*>(s + 4 * i);
    }
}

// XS: chunks of the reduction whose activations stay in registers (K <= 2048 XS), 0:
// loaded again for every tile.
template <int BITS, int NT, int XS, int EPI>
__global__ void __launch_bounds__(kRingThreads, 1)
gemv_ring_kernel(const __grid_constant__ RingMaps maps, const __grid_constant__ RingParams p)
{
    constexpr int B = ring_bits(BITS);
    constexpr int kPitch = ring_code_pitch(B), kPanels = ring_panels(B);
    constexpr int kPanelCols = kRingCols / kPanels;
    constexpr int kScaleOff = ring_code_bytes(B), kBiasOff = kScaleOff + 16 * ring_scale_pitch(5);
    constexpr int kStage = ring_stage_bytes(BITS);
    constexpr bool kAffine = BITS != 0;
    constexpr int kOuts = EPI == kEpiGlu ? 8 : 16;          // outputs per tile
    // shared-memory offset of rows 8h .. 8h + 7 of panel q
    auto panel_off = [](int h, int q) { return (EPI == kEpiGlu ? h * kPanels + q : 2 * q + h) * 8 * kPitch; };
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ __align__(8) uint64_t bars[2 * kRingMaxStages + 4];
    __shared__ float red[2][kRingWarps][16][8 * NT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](int s) { return bar0 + 8u * (uint32_t)s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (uint32_t)(kRingMaxStages + s); };
    auto sums_bar = [&](int b) { return bar0 + 8u * (uint32_t)(2 * kRingMaxStages + b); };       // a tile's sums are in red[b]
    auto taken_bar = [&](int b) { return bar0 + 8u * (uint32_t)(2 * kRingMaxStages + 2 + b); };  // ... and have been read
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), kRingWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(sums_bar(b), kRingWarps);
            mbar_init(taken_bar(b), kRingEpiWarps);
        }
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (threadIdx.x == 32 * kRingWarps) {
        for (int i = 0; i < (EPI == kEpiGlu ? 2 : 1); ++i) {
            tma_prefetch_desc(&maps.codes[i]);
            if (p.scale_bulk) tma_prefetch_desc(&maps.scales[i]);
            if (p.scale_bulk && kAffine) tma_prefetch_desc(&maps.biases[i]);
        }
    }
    __syncthreads();
    grid_dependency_wait();
    grid_dependents_launch();      // a following kernel's set-up may overlap this one (it waits before its reads)
    const int groups = p.K >> p.gs_shift;

    if (warp == kRingWarps) {
        // ---------------- producer: one lane per copy of a stage ----------------
        constexpr int kMats = EPI == kEpiGlu ? 2 : 1, kRows = 16 / kMats;
        const int sp = ring_scale_pitch(p.gs_shift), kinds = p.scale_bulk ? (kAffine ? 2 : 1) : 0;
        const uint32_t tx = (uint32_t)(16 * (kPanels * kPitch + kinds * sp));
        // this lane's copy: codes of (matrix, panel), then scales, then biases
        const int nc = kMats * kPanels;
        const int mat = lane < nc ? lane / kPanels : (lane - nc) % kMats, kind = lane < nc ? 0 : 1 + (lane - nc) / kMats;
        const bool mine = lane < nc + kinds * kMats;
        const int panel = lane < nc ? lane % kPanels : 0;
        const CUtensorMap* map = kind == 0 ? &maps.codes[mat] : kind == 1 ? &maps.scales[mat] : &maps.biases[mat];
        const int dst_off = kind == 0 ? (mat * kPanels + panel) * kRows * kPitch
                                      : (kind == 1 ? kScaleOff : kBiasOff) + mat * kRows * sp;
        const int x0 = kind == 0 ? panel * (kPanelCols * B / 64) : 0;
        const int xj = kind == 0 ? kRingCols * B / 64 : kRingCols >> p.gs_shift;
        int s = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int tile = blockIdx.x; tile < p.tiles && ok; tile += gridDim.x) {
            for (int j = 0; j < p.nchunks; ++j) {
                if (!mbar_wait_warp(empty_bar(s), ph ^ 1u)) { ok = false; break; }
                if (lane == 0) mbar_arrive_expect_tx(full_bar(s), tx);
                __syncwarp();
                if (mine)
                    tma_load_2d(smem_u32(ring) + (uint32_t)(s * kStage + dst_off), map, full_bar(s), x0 + j * xj,
                                tile * kOuts);
                ++issued;
                if (++s == p.stages) { s = 0; ph ^= 1u; }
            }
        }
        // every issued copy has landed before this CTA may exit
        for (int q = 0; q < p.stages && q < issued; ++q) {
            if (--s < 0) { s = p.stages - 1; ph ^= 1u; }
            mbar_wait_warp(full_bar(s), ph);
        }
        return;
    }

    if (warp > kRingWarps) {
        // ---------------- epilogue: consecutive threads on consecutive outputs ----------------
        int buf = 0;
        uint32_t ph = 0;
        for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
            constexpr int kPer = kOuts * 8 * NT / (32 * kRingEpiWarps);
            EpiOperands op[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int o = threadIdx.x - 32 * (kRingWarps + 1) + i * 32 * kRingEpiWarps, m = o / kOuts;
                const int n = tile * kOuts + o % kOuts;
                op[i] = EpiOperands{0.0f, 0.0f, 0.0f};
                if (m < p.M && n < p.N) op[i] = epi_operands<EPI>(p.e, m, n, p.N);   // in flight while the sums form
            }
            if (!mbar_wait_warp(sums_bar(buf), ph)) break;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int o = threadIdx.x - 32 * (kRingWarps + 1) + i * 32 * kRingEpiWarps, m = o / kOuts;
                const int r = o % kOuts, n = tile * kOuts + r;
                if (m >= p.M || n >= p.N) continue;
                float a = 0.0f, b = 0.0f;
#pragma unroll
                for (int w = 0; w < kRingWarps; ++w) {
                    a += red[buf][w][r][m];
                    if constexpr (EPI == kEpiGlu) b += red[buf][w][r + 8][m];
                }
                epi_finish<EPI>(p.e, op[i], a, b, m, n, p.N);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(taken_bar(buf));
            buf ^= 1;
            ph ^= (uint32_t)(buf == 0);
        }
        return;
    }

    // ---------------- compute ----------------
    const int g = lane >> 2, t = lane & 3;
    uint32_t xr[XS > 0 ? XS : 1][kRingSteps][NT][16];
    if constexpr (XS > 0) {
#pragma unroll
        for (int j = 0; j < XS; ++j)
#pragma unroll
            for (int i = 0; i < kRingSteps; ++i)
                ring_load_x<BITS, NT>(p, (j * kRingWarps + warp) * kRingSteps + i, g, t, xr[j][i]);
    }
    const int sp = ring_scale_pitch(p.gs_shift);
    const int col0 = 128 * kRingSteps * warp + 32 * t;                     // this thread's first columns of a chunk
    const uint8_t* codes0 = ring + panel_off(0, col0 / kPanelCols) + g * kPitch + col0 % kPanelCols * B / 8;
    const uint8_t* scales0 = ring + kScaleOff + g * sp;
    constexpr int kHalf = (EPI == kEpiGlu ? kPanels : 1) * 8 * kPitch;     // to the codes of row g + 8
    int s = 0, buf = 0;
    uint32_t ph = 0, rph = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x, buf ^= 1) {
        float acc[2][NT][4];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[e][n][i] = 0.0f;
        auto chunk = [&](int j, const uint32_t (&xb)[kRingSteps][NT][16]) {
            // columns past K: their codes and scales are 0 (the copies fill with 0, sr and
            // br start at 0) and so are their activations
            uint32_t cw[kRingSteps][2][B], sr[kRingSteps][2], br[kRingSteps][2];
            if (!p.scale_bulk) {
#pragma unroll
                for (int i = 0; i < kRingSteps; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        sr[i][h] = br[i][h] = 0u;
                        const int r = EPI == kEpiGlu ? tile * 8 + g : tile * 16 + 8 * h + g;
                        const int k = j * kRingCols + col0 + 128 * i;
                        const RingMat& w = p.w[EPI == kEpiGlu ? h : 0];
                        if (r < p.N && k < p.K) {
                            const int64_t gi = (int64_t)r * groups + (k >> p.gs_shift);
                            sr[i][h] = __ldg(w.scales + gi);
                            if constexpr (kAffine) br[i][h] = __ldg(w.biases + gi);
                        }
                    }
            }
            ok = ok && mbar_wait_warp(full_bar(s), ph);
            const uint8_t* cs = codes0 + s * kStage;
#pragma unroll
            for (int i = 0; i < kRingSteps; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) ring_load_codes<BITS>(cs + h * kHalf + 16 * B * i, cw[i][h]);
            if (p.scale_bulk) {
                const uint8_t* ss = scales0 + s * kStage;
#pragma unroll
                for (int i = 0; i < kRingSteps; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint8_t* q = ss + h * 8 * sp + ((col0 + 128 * i) >> p.gs_shift) * 2;
                        sr[i][h] = *reinterpret_cast<const uint16_t*>(q);
                        if constexpr (kAffine) br[i][h] = *reinterpret_cast<const uint16_t*>(q + (kBiasOff - kScaleOff));
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty_bar(s));
            if (++s == p.stages) { s = 0; ph ^= 1u; }
#pragma unroll
            for (int i = 0; i < kRingSteps; ++i) {
                uint32_t pa[2][16];
#pragma unroll
                for (int h = 0; h < 2; ++h) ring_dequant<BITS>(cw[i][h], sr[i][h], br[i][h], pa[h]);
#pragma unroll
                for (int q = 0; q < 8; ++q)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_bf16_16816(acc[q & 1][n], pa[0][2 * q], pa[1][2 * q], pa[0][2 * q + 1], pa[1][2 * q + 1],
                                       xb[i][n][2 * q], xb[i][n][2 * q + 1]);
            }
        };
        if constexpr (XS > 0) {
#pragma unroll
            for (int j = 0; j < XS; ++j)
                if (j < p.nchunks) chunk(j, xr[j]);
        } else {
            for (int j = 0; j < p.nchunks; ++j) {
                uint32_t xb[kRingSteps][NT][16];
#pragma unroll
                for (int i = 0; i < kRingSteps; ++i)
                    ring_load_x<BITS, NT>(p, (j * kRingWarps + warp) * kRingSteps + i, g, t, xb[i]);
                chunk(j, xb);
            }
        }
        ok = ok && mbar_wait_warp(taken_bar(buf), rph ^ 1u);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[buf][warp][g + 8 * (i >> 1)][8 * n + 2 * t + (i & 1)] = acc[0][n][i] + acc[1][n][i];
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(sums_bar(buf));        // after a timeout the tile is never stored
        rph ^= (uint32_t)(buf == 1);
    }
}

}  // namespace bq
