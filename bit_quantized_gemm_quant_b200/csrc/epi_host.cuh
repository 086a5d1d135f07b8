// epi_host.cuh -- host side of the products with an epilogue and of their
// gradients: argument checks, plans, workspaces and launches.  Included by
// bqgemm.cu, after the helpers it uses.
#pragma once

namespace bq {
namespace {

// One quantized matrix [N][K] as an entry point receives it.
struct QMat {
    const void* wq;
    const void* scales;
    const void* biases;
};

int bits_of(WFmt f)
{
    switch (f) {
    case WFmt::AFF2: return 2;
    case WFmt::AFF3: return 3;
    case WFmt::AFF6: return 6;
    case WFmt::AFF8: return 8;
    default: return 4;
    }
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

// The current device's SM count and shared memory, a B200's without a device.
void device_or_b200(int* num_sms, int* smem_optin)
{
    int dev;
    DeviceInfo di;
    *num_sms = 148;
    *smem_optin = 232448;
    if (cudaGetDevice(&dev) == cudaSuccess && current_device(&dev, &di) == BQ_OK) {
        *num_sms = di.num_sms;
        *smem_optin = di.max_smem_optin;
    }
    cudaGetLastError();
}

// ------------------------------------------------------------------ pair product
struct PairPlan {
    int bn = 32, stages = 0, pairs = 0;
    int codes = 0;                  // fused: code stages
    int wtiles = 3;                 // fused: bf16 weight tiles
    int halves = 1;                 // token tiles of bn per unit (fused: 1 or 2)
    int64_t tiles = 0;
    TailSplit split{};
    size_t ws_bytes = 0;
};

// What a block of the reduction costs a pair in SM clocks: block0, plus per token of the
// tile, plus as much as `crowd` when all pairs are busy.
struct PairCost {
    double block0, per_token, crowd;
    int max_halves;                 // token tiles per unit: with 2, max(1480, 555 + 4.67 per token)
};

// Token tile and split of the last round for `rows` D rows, M tokens and nk blocks of the
// reduction; shared memory: fixed_bytes, and per stage tok_bytes per token beside a_bytes.
// The least cost of a model in SM clocks: blocks as above, a fixed start per unit of work,
// the last unit's epilogue, and for a split last round the partial tiles' traffic and the
// kernel that sums them.  Its numbers are fitted to a B200 sweep over every tile width,
// one or two token tiles and every split below, for 72 problems of the fused kernel (2048
// x 8192 to 12288 x 4096, 24 to 2048 tokens, forward and gradient): the plan it picks is
// 1% slower than the problem's best on average, 6% at worst.
bool plan_pair(int64_t rows, int64_t M, int64_t nk, int num_sms, int smem_optin, int fixed_bytes, int a_bytes,
               int tok_bytes, const PairCost& pc, PairPlan* pl)
{
    const int64_t pairs = std::max(num_sms / 2, 1), rtiles = (rows + 255) / 256;
    const int64_t maxb = std::min<int64_t>(256, (M + 31) / 32 * 32);
    double best = 1e300;
    for (int halves = 1; halves <= pc.max_halves; ++halves) {
        for (int b = 32; b <= maxb; b += 32) {
            if (halves == 2 && M <= b) break;
            const int64_t tok = (int64_t)halves * b, tiles = ((M + tok - 1) / tok) * rtiles;
            const double start = halves == 2 ? 1500.0 + 12.0 * b : 1500.0, drain = 1000.0 + 8.0 * (double)tok;
            // a unit of n blocks with `busy` pairs at work
            auto unit = [&](int64_t n, int64_t busy) {
                const double block = halves == 2 ? std::max(1480.0, 555.0 + 4.67 * (double)tok)
                                                 : pc.block0 + pc.per_token * b +
                                                       pc.crowd * (double)std::min(busy, pairs) / (double)pairs;
                return (double)n * block + start;
            };
            auto consider = [&](double c, int64_t dp, int64_t tail_pairs) {
                if (c < best) {
                    best = c;
                    pl->bn = b;
                    pl->halves = halves;
                    pl->tiles = tiles;
                    pl->split.dp_tiles = (int)dp;
                    pl->split.tail = (int)(tiles - dp);
                    pl->split.tail_pairs = (int)tail_pairs;
                }
            };
            consider((double)((tiles + pairs - 1) / pairs) * unit(nk, tiles) + drain, tiles, 0);
            const int64_t dp = tiles / pairs * pairs, tail = tiles - dp;
            if (tail == 0) continue;
            // ranges of at least 2 blocks, at least one per tile: as many as there are pairs, or
            // a whole number per tile, so that none touches two tiles (4096 x 4096 affine
            // 4-bit, 128 tokens: 16.2 us with 4 per tile, 17.5 with 74 over 16 tiles)
            auto split = [&](int64_t tp) {
                const bool whole = tp % tail == 0;
                const double traffic = (double)(whole ? tp : tp + tail) * (double)tok * 256.0 * 8.0 / 2225.0;
                consider((double)(dp / pairs) * unit(nk, pairs) + unit((tail * nk + tp - 1) / tp, tp) + (whole ? 0.0 : start) +
                             drain + 4800.0 + traffic, dp, tp);
            };
            split(std::max<int64_t>(tail, std::min<int64_t>(pairs, tail * nk / 2)));
            for (int64_t s = 2; s * tail <= pairs && 2 * s <= nk; ++s) split(s * tail);
        }
    }
    pl->pairs = (int)pairs;
    pl->split.blocks = (int)nk;
    pl->stages = std::min<int>(kFpMaxTok, (smem_optin - 1024 - 512 - fixed_bytes) / (a_bytes + pl->bn * tok_bytes));
    pl->ws_bytes = pl->split.tail ? (size_t)2 * (size_t)pl->split.tail_pairs * (size_t)(pl->halves * pl->bn) * 256u * 4u : 0u;
    return pl->stages >= 2 && pl->tiles <= INT32_MAX / 256 && nk <= INT32_MAX / 2;
}

// launch_pdl with a 3-D grid.
template <typename KernelT, typename... Args>
bq_status launch_pdl_dim(KernelT kern, dim3 grid, int threads, size_t smem, cudaStream_t st, const Args&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
        cudaGetLastError();
        return BQ_ERR_CUDA;
    }
    return launch_status();
}

// The sums of the split last round, where the plan has one.
template <int EPI>
bq_status launch_reduce(const DeviceInfo& di, const PairPlan& pl, const PairParams& p, cudaStream_t st)
{
    if (pl.split.tail == 0) return BQ_OK;
    const int tok = pl.halves * pl.bn;
    const int64_t blocks = (int64_t)pl.split.tail * ((tok + kReduceTokens - 1) / kReduceTokens);
    return launch_pdl_dim(epi_reduce_kernel<EPI>, dim3((unsigned)blocks), 256, 0, st, (const float*)p.ws, p.e, p.M, p.N, tok,
                          p.m_tiles, p.split);
}

// D = sum over segs of A_i . B_i^T with the epilogue e.  A_i: bf16 weights, a_rows
// rows (K-major: D rows x red; MN: red x D rows); B_i: tokens [M][red], b_pitch
// elements apart.  outs: outputs per token (glu: of each of gate and up).
template <bool MN, int EPI>
bq_status launch_pair(const DeviceInfo& di, int dev, const PairPlan& pl, const uint16_t* const* A,
                      const uint16_t* const* B, int segs, int64_t rows, int64_t outs, int64_t M, int64_t red,
                      int64_t b_pitch, const EpiParams& e, void* ws, cudaStream_t st)
{
    auto kern = tc_pair_kernel<MN, EPI>;
    static bool attr_done[kMaxDevices] = {};
    if (!attr_done[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, di.max_smem_optin) != cudaSuccess)
            return BQ_ERR_CUDA;
        attr_done[dev] = true;
    }
    CUtensorMap ta[2], tb[2];
    for (int i = 0; i < 2; ++i) {
        const int j = i < segs ? i : 0;
        const bool a_ok = MN ? make_map(&ta[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, A[j], red, rows, 64, 64,
                                        CU_TENSOR_MAP_SWIZZLE_128B)
                             : make_map(&ta[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, A[j], rows, red, 128, 64,
                                        CU_TENSOR_MAP_SWIZZLE_128B);
        if (!a_ok || !make_map_pitch(&tb[i], B[j], M, red, b_pitch, pl.bn / 2, 64)) return BQ_ERR_CUDA;
    }
    PairParams p;
    p.e = e;
    p.M = (int)M;
    p.N = (int)outs;
    p.bn = pl.bn;
    p.stages = pl.stages;
    p.m_tiles = (int)((M + pl.bn - 1) / pl.bn);
    p.tiles = (int)pl.tiles;
    p.seg_blocks = (int)((red + 63) / 64);
    p.segs = segs;
    p.split = pl.split;
    p.ws = reinterpret_cast<float*>(ws);
    // every pair when there are whole rounds before the tail: the units are dealt by pair
    const unsigned grid = 2u * (unsigned)std::min<int64_t>(pl.split.tail && pl.split.dp_tiles ? pl.pairs
                                                           : pl.split.tail ? pl.split.tail_pairs : pl.tiles, pl.pairs);
    const size_t smem = std::max<size_t>(1024 + (size_t)pl.stages * pair_stage_bytes(pl.bn) + 512,
                                         (size_t)di.max_smem_optin / 2 + 1024);   // one CTA per SM (all of TMEM)
    kern<<<grid, kPairThreads, smem, st>>>(ta[0], ta[1], tb[0], tb[1], p);
    bq_status s = launch_status();
    return s != BQ_OK ? s : launch_reduce<EPI>(di, pl, p, st);
}

bq_status dequant_rows(WFmt fmt, const QMat* w, int count, uint16_t* out, int64_t N, int64_t K, int group_size,
                       bool interleave, const DeviceInfo& di, cudaStream_t st)
{
    DequantMat m[2];
    for (int i = 0; i < 2; ++i) {
        const QMat& q = w[i < count ? i : 0];
        m[i] = DequantMat{reinterpret_cast<const uint32_t*>(q.wq), reinterpret_cast<const uint16_t*>(q.scales),
                          reinterpret_cast<const uint16_t*>(q.biases)};
    }
    const int chunks = (int)(K / 8), shift = group_size == 32 ? 5 : group_size == 64 ? 6 : 7;
    const dim3 grid((unsigned)std::min<int64_t>((N * chunks + 255) / 256, (int64_t)di.num_sms * 16), (unsigned)count);
    switch (fmt) {
    case WFmt::Q4_0: dequant_rows_kernel<0><<<grid, 256, 0, st>>>(m[0], m[1], out, (int)N, chunks, shift, interleave); break;
    case WFmt::AFF2: dequant_rows_kernel<2><<<grid, 256, 0, st>>>(m[0], m[1], out, (int)N, chunks, shift, interleave); break;
    case WFmt::AFF3: dequant_rows_kernel<3><<<grid, 256, 0, st>>>(m[0], m[1], out, (int)N, chunks, shift, interleave); break;
    case WFmt::AFF4: dequant_rows_kernel<4><<<grid, 256, 0, st>>>(m[0], m[1], out, (int)N, chunks, shift, interleave); break;
    case WFmt::AFF6: dequant_rows_kernel<6><<<grid, 256, 0, st>>>(m[0], m[1], out, (int)N, chunks, shift, interleave); break;
    default: dequant_rows_kernel<8><<<grid, 256, 0, st>>>(m[0], m[1], out, (int)N, chunks, shift, interleave); break;
    }
    return launch_status();
}

// ------------------------------------------------------------------ decode sizes
constexpr int64_t kRingMaxM = 16;

// The ring kernel moves rows by tensor copies, so rows of codes must be 16-byte
// multiples (always so for 4 and 8 bits).
bool ring_applies(WFmt fmt, int64_t M, int64_t K) { return M <= kRingMaxM && K * bits_of(fmt) % 128 == 0; }

template <int BITS, int NT, int XS, int EPI>
bq_status launch_ring_cfg(const RingMaps& maps, RingParams& p, const DeviceInfo& di, int dev, cudaStream_t st)
{
    auto kern = gemv_ring_kernel<BITS, NT, XS, EPI>;
    constexpr int kStatic = 2 * kRingWarps * 16 * (8 * NT + 1) * 4 + 2 * kRingMaxStages * 8 + 64;
    const int room = di.max_smem_optin - kStatic - 1024;
    static bool attr_done[kMaxDevices] = {};
    if (!attr_done[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, room) != cudaSuccess) {
            cudaGetLastError();
            return BQ_ERR_CUDA;
        }
        attr_done[dev] = true;
    }
    p.stages = std::min(kRingMaxStages, room / ring_stage_bytes(BITS));
    return launch_pdl(kern, std::min(p.tiles, di.num_sms), kRingThreads, (size_t)p.stages * ring_stage_bytes(BITS), st, maps,
                      p);
}

// Activations loaded once for up to 4 chunks of 2048 columns and 8 tokens (2 chunks and 16
// tokens): 64 registers, in part spilled (see gemv_ring.cuh).
template <int BITS, int EPI>
bq_status launch_ring_bits(const QMat* w, RingParams& p, const DeviceInfo& di, int dev, cudaStream_t st)
{
    constexpr int mats = EPI == kEpiGlu ? 2 : 1, rows = 16 / mats, bits = ring_bits(BITS);
    RingMaps maps;
    for (int i = 0; i < 2; ++i) {
        const QMat& q = w[i < mats ? i : 0];
        bool ok = make_map(&maps.codes[i], CU_TENSOR_MAP_DATA_TYPE_UINT64, 8, q.wq, p.N, (int64_t)p.K * bits / 64, rows,
                           ring_code_pitch(bits) / 8, CU_TENSOR_MAP_SWIZZLE_NONE);
        if (p.scale_bulk)
            ok = ok && make_map(&maps.scales[i], CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, q.scales, p.N, p.K >> p.gs_shift, rows,
                                ring_scale_pitch(p.gs_shift) / 2, CU_TENSOR_MAP_SWIZZLE_NONE) &&
                 (BITS == 0 || make_map(&maps.biases[i], CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, q.biases, p.N,
                                        p.K >> p.gs_shift, rows, ring_scale_pitch(p.gs_shift) / 2,
                                        CU_TENSOR_MAP_SWIZZLE_NONE));
        if (!ok) return BQ_ERR_CUDA;
    }
    if constexpr (BITS == 0 || BITS == 4 || BITS == 8) {
        if (p.M <= 8 && p.nchunks <= 2) return launch_ring_cfg<BITS, 1, 2, EPI>(maps, p, di, dev, st);
        if (p.M <= 8 && p.nchunks <= 4) return launch_ring_cfg<BITS, 1, 4, EPI>(maps, p, di, dev, st);
        if (p.M > 8 && p.nchunks <= 2) return launch_ring_cfg<BITS, 2, 2, EPI>(maps, p, di, dev, st);
    }
    if (p.M <= 8) return launch_ring_cfg<BITS, 1, 0, EPI>(maps, p, di, dev, st);
    return launch_ring_cfg<BITS, 2, 0, EPI>(maps, p, di, dev, st);
}

template <int EPI>
bq_status launch_ring(WFmt fmt, const uint16_t* x, const QMat* w, const EpiParams& e, int64_t M, int64_t N, int64_t K,
                      int group_size, const DeviceInfo& di, int dev, cudaStream_t st)
{
    RingParams p;
    for (int i = 0; i < 2; ++i) {
        const QMat& q = w[EPI == kEpiGlu ? i : 0];
        p.w[i] = RingMat{reinterpret_cast<const uint16_t*>(q.scales), reinterpret_cast<const uint16_t*>(q.biases)};
    }
    p.x = x;
    p.e = e;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.gs_shift = group_size == 32 ? 5 : group_size == 64 ? 6 : 7;
    p.nchunks = (int)((K + kRingCols - 1) / kRingCols);
    p.scale_bulk = (K >> p.gs_shift) % 8 == 0;
    const int64_t outs = EPI == kEpiGlu ? 8 : 16;
    p.tiles = (int)((N + outs - 1) / outs);
    switch (fmt) {
    case WFmt::Q4_0: return launch_ring_bits<0, EPI>(w, p, di, dev, st);
    case WFmt::AFF2: return launch_ring_bits<2, EPI>(w, p, di, dev, st);
    case WFmt::AFF3: return launch_ring_bits<3, EPI>(w, p, di, dev, st);
    case WFmt::AFF4: return launch_ring_bits<4, EPI>(w, p, di, dev, st);
    case WFmt::AFF6: return launch_ring_bits<6, EPI>(w, p, di, dev, st);
    default: return launch_ring_bits<8, EPI>(w, p, di, dev, st);
    }
}

// ------------------------------------------------------------------ codes dequantized inside the pair product
// Shape of the packed scales: whole 256-row tiles and 128-column blocks forward, whole
// 128-row blocks and 256-column tiles for the gradient.
struct ScalePack {
    int64_t rows, cols, mat;        // rows per column block, padded columns, words per matrix (gradient)
    size_t bytes;
};

ScalePack scale_pack(bool mn, int mats, int64_t N, int64_t K)
{
    ScalePack s;
    if (mn) {
        s.rows = (N + 127) / 128 * 128;
        s.cols = (K + 255) / 256 * 256;
        s.mat = s.rows * (s.cols / 32);
        s.bytes = up256((size_t)mats * (size_t)s.mat * 4u);
    } else {
        s.rows = ((mats == 2 ? 32 * ((N + 15) / 16) : N) + 255) / 256 * 256;
        s.cols = (K + 127) / 128 * 128;
        s.mat = 0;
        s.bytes = up256((size_t)s.rows * (size_t)(s.cols / 32) * 4u);
    }
    return s;
}

int fp_mode(WFmt f) { return f == WFmt::Q4_0 ? kModeQ4_0 : f == WFmt::AFF4 ? kModeAff4 : kModeAff8; }

// The work of laying out the scales of w (1 or 2 matrices [N][K]) at `packed`, and its
// number of blocks (0: too many); interleave: for the glu forward product.
int64_t scale_pack_params(bool mn, const QMat* w, int mats, bool interleave, int64_t N, int64_t K, int group_size,
                          void* packed, ScalePackParams* pp)
{
    const ScalePack sp = scale_pack(mn, mats, N, K);
    for (int i = 0; i < 2; ++i) {
        const QMat& q = w[i < mats ? i : 0];
        pp->scales[i] = reinterpret_cast<const uint16_t*>(q.scales);
        pp->biases[i] = reinterpret_cast<const uint16_t*>(q.biases);
    }
    pp->out = reinterpret_cast<uint32_t*>(packed);
    pp->N = (int)N;
    pp->K = (int)K;
    pp->gs_shift = group_size == 32 ? 5 : group_size == 64 ? 6 : 7;
    pp->interleave = interleave;
    pp->cols = (int)sp.cols;
    pp->pack_rows = sp.rows;
    pp->pack_mat = sp.mat;
    pp->row_chunks = (int)((sp.rows / (interleave ? 2 : 1) + 31) / 32);
    pp->col_chunks = (int)((sp.cols + 2047) / 2048);
    const int64_t blocks = (int64_t)pp->row_chunks * pp->col_chunks * mats;
    return blocks <= INT32_MAX / 2 ? blocks : 0;
}

bq_status launch_scale_pack(bool mn, const QMat* w, int mats, bool interleave, int64_t N, int64_t K, int group_size,
                            void* packed, cudaStream_t st)
{
    ScalePackParams pp;
    const int64_t blocks = scale_pack_params(mn, w, mats, interleave, N, K, group_size, packed, &pp);
    return blocks ? launch_pdl_dim(scale_pack_kernel, dim3((unsigned)blocks), 256, 0, st, pp) : BQ_ERR_SHAPE;
}

// The product of launch_pair with the codes of w (1 or 2 matrices [N][K]) and their
// packed scales in place of bf16 weights.  Forward: B[0] = x, red = K; gradient (MN): B[i] = dz of matrix i,
// red = N.
template <int MODE, bool MN, int EPI, int H, int T>
bq_status launch_fused_pair(const DeviceInfo& di, int dev, const PairPlan& pl, const QMat* w, int mats,
                            const uint16_t* const* B, int64_t N, int64_t K, int64_t M, int64_t b_pitch, int group_size,
                            const EpiParams& e, void* packed, void* ws, cudaStream_t st)
{
    auto kern = tc_fused_pair_kernel<MODE, MN, EPI, H, T>;
    static bool attr_done[kMaxDevices] = {};
    if (!attr_done[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, di.max_smem_optin) != cudaSuccess) {
            cudaGetLastError();
            return BQ_ERR_CUDA;
        }
        attr_done[dev] = true;
    }
    constexpr int bits = MODE == kModeAff8 ? 8 : 4, row_bytes = 128 * bits / 8;
    constexpr CUtensorMapSwizzle sw = row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    const int64_t red = MN ? N : K, outs = MN ? K : N;
    CUtensorMap ta[2], tb[2];
    FpParams p;
    for (int i = 0; i < 2; ++i) {
        const QMat& q = w[i < mats ? i : 0];
        if (!make_map(&ta[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q.wq, N, K * bits / 8, epi_tile_rows<EPI>(128),
                      row_bytes, sw) ||
            !make_map_pitch(&tb[i], B[MN && i < mats ? i : 0], M, red, b_pitch, pl.bn / 2, 64))
            return BQ_ERR_CUDA;
    }
    const ScalePack sp = scale_pack(MN, EPI == kEpiGlu ? 2 : mats, N, K);
    p.codes = pl.codes;
    p.scales = reinterpret_cast<const uint32_t*>(packed);
    p.pack_rows = sp.rows;
    p.pack_mat = sp.mat;
    p.q.e = e;
    p.q.M = (int)M;
    p.q.N = (int)outs;
    p.q.bn = pl.bn;
    p.q.stages = pl.stages;
    p.q.m_tiles = (int)((M + H * pl.bn - 1) / (H * pl.bn));
    p.q.tiles = (int)pl.tiles;
    p.q.seg_blocks = (int)((red + 127) / 128);
    p.q.segs = MN ? mats : 1;
    p.q.split = pl.split;
    p.q.ws = reinterpret_cast<float*>(ws);
    // every pair when there are whole rounds before the tail: the units are dealt by pair
    const unsigned grid = 2u * (unsigned)std::min<int64_t>(pl.split.tail && pl.split.dp_tiles ? pl.pairs
                                                           : pl.split.tail ? pl.split.tail_pairs : pl.tiles, pl.pairs);
    const size_t smem = std::max<size_t>(1024 + fp_fixed_bytes(MODE, T, pl.codes) + (size_t)pl.stages * (size_t)pl.bn * 128u + 512,
                                         (size_t)di.max_smem_optin / 2 + 1024);   // one CTA per SM (all of TMEM)
    const bq_status s = launch_pdl_dim(kern, dim3(grid), kFpThreads, smem, st, ta[0], ta[1], tb[0], tb[1], p);
    return s != BQ_OK ? s : launch_reduce<EPI>(di, pl, p.q, st);
}

template <bool MN, int EPI>
bq_status launch_fused_pair_fmt(WFmt fmt, const DeviceInfo& di, int dev, const PairPlan& pl, const QMat* w, int mats,
                                const uint16_t* const* B, int64_t N, int64_t K, int64_t M, int64_t b_pitch,
                                int group_size, const EpiParams& e, void* packed, void* ws, cudaStream_t st)
{
    auto go = [&](auto mode) {
        constexpr int m = decltype(mode)::value;
        auto launch = [&](auto halves, auto wtiles) {
            return launch_fused_pair<m, MN, EPI, decltype(halves)::value, decltype(wtiles)::value>(
                di, dev, pl, w, mats, B, N, K, M, b_pitch, group_size, e, packed, ws, st);
        };
        using One = std::integral_constant<int, 1>;
        using Two = std::integral_constant<int, 2>;
        using Three = std::integral_constant<int, 3>;
        if constexpr (MN && m == kModeAff8)
            return pl.halves == 2 ? launch(Two{}, Two{}) : launch(One{}, Two{});
        else if constexpr (MN)
            return pl.halves == 2 ? launch(Two{}, Three{}) : launch(One{}, Three{});
        else if constexpr (m == kModeAff8)
            return pl.wtiles == 2 ? launch(One{}, Two{}) : launch(One{}, Three{});
        else
            return launch(One{}, Three{});
    };
    if (fmt == WFmt::Q4_0) return go(std::integral_constant<int, kModeQ4_0>{});
    if (fmt == WFmt::AFF4) return go(std::integral_constant<int, kModeAff4>{});
    return go(std::integral_constant<int, kModeAff8>{});
}

// ------------------------------------------------------------------ layouts of the workspaces
// Forward: the packed scales or the bf16 weights (glu: interleaved, in whole blocks of
// 16 rows), then the partial sums of the split tiles.  Gradient: the same, then padded copies of the
// gradients when N is not a multiple of 8 (their rows must start on 16 bytes), the
// biases' partial sums, the product's partial sums.
struct EpiWs {
    bool fused = false;             // codes dequantized inside the product: no bf16 weights
    PairPlan pl;
    int64_t rows = 0;               // D rows of the product
    size_t off_pad = 0, off_part = 0, off_split = 0, bytes = 0;   // the bf16 weights or packed scales are at 0
    int64_t pitch = 0;              // elements per row of the product's token operand
    int row_blocks = 0, rows_per_block = 0;
};

// Q4_0 and affine 4- and 8-bit codes are dequantized inside the product, which has row widths
// and conversions for these two only; the others go through a bf16 copy of W, written and read back
// (12288 x 4096, 64 tokens: 56 to 59 us where 4 bits take 25; 2048 tokens: 165 to 169 and 142).
// A block's rows of 2, 3 and 6 bits, 32, 48 and 96 bytes, could be copied as well wherever K
// times the bits is a multiple of 128.  The costs of that form's blocks are estimates, not fitted.
// Two token tiles per unit only for gradients: their epilogue is a plain store and their
// reductions are long (12288 x 4096, 2048 tokens: 8-bit with gelu and bias 193 us with one,
// 170 with two; gated affine 4-bit 317 and 309).  Forward the exposed epilogue costs as much
// as the dequantization saved (12288 x 4096 affine 4-bit with gelu, 512 tokens: 51 and 60;
// 8-bit, 400 tokens, no activation: 54 and 52).
bool plan_epi_product(WFmt fmt, bool gradient, int64_t rows, int64_t M, int segs, int64_t red, int num_sms,
                      int smem_optin, EpiWs* w)
{
    w->rows = rows;
    w->fused = has_fast_paths(fmt);
    if (!w->fused)      // blocks of 64
        return plan_pair(rows, M, segs * ((red + 63) / 64), num_sms, smem_optin, 0, (int)kPairABytes, 64,
                         PairCost{300.0, 1.5, 0.0, 1}, &w->pl);
    const int mode = fp_mode(fmt);
    int wtiles = mode == kModeAff8 ? 2 : 3;      // bf16 weight tiles: 8-bit codes leave room for two of them
    if (!plan_pair(rows, M, segs * ((red + 127) / 128), num_sms, smem_optin, (int)fp_fixed_bytes(mode, wtiles, 2), 0, 128,
                   PairCost{980.0, 1.3, 300.0, gradient ? 2 : 1}, &w->pl))
        return false;
    auto token_tiles = [&](int wt, int codes) {
        return (smem_optin - 1024 - 512 - (int)fp_fixed_bytes(mode, wt, codes)) / (w->pl.bn * 128);
    };
    // 8-bit forward: three weight tiles where they leave room for three token tiles (4096 x
    // 4096, 1999 tokens in tiles of 224, with residual and z: 67 us with two weight tiles, 64.5
    // with three; 12288 x 4096, 4096 tokens in tiles of 256, where two token tiles would be left:
    // 322 and 333).
    if (mode == kModeAff8 && !gradient && token_tiles(3, 2) >= 3) wtiles = 3;
    // Four code stages where they leave room for three token tiles, else two: 1 to 8% apart
    // below 256 tokens a tile, and 12% the other way at 256, where two token tiles would be
    // left.
    w->pl.wtiles = wtiles;
    w->pl.codes = token_tiles(wtiles, kFpMaxCodes) >= 3 ? kFpMaxCodes : 2;
    w->pl.stages = std::min<int>(kFpMaxTok, token_tiles(wtiles, w->pl.codes));
    return true;
}

bool plan_forward(WFmt fmt, int mats, int64_t M, int64_t N, int64_t K, int num_sms, int smem_optin, EpiWs* w)
{
    // glu: tiles of 32 rows per 16 outputs
    if (!plan_epi_product(fmt, false, mats == 2 ? 32 * ((N + 15) / 16) : N, M, 1, K, num_sms, smem_optin, w)) return false;
    w->off_split = w->fused ? scale_pack(false, mats, N, K).bytes : up256((size_t)w->rows * (size_t)K * 2u);
    w->bytes = w->off_split + w->pl.ws_bytes;
    return true;
}

bool plan_backward(WFmt fmt, int mats, int64_t M, int64_t N, int64_t K, int num_sms, int smem_optin, EpiWs* w)
{
    if (K > 0 && !plan_epi_product(fmt, true, K, M, mats, N, num_sms, smem_optin, w)) return false;
    w->pitch = (N + 7) / 8 * 8;
    // blocks of 8 warps over rows of tokens: about 8 blocks per SM, at least 32 rows each
    const int64_t cols = std::max<int64_t>(1, (N + 255) / 256);
    const int64_t want = std::max<int64_t>(1, (int64_t)num_sms * 8 / cols);
    const int64_t rpb = std::max<int64_t>(32, ((M + want - 1) / want + 7) / 8 * 8);
    w->rows_per_block = (int)rpb;
    w->row_blocks = (int)((M + rpb - 1) / rpb);
    size_t off = w->fused ? scale_pack(true, mats, N, K).bytes : up256((size_t)mats * (size_t)N * (size_t)K * 2u);
    w->off_pad = off;
    if (N % 8 != 0) off += (size_t)mats * up256((size_t)M * (size_t)w->pitch * 2u);
    w->off_part = off;
    off += up256((size_t)w->row_blocks * (size_t)mats * (size_t)N * 4u);
    w->off_split = off;
    w->bytes = off + w->pl.ws_bytes;
    return true;
}

// The caller's workspace (BQ_ERR_WORKSPACE when it is too small) or the stream's buffer.
bq_status epi_workspace(int dev, cudaStream_t st, void* workspace, size_t workspace_bytes, size_t need, void** out)
{
    if (need == 0 || workspace) {
        *out = workspace;
        return workspace_bytes < need ? BQ_ERR_WORKSPACE : BQ_OK;
    }
    try {
        return library_workspace(dev, st, need, out);
    } catch (...) {                      // its tables could not grow: no exception leaves a C entry
        return BQ_ERR_CUDA;
    }
}

bool sizes_ok(int64_t M, int64_t N, int64_t K)
{
    // 32-bit tile, row and column numbers in the kernels, with room for a tile's width
    return M <= INT32_MAX - 1024 && N <= INT32_MAX / 2 - 1024 && K <= 65535 * 2048;
}

// ------------------------------------------------------------------ forward
template <int EPI>
bq_status epi_forward(const uint16_t* x, const QMat* w, const EpiParams& e, int64_t M, int64_t N, int64_t K,
                      int group_size, int bits, void* workspace, size_t workspace_bytes, cudaStream_t st)
{
    constexpr int mats = EPI == kEpiGlu ? 2 : 1;
    if (M < 0 || N < 0 || K < 0 || !sizes_ok(M, N, K)) return BQ_ERR_SHAPE;
    if (e.act < kActNone || e.act > kActSilu) return BQ_ERR_UNSUPPORTED;
    if (mats == 2 && (w[0].biases == nullptr) != (w[1].biases == nullptr)) return BQ_ERR_NULL;   // one format
    WFmt fmt;
    bq_status s = check_format(w[0].biases, N, K, group_size, bits, &fmt);
    if (s != BQ_OK) return s;
    if (M == 0 || N == 0) return BQ_OK;
    if (!e.y || (EPI == kEpiGlu && (e.pre == nullptr) != (e.pre2 == nullptr))) return BQ_ERR_NULL;
    for (const void* q : {(const void*)e.y, (const void*)e.bias, (const void*)e.bias2, (const void*)e.res,
                          (const void*)e.pre, (const void*)e.pre2, (const void*)workspace})
        if (!aligned16(q)) return BQ_ERR_ALIGN;
    if (K > 0) {
        if (!x) return BQ_ERR_NULL;
        if (!aligned16(x)) return BQ_ERR_ALIGN;
        for (int i = 0; i < mats; ++i) {
            if (!w[i].wq || !w[i].scales) return BQ_ERR_NULL;
            if (!aligned16(w[i].wq) || !aligned16(w[i].scales) || !aligned16(w[i].biases)) return BQ_ERR_ALIGN;
        }
    }
    int dev;
    DeviceInfo di;
    if ((s = current_device(&dev, &di)) != BQ_OK) return s;
    if (K == 0) {
        epi_empty_kernel<EPI><<<grid_for(M * N, 256, di), 256, 0, st>>>(e, M, (int)N);
        return launch_status();
    }
    if (ring_applies(fmt, M, K)) return launch_ring<EPI>(fmt, x, w, e, M, N, K, group_size, di, dev, st);
    EpiWs ws;
    if (!plan_forward(fmt, mats, M, N, K, di.num_sms, di.max_smem_optin, &ws)) return BQ_ERR_SHAPE;   // too many tiles
    void* buf = nullptr;
    if ((s = epi_workspace(dev, st, workspace, workspace_bytes, ws.bytes, &buf)) != BQ_OK) return s;
    if (ws.fused) {
        if ((s = launch_scale_pack(false, w, mats, mats == 2, N, K, group_size, buf, st)) != BQ_OK) return s;
        return launch_fused_pair_fmt<false, EPI>(fmt, di, dev, ws.pl, w, mats, &x, N, K, M, K, group_size, e, buf,
                                                 reinterpret_cast<uint8_t*>(buf) + ws.off_split, st);
    }
    uint16_t* wb = reinterpret_cast<uint16_t*>(buf);
    if ((s = dequant_rows(fmt, w, mats, wb, N, K, group_size, mats == 2, di, st)) != BQ_OK) return s;
    return launch_pair<false, EPI>(di, dev, ws.pl, &wb, &x, 1, ws.rows, N, M, K, K, e,
                                   reinterpret_cast<uint8_t*>(buf) + ws.off_split, st);
}

// ------------------------------------------------------------------ backward
template <bool GLU, int V>
bq_status launch_epi_grad_v(EpiGradParams& p, int act, int row_blocks, cudaStream_t st)
{
    p.col_blocks = (int)(((int64_t)p.N + 32 * V - 1) / (32 * V));
    const int64_t blocks = p.pack_blocks + (int64_t)p.col_blocks * row_blocks;
    if (blocks > INT32_MAX) return BQ_ERR_SHAPE;
    auto go = [&](auto kern) { return launch_pdl_dim(kern, dim3((unsigned)blocks), 256, 0, st, p); };
    switch (act) {
    case kActRelu: return go(epi_grad_kernel<GLU, kActRelu, V>);
    case kActGelu: return go(epi_grad_kernel<GLU, kActGelu, V>);
    case kActGeluTanh: return go(epi_grad_kernel<GLU, kActGeluTanh, V>);
    case kActSilu: return go(epi_grad_kernel<GLU, kActSilu, V>);
    default: return go(epi_grad_kernel<GLU, kActNone, V>);
    }
}

// dy [M][N] and the saved z (glu: g, u) to dz (dg, du), dx and the biases' gradients.
struct EpiBackward {
    const uint16_t* dy;
    const uint16_t* pre[2];
    uint16_t* dx;
    uint16_t* d[2];
    uint16_t* db[2];
};

template <bool GLU>
bq_status epi_backward(const EpiBackward& b, const QMat* w, int act, int64_t M, int64_t N, int64_t K, int group_size,
                       int bits, void* workspace, size_t workspace_bytes, cudaStream_t st)
{
    constexpr int mats = GLU ? 2 : 1;
    if (M < 0 || N < 0 || K < 0 || !sizes_ok(M, N, K)) return BQ_ERR_SHAPE;
    if (act < kActNone || act > kActSilu) return BQ_ERR_UNSUPPORTED;
    if (GLU && (w[0].biases == nullptr) != (w[1].biases == nullptr)) return BQ_ERR_NULL;
    WFmt fmt;
    bq_status s = check_format(w[0].biases, N, K, group_size, bits, &fmt);
    if (s != BQ_OK) return s;
    const bool none = !GLU && act == kActNone;          // dz is dy
    const bool any_db = b.db[0] || b.db[1];
    for (const void* q : {(const void*)b.dy, (const void*)b.pre[0], (const void*)b.pre[1], (const void*)b.dx,
                          (const void*)b.d[0], (const void*)b.d[1], (const void*)b.db[0], (const void*)b.db[1],
                          (const void*)workspace})
        if (!aligned16(q)) return BQ_ERR_ALIGN;
    if (M > 0 && K > 0 && !b.dx) return BQ_ERR_NULL;
    if (M > 0 && N > 0) {
        if (!b.dy || (!none && (!b.pre[0] || !b.d[0])) || (GLU && (!b.pre[1] || !b.d[1]))) return BQ_ERR_NULL;
        for (int i = 0; K > 0 && i < mats; ++i) {
            if (!w[i].wq || !w[i].scales) return BQ_ERR_NULL;
            if (!aligned16(w[i].wq) || !aligned16(w[i].scales) || !aligned16(w[i].biases)) return BQ_ERR_ALIGN;
        }
    }
    if ((M == 0 || K == 0) && (M == 0 || N == 0) && !(any_db && N > 0)) return BQ_OK;   // nothing to write
    int dev;
    DeviceInfo di;
    if ((s = current_device(&dev, &di)) != BQ_OK) return s;
    if (M == 0) {                                        // sums over no tokens
        for (int i = 0; i < mats; ++i)
            if (b.db[i] && cudaMemsetAsync(b.db[i], 0, (size_t)N * 2u, st) != cudaSuccess) return BQ_ERR_CUDA;
        return BQ_OK;
    }
    if (N == 0)                                          // a sum over no outputs
        return cudaMemsetAsync(b.dx, 0, (size_t)M * (size_t)K * 2u, st) == cudaSuccess ? BQ_OK : BQ_ERR_CUDA;
    EpiWs ws;
    if (!plan_backward(fmt, mats, M, N, K, di.num_sms, di.max_smem_optin, &ws)) return BQ_ERR_SHAPE;
    void* buf = nullptr;
    if ((s = epi_workspace(dev, st, workspace, workspace_bytes, ws.bytes, &buf)) != BQ_OK) return s;
    uint8_t* base = reinterpret_cast<uint8_t*>(buf);
    const bool pad = N % 8 != 0;
    uint16_t* padded[2] = {reinterpret_cast<uint16_t*>(base + ws.off_pad),
                           reinterpret_cast<uint16_t*>(base + ws.off_pad + up256((size_t)M * ws.pitch * 2u))};
    const bool fused = K > 0 && ws.fused;
    if (fused && none && !any_db && !pad) {
        if ((s = launch_scale_pack(true, w, mats, false, N, K, group_size, base, st)) != BQ_OK) return s;
    } else if (!none || any_db || pad) {
        EpiGradParams p;
        p.pack_blocks = 0;
        if (fused && (p.pack_blocks = (int)scale_pack_params(true, w, mats, false, N, K, group_size, base, &p.pack)) == 0)
            return BQ_ERR_SHAPE;
        p.dy = b.dy;
        p.z = b.pre[0];
        p.u = b.pre[1];
        p.dz = none ? nullptr : b.d[0];
        p.du = b.d[1];
        p.dz_pad = pad ? padded[0] : nullptr;
        p.du_pad = pad && GLU ? padded[1] : nullptr;
        p.part = any_db ? reinterpret_cast<float*>(base + ws.off_part) : nullptr;
        p.M = M;
        p.N = (int)N;
        p.pitch = (int)ws.pitch;
        p.rows_per_block = ws.rows_per_block;
        s = pad ? launch_epi_grad_v<GLU, 1>(p, act, ws.row_blocks, st) : launch_epi_grad_v<GLU, 8>(p, act, ws.row_blocks, st);
        if (s != BQ_OK) return s;
        if (any_db) {
            s = launch_pdl_dim(epi_bias_grad_kernel, dim3((unsigned)((N + 31) / 32), (unsigned)mats), 256, 0, st,
                               (const float*)p.part, b.db[0], b.db[1], (int)N, mats, ws.row_blocks);
            if (s != BQ_OK) return s;
        }
    }
    if (K == 0) return BQ_OK;
    const uint16_t* B[2] = {pad ? padded[0] : none ? b.dy : b.d[0], pad ? padded[1] : b.d[1]};
    EpiParams e;
    e.y = b.dx;
    if (fused)
        return launch_fused_pair_fmt<true, kEpiPlain>(fmt, di, dev, ws.pl, w, mats, B, N, K, M, pad ? ws.pitch : N,
                                                      group_size, e, base, base + ws.off_split, st);
    uint16_t* wb = reinterpret_cast<uint16_t*>(base);
    if ((s = dequant_rows(fmt, w, mats, wb, N, K, group_size, false, di, st)) != BQ_OK) return s;
    const uint16_t* A[2] = {wb, wb + (size_t)N * (size_t)K};
    return launch_pair<true, kEpiPlain>(di, dev, ws.pl, A, B, mats, K, K, M, N, pad ? ws.pitch : N, e,
                                        base + ws.off_split, st);
}

}  // namespace
}  // namespace bq
