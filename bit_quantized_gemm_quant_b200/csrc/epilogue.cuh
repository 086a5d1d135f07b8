// epilogue.cuh -- what a product with quantized weights does with its fp32 sums
// before they are rounded: bias, activation, residual and gate, the activations'
// derivatives, and the elementwise half of the backward pass.
//
//   act:  z = sum + bias,  y = residual + act(z)
//   glu:  g = sum_g + gate_bias,  u = sum_u + up_bias,  h = act(g) u
//
// All arithmetic is fp32; y, h and the saved z, g, u are each rounded once, to
// bf16, from the unrounded values (h does not see the rounding of a saved g).
#pragma once

#include "common.cuh"
#include "scale_pack.cuh"

namespace bq {

enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

// What a kernel's epilogue computes: kEpiPlain stores the sums (quant_matmul),
// kEpiAct and kEpiGlu the two forms above.
enum : int { kEpiPlain = 0, kEpiAct = 1, kEpiGlu = 2 };

// Operands of an epilogue; [M][N] arrays share the output's layout.  residual may
// be y itself: each element is read and then written by one thread.
struct EpiParams {
    const uint16_t* bias = nullptr;      // act: [N] or NULL; glu: gate_bias
    const uint16_t* bias2 = nullptr;     // glu: up_bias
    const uint16_t* res = nullptr;       // act: [M][N] or NULL
    uint16_t* y = nullptr;               // y or h
    uint16_t* pre = nullptr;             // saved z or g, or NULL
    uint16_t* pre2 = nullptr;            // glu: saved u (with pre)
    int act = kActNone;
};

// 2^x and 1 / x by the hardware's approximations (each within 2^-22 of the value; results below
// the normal range become 0), and e^x through the first: one multiply and one special-function
// instruction, without the range scaling of the library functions.  x log2(e) is rounded
// before the exponential, so e^x is within (|x| + 4) 2^-23 of itself: 2^-21 near 0, 2^-16.5 at
// the ends of the range, |x| = 87, far below a bf16 rounding throughout.  The gelu gradient of
// 2048 x 12288 is bound by issue.
BQ_DEVINL float exp_approx(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}

BQ_DEVINL float rcp_approx(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + e^-z); 0 where e^-z overflows.
BQ_DEVINL float sigmoid_f(float z) { return rcp_approx(1.0f + exp_approx(-z)); }

// gelu_tanh through 0.5 (1 + tanh a) = sigmoid(2 a), a = sqrt(2/pi) (z + 0.044715 z^3).
constexpr float kGeluTanhA = 1.5957691216057308f;        // 2 sqrt(2/pi)
constexpr float kGeluTanhB = 0.044715f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// The normal distribution function.  With t = 1 / (1 + 0.35 |z|) the tail 1 - Phi(|z|) is
// t q(t) e^(-z^2 / 2): e^(x^2 / 2) (1 - Phi(x)) falls like 1 / x, as t does, and q is the polynomial
// of degree 6 whose largest error, relative to the tail and weighted by the exponential's own
// (1.5 z^2 / 2 + 4) 2^-23, is least over 0 <= x <= 13.3 (a linear program over 6000 points).
// Evaluated in fp32 t q(t) is within 2e-6 of the tail at |z| <= 3 and within 7.2e-6 at 13.3,
// where the density leaves the normal range; Phi is within 4e-7 everywhere.  Taking the tail
// itself keeps Phi(z) for z << 0 free of cancellation.  (A fit of the absolute error alone,
// erf to 1.5e-7 with degree 4, is off by 0.2% of the tail at z = -5 and by 2% at -10, more than
// a bf16 rounding; 12288 x 4096, 512 tokens take 49.8 us with it and 50.2 with this one.)  `e`
// returns e^(-z^2 / 2), the density times sqrt(2 pi).  (erfcf in this place made the epilogue of
// that product take 19 us.)
BQ_DEVINL float normal_cdf(float z, float& e)
{
    const float t = rcp_approx(fmaf(0.35f, fabsf(z), 1.0f));
    e = exp_approx(-0.5f * z * z);
    float q = fmaf(t, 0.0462969691f, -0.191046044f);
    q = fmaf(t, q, 0.221504465f);
    q = fmaf(t, q, 0.00059047807f);
    q = fmaf(t, q, 0.146686837f);
    q = fmaf(t, q, 0.136131853f);
    q = fmaf(t, q, 0.139835477f) * t * e;
    return z < 0.0f ? q : 1.0f - q;
}

template <int ACT>
BQ_DEVINL float act_f(float z)
{
    if constexpr (ACT == kActRelu) return z < 0.0f ? 0.0f : z;                    // NaN stays NaN
    if constexpr (ACT == kActGelu) {
        float e;
        return z * normal_cdf(z, e);
    }
    if constexpr (ACT == kActGeluTanh) return z * sigmoid_f(kGeluTanhA * z * fmaf(kGeluTanhB * z, z, 1.0f));
    if constexpr (ACT == kActSilu) return z * sigmoid_f(z);
    return z;
}

// The derivative; where the sigmoid is 0 or 1 (or the density 0) in fp32 the term
// it multiplies is dropped, so that large |z| gives 0 or 1 and not inf * 0.
template <int ACT>
BQ_DEVINL float dact_f(float z)
{
    if constexpr (ACT == kActRelu) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    if constexpr (ACT == kActGelu) {
        float e;
        const float c = normal_cdf(z, e);
        return e == 0.0f ? c : fmaf(kInvSqrt2Pi * z, e, c);
    }
    if constexpr (ACT == kActGeluTanh) {
        const float p = sigmoid_f(kGeluTanhA * z * fmaf(kGeluTanhB * z, z, 1.0f)), t = p * (1.0f - p);
        return t == 0.0f ? p : fmaf(z * t, kGeluTanhA * fmaf(3.0f * kGeluTanhB * z, z, 1.0f), p);
    }
    if constexpr (ACT == kActSilu) {
        const float p = sigmoid_f(z), t = p * (1.0f - p);
        return t == 0.0f ? p : fmaf(z, t, p);
    }
    return 1.0f;
}

// act over an array, the choice made once for all of it.
template <int CNT>
BQ_DEVINL void act_n(float (&z)[CNT], int act)
{
    switch (act) {
    case kActRelu:
#pragma unroll
        for (int i = 0; i < CNT; ++i) z[i] = act_f<kActRelu>(z[i]);
        break;
    case kActGelu:
#pragma unroll
        for (int i = 0; i < CNT; ++i) z[i] = act_f<kActGelu>(z[i]);
        break;
    case kActGeluTanh:
#pragma unroll
        for (int i = 0; i < CNT; ++i) z[i] = act_f<kActGeluTanh>(z[i]);
        break;
    case kActSilu:
#pragma unroll
        for (int i = 0; i < CNT; ++i) z[i] = act_f<kActSilu>(z[i]);
        break;
    default: break;
    }
}

// One output element: its operands, which can be loaded ahead of the sums, and the
// result from the sums (glu: s and s2).
struct EpiOperands {
    float b, b2, r;
};

template <int EPI>
BQ_DEVINL EpiOperands epi_operands(const EpiParams& e, int64_t m, int n, int64_t N)
{
    EpiOperands p;
    p.b = e.bias ? bf16_bits_to_f32(e.bias[n]) : 0.0f;
    p.b2 = EPI == kEpiGlu && e.bias2 ? bf16_bits_to_f32(e.bias2[n]) : 0.0f;
    p.r = EPI == kEpiAct && e.res ? bf16_bits_to_f32(e.res[m * N + n]) : 0.0f;
    return p;
}

template <int EPI>
BQ_DEVINL void epi_finish(const EpiParams& e, const EpiOperands& p, float s, float s2, int64_t m, int n, int64_t N)
{
    const int64_t o = m * N + n;
    float z[1] = {s + p.b};
    if constexpr (EPI == kEpiGlu) {
        const float u = s2 + p.b2;
        if (e.pre) {
            e.pre[o] = (uint16_t)f32_to_bf16_bits(z[0]);
            e.pre2[o] = (uint16_t)f32_to_bf16_bits(u);
        }
        act_n<1>(z, e.act);
        e.y[o] = (uint16_t)f32_to_bf16_bits(z[0] * u);
    } else {
        if (e.pre) e.pre[o] = (uint16_t)f32_to_bf16_bits(z[0]);
        act_n<1>(z, e.act);
        e.y[o] = (uint16_t)f32_to_bf16_bits(e.res ? z[0] + p.r : z[0]);
    }
}

template <int EPI>
BQ_DEVINL void epi_one(const EpiParams& e, float s, float s2, int64_t m, int n, int64_t N)
{
    epi_finish<EPI>(e, epi_operands<EPI>(e, m, n, N), s, s2, m, n, N);
}

// The output row (column n of y) that row `r` of a weight tile stands for.  glu
// tiles hold 16 gate rows, then the 16 up rows of the same outputs, and so on, so
// that both sums of an output sit in one warp's 32 tensor-memory lanes.
template <int EPI>
__host__ __device__ constexpr int epi_tile_rows(int rows) { return EPI == kEpiGlu ? rows / 2 : rows; }

template <int EPI>
BQ_DEVINL int epi_out_row(int r) { return EPI == kEpiGlu ? 16 * (r >> 5) + (r & 15) : r; }

// Per-thread state of a tensor-core tile's epilogue: this thread's output row.
template <int EPI>
struct EpiRow {
    int n;
    bool ok;
    float b, b2;
};

template <int EPI>
BQ_DEVINL EpiRow<EPI> epi_row(const EpiParams& e, int n, int N)
{
    EpiRow<EPI> r;
    r.n = n;
    r.ok = n < N;
    r.b = r.ok && e.bias ? bf16_bits_to_f32(__ldg(e.bias + n)) : 0.0f;
    r.b2 = 0.0f;
    if constexpr (EPI == kEpiGlu) r.b2 = r.ok && e.bias2 ? bf16_bits_to_f32(__ldg(e.bias2 + n)) : 0.0f;
    return r;
}

// Consecutive tokens (mb ...) of one tile row from a tensor-memory load: 16 with glu, else
// 8.  The whole warp calls it: with glu, lanes l and l + 16 hold the gate and the up sum
// of one output and trade every second token by one shuffle, so that each lane ends with
// both sums of 8 outputs.  FULL: all the tokens exist.  (The code shares the instruction
// cache with the dequantization: at 12288 x 4096, 512 tokens, act took 71 us with 8
// tokens at a time, 75 with 16, 84 with 16 and a FULL copy; glu, whose activations are
// fewer per token, was fastest with 16 and both copies.)
template <int EPI> constexpr int kEpiTokens = EPI == kEpiGlu ? 16 : 8;

template <int EPI, bool FULL, int T>
BQ_DEVINL void epi_store_tokens(const EpiParams& e, const EpiRow<EPI>& r, const uint32_t (&v)[T], int mb, int M, int64_t N)
{
    if constexpr (EPI == kEpiGlu) {
        const int up = (threadIdx.x >> 4) & 1;
        float g[T / 2], u[T / 2];
#pragma unroll
        for (int j = 0; j < T / 2; ++j) {
            const uint32_t mine = up ? v[2 * j + 1] : v[2 * j];
            const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? v[2 * j] : v[2 * j + 1], 16);
            g[j] = __uint_as_float(up ? got : mine) + r.b;
            u[j] = __uint_as_float(up ? mine : got) + r.b2;
        }
        if (!r.ok) return;
        const int m = mb + up;
        int64_t o = (int64_t)m * N + r.n;
        if (e.pre) {
            int64_t q = o;
#pragma unroll
            for (int j = 0; j < T / 2; ++j, q += 2 * N)
                if (FULL || m + 2 * j < M) {
                    e.pre[q] = (uint16_t)f32_to_bf16_bits(g[j]);
                    e.pre2[q] = (uint16_t)f32_to_bf16_bits(u[j]);
                }
        }
        act_n<T / 2>(g, e.act);
#pragma unroll
        for (int j = 0; j < T / 2; ++j, o += 2 * N)
            if (FULL || m + 2 * j < M) e.y[o] = (uint16_t)f32_to_bf16_bits(g[j] * u[j]);
    } else {
        if (!r.ok) return;
        int64_t o = (int64_t)mb * N + r.n;
        float z[T];
#pragma unroll
        for (int j = 0; j < T; ++j) z[j] = __uint_as_float(v[j]) + r.b;
        if constexpr (EPI == kEpiAct) {
            uint32_t q[T];
            if (e.res) {
                int64_t i = o;
#pragma unroll
                for (int j = 0; j < T; ++j, i += N) q[j] = FULL || mb + j < M ? e.res[i] : 0u;
            }
            if (e.pre) {
                int64_t i = o;
#pragma unroll
                for (int j = 0; j < T; ++j, i += N)
                    if (FULL || mb + j < M) e.pre[i] = (uint16_t)f32_to_bf16_bits(z[j]);
            }
            act_n<T>(z, e.act);
            if (e.res) {
#pragma unroll
                for (int j = 0; j < T; ++j) z[j] += bf16_bits_to_f32(q[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < T; ++j, o += N)
            if (FULL || mb + j < M) e.y[o] = (uint16_t)f32_to_bf16_bits(z[j]);
    }
}

template <int EPI, int T>
BQ_DEVINL void epi_store(const EpiParams& e, const EpiRow<EPI>& r, const uint32_t (&v)[T], int mb, int M, int64_t N)
{
    if (EPI == kEpiGlu && mb + T <= M)                    // warp-uniform
        epi_store_tokens<EPI, true, T>(e, r, v, mb, M, N);
    else
        epi_store_tokens<EPI, false, T>(e, r, v, mb, M, N);
}

// How the pair products cut their work: tiles [0, dp_tiles) whole, pair i taking tiles
// i, i + pairs, ...; the blocks of the other `tail` tiles, in order, are dealt to the
// first `tail_pairs` pairs in equal consecutive ranges (tail <= tail_pairs, so a range
// touches at most two tiles).  So the last round fills all pairs whatever the number of
// tiles: 128 tiles on 74 pairs cost 1.73 tiles' time instead of 2.  A range's part of a
// tile is an fp32 partial tile in slot 2 i + (0 or 1).
struct TailSplit {
    int dp_tiles, tail, tail_pairs;
    int blocks;                                    // 64-element blocks per tile
    __host__ __device__ int64_t range_begin(int i) const { return (int64_t)i * tail * blocks / tail_pairs; }
};

// Four outputs n0 .. n0 + 3 (n0 a multiple of 4) of token m from their sums; 8-byte stores
// where rows start on 8 bytes.
template <int EPI>
BQ_DEVINL void epi_four(const EpiParams& e, const float (&s)[4], const float (&s2)[4], int64_t m, int n0, int N)
{
    if ((N & 3) != 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (n0 + k < N) epi_one<EPI>(e, s[k], s2[k], m, n0 + k, N);
        return;
    }
    const int64_t o = m * N + n0;
    auto four = [](const uint16_t* q, float (&v)[4]) {
        const uint2 w = *reinterpret_cast<const uint2*>(q);
        v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xFFFF0000u);
        v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xFFFF0000u);
    };
    auto put = [](uint16_t* q, const float (&v)[4]) {
        *reinterpret_cast<uint2*>(q) = make_uint2(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]));
    };
    float z[4] = {s[0], s[1], s[2], s[3]}, v[4];
    if (EPI != kEpiPlain && e.bias) {
        four(e.bias + n0, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] += v[k];
    }
    if constexpr (EPI == kEpiGlu) {
        float u[4] = {s2[0], s2[1], s2[2], s2[3]};
        if (e.bias2) {
            four(e.bias2 + n0, v);
#pragma unroll
            for (int k = 0; k < 4; ++k) u[k] += v[k];
        }
        if (e.pre) {
            put(e.pre + o, z);
            put(e.pre2 + o, u);
        }
        act_n<4>(z, e.act);
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] *= u[k];
    } else if constexpr (EPI == kEpiAct) {
        if (e.pre) put(e.pre + o, z);
        act_n<4>(z, e.act);
        if (e.res) {
            four(e.res + o, v);
#pragma unroll
            for (int k = 0; k < 4; ++k) z[k] += v[k];
        }
    }
    put(e.y + o, z);
}

// Sums the partial tiles of the tail in the order of their blocks and applies the
// epilogue.  Partials: [slot][token of the tile (bn)][row of the tile (256)].  A block
// takes kReduceTokens tokens of one tile, a thread 4 outputs of a token, one round of its loop
// (glu, whose tiles hold half as many outputs: half of the threads); a tile's partials (3 to 6 as a rule) are loaded four at a time.  Bound by L2, which still
// holds what the product has just written.  (Gated gradient of 2 x 8192 x 2048, 512 tokens:
// 46.1 us with 8 tokens a block, 44.8 with 4, 45.7 with 2; of 2 x 12288 x 4096, 2048 tokens:
// 326, 327, 331.)
constexpr int kReduceTokens = 4;

template <int EPI>
__global__ void __launch_bounds__(256)
epi_reduce_kernel(const float* __restrict__ ws, EpiParams e, int M, int N, int bn, int m_tiles, TailSplit t)
{
    constexpr int kGroups = epi_tile_rows<EPI>(256) / 4;              // 4-output groups per token
    const int chunks = (bn + kReduceTokens - 1) / kReduceTokens;
    const int j = (int)blockIdx.x / chunks, c0 = ((int)blockIdx.x - j * chunks) * kReduceTokens;
    const int tok0 = ((t.dp_tiles + j) % m_tiles) * bn;
    const int64_t out0 = (int64_t)((t.dp_tiles + j) / m_tiles) * epi_tile_rows<EPI>(256);
    // the ranges that share the tile: from the last one that begins at or before it
    const int64_t all = (int64_t)t.tail * t.blocks, begin = (int64_t)j * t.blocks, end = begin + t.blocks;
    const int p0 = (int)(((begin + 1) * t.tail_pairs + all - 1) / all) - 1;
    const int p1 = (int)((end * t.tail_pairs + all - 1) / all);      // ranges [p0, p1): the next begins at or past the end
    const int64_t slot = (int64_t)bn * 256;
    const float* first = ws + (2 * p0 + (t.range_begin(p0) < begin ? 1 : 0)) * slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll 2
    for (int i = threadIdx.x; i < kReduceTokens * kGroups; i += 256) {
        const int m = c0 + i / kGroups, r4 = i % kGroups * 4;
        const int64_t n0 = out0 + r4;
        if (m >= bn || tok0 + m >= M || n0 >= N) continue;
        const int64_t at = (int64_t)m * 256 + (EPI == kEpiGlu ? 32 * (r4 >> 4) + (r4 & 15) : r4);
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
        for (int p = p0; p < p1; p += 4) {
            float4 a[4], b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                a[k] = b[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (p + k < p1) {
                    const float* src = (p + k == p0 ? first : ws + 2 * (p + k) * slot) + at;
                    a[k] = *reinterpret_cast<const float4*>(src);
                    if constexpr (EPI == kEpiGlu) b[k] = *reinterpret_cast<const float4*>(src + 16);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                s[0] += a[k].x; s[1] += a[k].y; s[2] += a[k].z; s[3] += a[k].w;
                if constexpr (EPI == kEpiGlu) { s2[0] += b[k].x; s2[1] += b[k].y; s2[2] += b[k].z; s2[3] += b[k].w; }
            }
        }
        epi_four<EPI>(e, s, s2, tok0 + m, (int)n0, N);
    }
}

// K = 0: every sum is empty.
template <int EPI>
__global__ void __launch_bounds__(256) epi_empty_kernel(EpiParams e, int64_t M, int N)
{
    const int64_t total = M * N;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x)
        epi_one<EPI>(e, 0.0f, 0.0f, i / N, (int)(i % N), N);
}

// ------------------------------------------------------------------ backward, elementwise half
// act:  dz = dy act'(z);   glu:  dg = dh u act'(g),  du = dh act(g)
// with the column sums over tokens (the biases' gradients) when asked for: they are
// sums of the unrounded fp32 values, per block of rows here and over the blocks in
// epi_bias_grad_kernel, both in a fixed order.
//
// Bound by HBM: act reads 2 and writes 1 bf16 [M][N] array, glu reads 3 and writes
// 2.  A block takes 32 x V columns; its 8 warps take every 8th row, R of them at a time.
// V = 8 (16-byte loads) when every row starts on 16 bytes, else 1.  The first `pack_blocks`
// blocks lay out the weights' scales for the product that follows (scale_pack.cuh), which
// would otherwise be a kernel and its start-up latency ahead of this one.
struct EpiGradParams {
    const uint16_t* dy;
    const uint16_t* z;         // act: z; glu: g
    const uint16_t* u;         // glu
    uint16_t* dz;              // act: dz; glu: dg
    uint16_t* du;              // glu
    uint16_t* dz_pad;          // copies with rows of `pitch` elements for the product (N % 8 != 0), or NULL
    uint16_t* du_pad;
    float* part;               // [row blocks][1 or 2][N] column sums, or NULL
    int64_t M;
    int N, pitch, rows_per_block;
    int col_blocks, pack_blocks;
    ScalePackParams pack;
};

template <bool GLU, int ACT, int V>
__global__ void __launch_bounds__(256) epi_grad_kernel(const __grid_constant__ EpiGradParams p)
{
    __shared__ uint32_t smem[kScalePackWords > 256 * V ? kScalePackWords : 256 * V];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if ((int)blockIdx.x < p.pack_blocks) {
        scale_pack_block(p.pack, smem, blockIdx.x);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cb = ((int)blockIdx.x - p.pack_blocks) % p.col_blocks, rb = ((int)blockIdx.x - p.pack_blocks) / p.col_blocks;
    const int n = (cb * 32 + lane) * V;                // N is below 2^30
    const int64_t m_end = min(p.M, (int64_t)(rb + 1) * p.rows_per_block);
    float sz[V], su[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sz[i] = su[i] = 0.0f;
    // R rows at a time, all of their loads in flight before the first is used
    constexpr int R = V == 8 ? 2 : 4;
    const uint16_t* __restrict__ dy = p.dy;
    const uint16_t* __restrict__ z = p.z;
    const uint16_t* __restrict__ u = p.u;
    if (n < p.N) {
        for (int64_t m0 = (int64_t)rb * p.rows_per_block + warp; m0 < m_end; m0 += 8 * R) {
            __align__(16) uint16_t vd[R][V], vz[R][V], vu[R][V];
#pragma unroll
            for (int q = 0; q < R; ++q) {
                const int64_t o = min(m0 + 8 * q, m_end - 1) * p.N + n;
                if constexpr (V == 8) {
                    *reinterpret_cast<uint4*>(vd[q]) = *reinterpret_cast<const uint4*>(dy + o);
                    if constexpr (ACT != kActNone || GLU) *reinterpret_cast<uint4*>(vz[q]) = *reinterpret_cast<const uint4*>(z + o);
                    if constexpr (GLU) *reinterpret_cast<uint4*>(vu[q]) = *reinterpret_cast<const uint4*>(u + o);
                } else {
                    vd[q][0] = dy[o];
                    if constexpr (ACT != kActNone || GLU) vz[q][0] = z[o];
                    if constexpr (GLU) vu[q][0] = u[o];
                }
            }
#pragma unroll
            for (int q = 0; q < R; ++q) {
                const int64_t m = m0 + 8 * q;
                if (m >= m_end) break;
                const int64_t o = m * p.N + n;
                float oz[V], ou[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = bf16_bits_to_f32(vd[q][i]);
                    oz[i] = d;
                    if constexpr (GLU) {
                        const float g = bf16_bits_to_f32(vz[q][i]);
                        oz[i] = d * bf16_bits_to_f32(vu[q][i]) * dact_f<ACT>(g);
                        su[i] += ou[i] = d * act_f<ACT>(g);
                    } else if constexpr (ACT != kActNone) {
                        oz[i] = d * dact_f<ACT>(bf16_bits_to_f32(vz[q][i]));
                    }
                    sz[i] += oz[i];
                }
                if constexpr (V == 8) {
                    auto put = [](uint16_t* to, const float (&v)[V]) {
                        *reinterpret_cast<uint4*>(to) = make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]),
                                                                   pack_bf16x2_rn(v[4], v[5]), pack_bf16x2_rn(v[6], v[7]));
                    };
                    if (p.dz) put(p.dz + o, oz);
                    if constexpr (GLU) put(p.du + o, ou);
                } else {
                    const uint16_t zb = (uint16_t)f32_to_bf16_bits(oz[0]);
                    if (p.dz) p.dz[o] = zb;
                    if (p.dz_pad) p.dz_pad[m * p.pitch + n] = zb;
                    if constexpr (GLU) {
                        const uint16_t ub = (uint16_t)f32_to_bf16_bits(ou[0]);
                        p.du[o] = ub;
                        if (p.du_pad) p.du_pad[m * p.pitch + n] = ub;
                    }
                }
            }
        }
    }
    if (p.part) {
        float(*red)[32 * V] = reinterpret_cast<float(*)[32 * V]>(smem);
#pragma unroll
        for (int k = 0; k < (GLU ? 2 : 1); ++k) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < V; ++i) red[warp][lane * V + i] = k ? su[i] : sz[i];
            __syncthreads();
            for (int c = threadIdx.x; c < 32 * V; c += 256) {
                const int64_t col = (int64_t)cb * 32 * V + c;
                if (col >= p.N) break;
                float s = 0.0f;
#pragma unroll
                for (int w = 0; w < 8; ++w) s += red[w][c];
                p.part[((int64_t)rb * (GLU ? 2 : 1) + k) * p.N + col] = s;
            }
        }
    }
}

// db[k][n] = bf16(sum over row blocks of part[block][k][n]): a block takes 32 columns, its
// 8 warps every eighth row block; their sums are added in warp order.
__global__ void __launch_bounds__(256)
epi_bias_grad_kernel(const float* __restrict__ part, uint16_t* __restrict__ db0, uint16_t* __restrict__ db1, int N,
                     int kinds, int blocks)
{
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = blockIdx.y;
    const int64_t n = (int64_t)blockIdx.x * 32 + lane;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    float s = 0.0f;
    if (n < N) {
#pragma unroll 4
        for (int b = warp; b < blocks; b += 8) s += part[((int64_t)b * kinds + k) * N + n];
    }
    red[warp][lane] = s;
    __syncthreads();
    uint16_t* o = k ? db1 : db0;
    if (warp == 0 && n < N && o) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += red[w][lane];
        o[n] = (uint16_t)f32_to_bf16_bits(t);
    }
}

}  // namespace bq
