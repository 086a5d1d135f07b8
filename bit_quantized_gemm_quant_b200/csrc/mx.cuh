// mx.cuh -- microscaled (MX) rows: conversions, quantizers and dequantizers.
//
// The formats are those of the OCP Microscaling Formats specification v1.0: blocks of 32
// consecutive elements of a row share a power of two X = 2^(byte - 127) (E8M0; byte 255 is
// NaN), and an element stands for X times its value in a small type:
//   MXFP8  E4M3: 1 sign, 4 exponent, 3 mantissa bits, largest value 448, no infinity
//   MXFP4  E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; two per byte, the first low
// The quantizers follow its section 6.3: X = 2^(floor(log2(amax)) - emax) with amax the
// block's largest magnitude and emax that of the type's largest power of two (8; 2), each
// element rounded to nearest, ties to even, and saturated.  What the specification leaves
// open: X is at least 2^-127 (so a block of zeros has byte 0), and a block that holds a NaN or an infinity
// becomes NaN as a whole (byte 255, codes 0): neither type could hold it element by element.
#pragma once

#include "common.cuh"

namespace bq {

constexpr uint32_t kMxNan = 255;

// Largest power of two of the element type, by its bits.
template <int BITS>
__host__ __device__ constexpr uint32_t mx_emax() { return BITS == 8 ? 8u : 2u; }

// The scale's byte from the bit pattern of amax (sign off).  The exponent field of a finite
// fp32 is floor(log2) + 127; of a subnormal one it is 0, where the floor at 2^-127 holds anyway.
template <int BITS>
BQ_DEVINL uint32_t mx_scale_byte(uint32_t amax_bits)
{
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? kMxNan : e > mx_emax<BITS>() ? e - mx_emax<BITS>() : 0u;
}

// 1 / X, 0 for a NaN scale.  Multiplying by it is exact (but for results below 2^-126, which
// round to the type's 0 either way).
BQ_DEVINL float mx_inverse(uint32_t byte) { return byte == kMxNan ? 0.0f : __uint_as_float((254u - byte) << 23); }

// X itself, as fp32 and as bf16 bits (exact: 2^-127 is subnormal in both).
BQ_DEVINL float mx_scale(uint32_t byte)
{
    return byte == kMxNan ? __uint_as_float(0x7FC00000u) : byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}
BQ_DEVINL uint32_t mx_scale_bf16(uint32_t byte) { return byte == kMxNan ? 0x7FC0u : byte == 0 ? 0x0040u : byte << 7; }

// Four values to E4M3 (first in the low byte), eight to E2M1 (first in the low nibble): to
// nearest even, saturated.
BQ_DEVINL uint32_t to_e4m3x4(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}" : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

BQ_DEVINL uint32_t to_e2m1x8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r) : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight E2M1 codes times X (s2: two of its bf16) to bf16 pairs.  A code's exponent and mantissa
// bits, put where bf16 has its lowest ones of each, are the value times 2^-126 (the subnormal
// code included), and its sign goes to the top: so a multiplication by 2^126 makes the value.  Two codes
// four places apart are made at a time, in the halves of a register; then pairs are put together.  (Bound by
// the ALU, which the left shifts and products leave alone: a table lookup by byte permutes, with
// the signs moved one by one, took twice its instructions, and 300 x 2048 x 8192's gradient 21 us.)
BQ_DEVINL void e2m1x8_scaled(uint32_t w, uint32_t s2, uint32_t (&out)[4])
{
    constexpr uint32_t kMag = 0x01C001C0u, kSign = 0x80008000u, kUp = 0x7E807E80u;      // 2^126 twice
    uint32_t v[4];
    v[0] = ((w << 6) & kMag) | ((w << 12) & kSign);
    v[1] = ((w << 2) & kMag) | ((w << 8) & kSign);
    v[2] = ((w >> 2) & kMag) | ((w << 4) & kSign);
    v[3] = ((w >> 6) & kMag) | (w & kSign);
#pragma unroll
    for (int n = 0; n < 4; ++n) v[n] = hmul2_bf16(hmul2_bf16(v[n], kUp), s2);
    out[0] = prmt(v[0], v[1], 0x5410u);
    out[1] = prmt(v[2], v[3], 0x5410u);
    out[2] = prmt(v[0], v[1], 0x7632u);
    out[3] = prmt(v[2], v[3], 0x7632u);
}

// 32 of them, as the pair products' other conversions write them.
BQ_DEVINL void deq_mx4_half(uint4 raw, uint32_t s2, uint32_t (&out)[16])
{
    const uint32_t words[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t v[4];
        e2m1x8_scaled(words[i], s2, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) out[4 * i + j] = v[j];
    }
}

// Two E4M3 codes to fp32 (exact).
BQ_DEVINL void e4m3x2_to_f32(uint32_t w, float& a, float& b)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
    const __half2 v = *reinterpret_cast<__half2*>(&h);
    a = __low2float(v);
    b = __high2float(v);
}

// The larger magnitudes of three; NaN if there is one.
BQ_DEVINL float amax3(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The bits of the largest magnitude of 8 values in each of 4 consecutive lanes (a block of
// 32); a NaN's if there is one.
BQ_DEVINL uint32_t block_amax_bits(const float (&v)[8])
{
    float a = amax3(amax3(v[0], v[1], v[2]), amax3(v[3], v[4], v[5]), amax3(v[6], v[7], v[7]));
    a = amax3(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1), a);
    a = amax3(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2), a);
    return __float_as_uint(a);
}

// 8 of the values of a block, whose other 24 are in the lanes' neighbours, to codes at
// element `at` (a multiple of 8) of the codes, and the block's scale.  `live`: this lane's values exist
// (all lanes of the warp come here).
template <int BITS>
BQ_DEVINL void mx_store8(const float (&v)[8], uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t at, bool live)
{
    const uint32_t byte = mx_scale_byte<BITS>(block_amax_bits(v));
    const uint64_t inv = f32x2_splat(mx_inverse(byte));
    const bool whole = byte != kMxNan;
    float t[8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f32x2_unpack(mul_f32x2(f32x2_pack(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1])), inv), t[2 * i], t[2 * i + 1]);
    if (!live) return;
    if constexpr (BITS == 8) {
        const uint32_t lo = to_e4m3x4(t[0], t[1], t[2], t[3]), hi = to_e4m3x4(t[4], t[5], t[6], t[7]);
        *reinterpret_cast<uint2*>(codes + at) = make_uint2(whole ? lo : 0u, whole ? hi : 0u);
    } else {
        const uint32_t c = to_e2m1x8(t);
        *reinterpret_cast<uint32_t*>(codes + at / 2) = whole ? c : 0u;
    }
    if ((at & 31) == 0) scales[at >> 5] = (uint8_t)byte;
}

// 8 consecutive elements as fp32.
template <bool F32>
BQ_DEVINL void load8(const void* x, int64_t at, float (&v)[8])
{
    if constexpr (F32) {
        const float* p = reinterpret_cast<const float*>(x) + at;
        const uint4 a = ldg_stream(p), b = ldg_stream(p + 4);
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    } else {
        const uint4 a = ldg_stream(reinterpret_cast<const uint16_t*>(x) + at);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

// ------------------------------------------------------------------ quantize
// A thread takes 8 elements, 4 threads a block, and kMxEach such pieces a CTA's width apart, all of whose
// loads are in flight before the first is used.  Rows are whole blocks, so the matrix is one run of `n`
// elements (a multiple of 32).  Bound by HBM.
constexpr int kMxEach = 4;
constexpr int64_t kMxSpan = 256 * 8 * kMxEach;               // elements of a CTA

template <int BITS, bool F32>
__global__ void __launch_bounds__(256)
mx_quantize_kernel(const void* __restrict__ x, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t n)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int64_t base = (int64_t)blockIdx.x * kMxSpan; base < n; base += (int64_t)gridDim.x * kMxSpan) {
        float v[kMxEach][8];
#pragma unroll
        for (int i = 0; i < kMxEach; ++i) {
            const int64_t at = base + (i * 256 + threadIdx.x) * 8;
            if (at < n) {
                load8<F32>(x, at, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < kMxEach; ++i) {
            const int64_t at = base + (i * 256 + threadIdx.x) * 8;
            mx_store8<BITS>(v[i], codes, scales, at, at < n);
        }
    }
}

// ------------------------------------------------------------------ dequantize
// out = bf16_rne(X * element): exact unless it leaves bf16's range (beyond it infinity, below 2^-133 to
// nearest even; a NaN scale gives NaN).  Work as in the quantizer.  Bound by HBM, mostly by the writes.
template <int BITS>
__global__ void __launch_bounds__(256)
mx_dequant_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, uint16_t* __restrict__ out, int64_t n)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int64_t base = (int64_t)blockIdx.x * kMxSpan; base < n; base += (int64_t)gridDim.x * kMxSpan) {
        uint2 w[kMxEach];
        uint32_t byte[kMxEach];
#pragma unroll
        for (int i = 0; i < kMxEach; ++i) {
            const int64_t at = base + (i * 256 + threadIdx.x) * 8;
            w[i] = make_uint2(0u, 0u);
            byte[i] = 0;
            if (at >= n) continue;
            if constexpr (BITS == 8) w[i] = __ldg(reinterpret_cast<const uint2*>(codes + at));
            else w[i].x = __ldg(reinterpret_cast<const uint32_t*>(codes + at / 2));
            byte[i] = __ldg(scales + (at >> 5));
        }
#pragma unroll
        for (int i = 0; i < kMxEach; ++i) {
            const int64_t at = base + (i * 256 + threadIdx.x) * 8;
            if (at >= n) continue;
            uint32_t o[4];
            if constexpr (BITS == 4) {
                const uint32_t s = mx_scale_bf16(byte[i]) * 0x10001u;
                e2m1x8_scaled(w[i].x, s, o);
            } else {
                const float s = mx_scale(byte[i]);
                float v[8];
                e4m3x2_to_f32(w[i].x, v[0], v[1]);
                e4m3x2_to_f32(w[i].x >> 16, v[2], v[3]);
                e4m3x2_to_f32(w[i].y, v[4], v[5]);
                e4m3x2_to_f32(w[i].y >> 16, v[6], v[7]);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2_rn(__fmul_rn(v[2 * j], s), __fmul_rn(v[2 * j + 1], s));
            }
            *reinterpret_cast<uint4*>(out + at) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// ------------------------------------------------------------------ longer rows
// Rows of 16-byte units to longer ones, zeros behind: [rows][in] to [rows][out] units.  (Codes of W for
// products whose copies want rows of whole 128 codes.)  Blocks of 256 threads, kMxPadSpan units each,
// of a launch with other work (mx_pack_kernel).
struct MxPadParams {
    const uint4* from;
    uint4* to;
    int64_t rows;
    int in, out;
};
constexpr int kMxPadSpan = 1024;

BQ_DEVINL void mx_pad_block(const MxPadParams& p, int64_t block)
{
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t i = block * kMxPadSpan + 256 * j + threadIdx.x, r = i / p.out;
        const int c = (int)(i - r * p.out);
        v[j] = r < p.rows && c < p.in ? ldg_stream(p.from + r * p.in + c) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t i = block * kMxPadSpan + 256 * j + threadIdx.x;
        if (i < p.rows * p.out) p.to[i] = v[j];
    }
}

}  // namespace bq
