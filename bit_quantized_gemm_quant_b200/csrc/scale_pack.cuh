// scale_pack.cuh -- the scales of quantized weights laid out for the fused pair products
// (tc_fused_pair.cuh): words of 32 weights, [column block of 128][row][4]; forward the
// rows are the product's tile rows (glu: interleaved, see epi_out_row), for the gradient
// those of the matrix, one matrix after the other.  Rows and columns are padded to whole
// tiles with weights of 0.  A word holds scale and bias (bf16), or Q4_0's d as d_hi + d_lo
// (see gemv.cuh).
//
// A block takes 32 rows x 2048 columns through shared memory: reads run along the rows of
// the scales, writes along the rows of the result.  1.6 us by itself for 704 x 1024, latency
// throughout; 12288 x 4096 reads 3 to 6 MB and writes 6.
#pragma once

#include "common.cuh"

namespace bq {

struct ScalePackParams {
    const uint16_t* scales[2];
    const uint16_t* biases[2];     // NULL: Q4_0
    uint32_t* out;
    int N, K, gs_shift, interleave;
    int cols;                      // padded columns
    int row_chunks, col_chunks;    // blocks per matrix
    int64_t pack_rows, pack_mat;   // rows per column block; gradient: words per matrix
};

constexpr int kScalePackWords = 32 * 65;       // shared memory of a block

BQ_DEVINL void scale_pack_block(const ScalePackParams& p, uint32_t* smem, int block)
{
    const int per_mat = p.row_chunks * p.col_chunks, mat = block >= per_mat;
    block -= mat ? per_mat : 0;
    const int n0 = block % p.row_chunks * 32, k0 = block / p.row_chunks * 2048;
    const int per_row = p.K >> p.gs_shift;
    const uint16_t* sc = mat ? p.scales[1] : p.scales[0];
    const uint16_t* bi = mat ? p.biases[1] : p.biases[0];
    // all loads in flight before the first is used
    constexpr int kEach = 32 * 64 / 256;
    uint32_t v[kEach], w[kEach];
    const int h = threadIdx.x & 63, k = k0 + 32 * h, r0 = threadIdx.x >> 6;
    const int64_t g0 = (int64_t)(n0 + r0) * per_row + (k >> p.gs_shift);
#pragma unroll
    for (int i = 0; i < kEach; ++i) v[i] = n0 + r0 + 4 * i < p.N && k < p.K ? __ldg(sc + (g0 + (int64_t)(4 * i) * per_row)) : 0u;
    if (bi) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) w[i] = n0 + r0 + 4 * i < p.N && k < p.K ? __ldg(bi + (g0 + (int64_t)(4 * i) * per_row)) : 0u;
    } else {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const float d = f16_bits_to_f32((uint16_t)v[i]);
            v[i] = f32_to_bf16_bits(d);
            w[i] = f32_to_bf16_bits(__fsub_rn(d, bf16_bits_to_f32(v[i])));
        }
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) smem[(r0 + 4 * i) * 65 + h] = v[i] | w[i] << 16;
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * 16; i += 256) {
        const int r = i & 31, c = i >> 5, n = n0 + r;
        const int64_t blk = k0 / 128 + c;
        if (blk * 128 >= p.cols) continue;
        const int64_t row = p.interleave ? 32 * (int64_t)(n >> 4) + (n & 15) + 16 * mat : n;
        if (row >= p.pack_rows) continue;
        const uint32_t* s = smem + r * 65 + 4 * c;
        *reinterpret_cast<uint4*>(p.out + mat * p.pack_mat + (blk * p.pack_rows + row) * 4) = make_uint4(s[0], s[1], s[2], s[3]);
    }
}

__global__ void __launch_bounds__(256) scale_pack_kernel(const __grid_constant__ ScalePackParams p)
{
    __shared__ uint32_t smem[kScalePackWords];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    scale_pack_block(p, smem, blockIdx.x);
}

}  // namespace bq
