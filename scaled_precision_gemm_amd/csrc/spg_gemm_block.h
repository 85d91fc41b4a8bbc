// Internal declarations of the block-scaled FP8 products (E4M3 codes, one
// fp32 scale per 128 K-elements of a token row and per 128 x 128 block of
// weights), dense and per expert.
#pragma once

#include "spg_common.h"

namespace spg {

// GemmArgs first: it starts the kernel-argument segment (see out_at).
// Scale planes: sa [groups, a_rows] (group-major; batch entries
// g.sa_bstride floats apart; experts: 0), sw with the block of W row n and K
// group k at (n / 128) * sw_rs + k * sw_gs (batch entries / experts
// g.sw_bstride apart).  A stride of 0 is one plane for all, whatever the
// codes' strides are.
struct BlockArgs {
    GemmArgs g;
    int64_t a_rows;           // rows of A and of its scale plane
    int32_t sw_rs, sw_gs;
    int32_t groups;           // ceil(K / 128)
    int32_t sw_words;         // floats of one weight matrix's scale plane
    // Experts' products (experts > 0): rows [offsets[e], offsets[e + 1]) of
    // the output are expert e's; row r is made from A row row_index[r] (r
    // when null).  g.M is the number of output rows.
    const int32_t *offsets;
    const int32_t *row_index;
    int32_t experts;
};

// Tiles of 256 or 128 token rows x 256 weight rows.
hipError_t launch_gemm_block_tiles(const BlockArgs &a, int bm, int64_t workgroups, hipStream_t s);
// 16- or 32-row tiles (experts: 16) x narrow_cols() output columns.
hipError_t launch_gemm_block_narrow(const BlockArgs &a, int bm, int64_t workgroups, hipStream_t s);
// Sum of the K slices' partial tiles and the epilogue.
hipError_t launch_gemm_block_reduce(const BlockArgs &a, int bm, hipStream_t s);
hipError_t launch_quantize_block128(const uint16_t *x, int64_t batch, int64_t rows, int64_t K, int64_t ldx,
                                    int64_t bstride, uint8_t *q, int64_t ldq, int64_t qbstride, float *scale,
                                    int tiling, hipStream_t s);

}  // namespace spg
