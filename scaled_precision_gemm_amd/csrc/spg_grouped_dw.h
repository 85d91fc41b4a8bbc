// Internal declarations of the experts' weight gradients.
#pragma once

#include "spg_common.h"

namespace spg {

struct GroupedDwArgs {
    const uint16_t *dy, *x;             // [R, N], [x_rows, K], row strides ldy, ldx
    const int32_t *offsets;             // [E + 1]
    const int32_t *row_index;           // [R] or null
    const void *add;                    // [E, N, K] in the output's type or null, row stride lda, expert stride stride_a
    void *out;                          // [E, N, K], ldo, stride_o
    float *partials;                    // slices > 1: [tiles, slices, tile_n, 256]
    int64_t R, x_rows, N, K, ldy, ldx, lda, stride_a, ldo, stride_o;
    int32_t E, out_fp32;
    int32_t lines;                      // rows of out and add begin on 128-byte lines
    int32_t slices;                     // parts of every expert's rows, summed by a second launch
    int32_t tile_n;                     // tiles of tile_n (128 or 256) n x 256 k
    uint32_t tiles_n, tiles_k;          // tiles of one expert
    int32_t unit_n, unit_k;             // dealt to an XCD together: tiles_k / 2^unit_k tiles of 2^unit_n rows of tiles
    FastDiv div_k, div_n, div_slice;    // by tiles_k, tiles_n, slices
    FastDiv div_width;                  // by tiles_k / 2^unit_k
};
constexpr int kDwTile = 256;             // k of a tile
constexpr int kDwMaxSlices = 16;
hipError_t launch_grouped_dw(const GroupedDwArgs &a, hipStream_t s);

}  // namespace spg
