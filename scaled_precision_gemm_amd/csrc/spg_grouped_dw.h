// Internal declarations of the experts' weight gradients.
#pragma once

#include "spg_api_checks.h"

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

// ---- plan and dealing (in the host's build as well) -----------------------------
// Tiles of 256 n x 256 k; 128 n where those would leave half of the compute
// units (256 on an MI355X) idle (fp32, us: 4096 x 2048 over 4000 rows 97 -> 76, 8
// experts of 1024 x 512 and 1024 rows 28.5 -> 23.7; 5120 x 5120 over 4096 rows, 400
// tiles, 221 -> 265).  Those experts' rows are cut into s parts, at most one a unit:
// a tile's walk takes rows / 76 us, which s divides, the second launch 3 us, and
// every partial tile 0.06 (512 x 512 over 4096 rows, 8 tiles: s = 1 58 us, 4 23, 8
// 19, 16 20; 2048 x 2048 over 4096 rows, 128 tiles: 1 65, 2 53; over 1024 rows 22.7
// and 29.6).
//
// Units of four rows of tiles, or two, and about eight tiles of a row, where
// every XCD gets eight of them, or one expert's tiles, which are alike, come out
// even; else single rows of tiles (us, bf16: 64 experts' 8 x 8 tiles over 32768
// gathered rows, units of 1 / 2 / 4 / 8 rows 333 / 325 / 319 / 327; 16 experts'
// over 16384 rows, 128 rows of tiles, 144 / 136 / 147 / 187; one expert's 16 x 16
// over 32768 rows 848, 4 x 8 835; 32 x 32 over 8192 rows 855, 4 x 8 832; 16 x 128
// over 8192 rows 1790, 4 x 16 1873).  Where the last unit's rows are not whole, at
// most eight parts: an XCD then meets each unit's rows in one turn.  With more it
// would come back to the last unit's in the next one, and have tiles behind places
// past the last expert, where workgroups stop.  N and K are above 0.
inline void plan_grouped_dw(const spg_grouped_dw_desc &d, GroupedDwArgs &a)
{
    const int64_t tiles_k = cdiv(d.K, kDwTile);
    a.tile_n = d.experts * cdiv(d.N, 256) * tiles_k <= 128 ? 128 : 256;
    const int64_t tiles_n = cdiv(d.N, a.tile_n), tiles = d.experts * tiles_n * tiles_k;
    a.slices = 1;
    const int64_t rows = d.rows / d.experts, units = 256 / tiles;
    const int64_t most = units < kDwMaxSlices ? units : kDwMaxSlices;
    int64_t best = rows * 100 / 76;                         // hundredths of a us
    for (int64_t s = 2; s <= most; ++s) {
        const int64_t t = rows * 100 / (76 * s) + 300 + 6 * tiles * s;
        if (t < best) {
            best = t;
            a.slices = (int32_t)s;
        }
    }
    a.tiles_n = (uint32_t)tiles_n;
    a.tiles_k = (uint32_t)tiles_k;
    a.div_n = make_fastdiv(a.tiles_n);
    a.div_k = make_fastdiv(a.tiles_k);
    a.div_slice = make_fastdiv((uint32_t)a.slices);
    const int64_t rows_of_tiles = d.experts * a.slices * tiles_n;
    a.unit_n = a.unit_k = 0;
    for (int32_t n = 2; n >= 1 && a.unit_n == 0; --n) {
        const bool whole = rows_of_tiles % (1 << n) == 0;
        int32_t parts = 0;
        while ((whole || parts < 3) && (tiles_k >> parts) % 2 == 0 && (tiles_k >> parts) > 8) ++parts;
        const int64_t dealt = cdiv(rows_of_tiles, 1 << n) << parts;
        const bool even = d.experts == 1 && whole && dealt % 8 == 0;
        if (tiles_n >= (1 << n) && (dealt >= 64 || even)) {
            a.unit_n = n;
            a.unit_k = parts;
        }
    }
    a.div_width = make_fastdiv(a.tiles_k >> a.unit_k);
}

// Workgroups: one per compute unit (of the 256 of an MI355X), or as many on
// each XCD as it has tiles.  Workgroup b runs on XCD b % 8.
inline unsigned dw_grid(const GroupedDwArgs &a)
{
    const int64_t rows = (int64_t)a.E * a.slices * a.tiles_n, units = cdiv(rows, 1 << a.unit_n) << a.unit_k;
    const int64_t most = (cdiv(units, 8) << a.unit_n) * (a.tiles_k >> a.unit_k);
    return (unsigned)(8 * (most < 32 ? most : 32));
}

// Place of the workgroup's k-th tile in its XCD's list: one of every grid / 8,
// from the front and from the back in turn, so that with the experts in the
// order of their rows all workgroups get about as much.
__host__ __device__ __forceinline__ uint32_t dw_item(uint32_t grid, uint32_t workgroup, uint32_t k)
{
    const uint32_t step = grid >> 3, first = workgroup >> 3;
    return k * step + ((k & 1) ? step - 1 - first : first);
}

// Tile i of an XCD's list; place >= E: neither it nor any behind it.  Tiles come in the order expert
// (`place` counts them most rows first among each 64), slice, row of tiles,
// tile.  Units of 2^unit_n consecutive rows of tiles, each row cut into 2^unit_k
// parts, stay on one XCD, whose L2 then reads the unit's X and dY once for all of
// its tiles; units are dealt to the XCDs in turn, from the first to the last and
// back, so that all get about as much, however uneven the experts.
struct DwPlace {
    uint32_t place, slice, tn, tk;
};
__host__ __device__ __forceinline__ DwPlace dw_place(const GroupedDwArgs &a, uint32_t xcd, uint32_t i)
{
    const uint32_t width = a.tiles_k >> a.unit_k;
    const uint32_t j = fdiv_q(i, a.div_width);                    // units' rows of this XCD before it
    const uint32_t turn = j >> a.unit_n, u = turn * 8u + ((turn & 1u) ? 7u - xcd : xcd);
    const uint32_t row = ((u >> a.unit_k) << a.unit_n) + (j & ((1u << a.unit_n) - 1u));
    const uint32_t es = fdiv_q(row, a.div_n);
    DwPlace p;
    p.place = fdiv_q(es, a.div_slice);
    p.slice = es - p.place * (uint32_t)a.slices;
    p.tn = row - es * a.tiles_n;
    p.tk = i - j * width + (u & ((1u << a.unit_k) - 1u)) * width;
    return p;
}

}  // namespace spg
