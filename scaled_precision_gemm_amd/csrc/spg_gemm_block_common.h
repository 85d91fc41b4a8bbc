// Device pieces shared by the block-scaled FP8 kernels.
//
//   y[m, n] = sum_g sa[m, g] sw[n / 128, g] sum_{k in group g} a[m, k] w[n, k]
//
// The scales change along K, so they cannot be applied after the whole
// accumulation as for the row- and tensor-scaled formats: each group of 128
// K-elements is multiplied by the matrix cores into its own fp32 partial
// product P, which joins the accumulator as acc += P (sa sw) in the vector
// unit.  One multiply-add per 128 products: at the matrix cores' full rate
// the vector unit is half busy.  The factor sa sw is formed in fp32 once per
// (token, weight block, group).
#pragma once

#include "spg_gemm_block.h"
#include "spg_gemm_common.h"

namespace spg {
namespace block {

using namespace gemm;

constexpr int kGroup = 128;

// One output tile of an expert: token rows [m0, end) of the output.
struct ExpertTile {
    int32_t expert;      // -1: no such tile
    uint32_t column;     // its tile column
    uint32_t id;         // among all tiles
    int64_t m0, end;
};

// Rows of expert e and the first of them.  The offsets are the caller's device
// data: they are clamped to [0, rows] and a decreasing pair is an empty
// expert, so no row outside the output is ever touched.
__device__ __forceinline__ int32_t expert_rows(const BlockArgs &a, int e, int32_t &r0)
{
    const int32_t n = (int32_t)a.g.M;
    if (e >= a.experts) {
        r0 = 0;
        return 0;
    }
    const int32_t lo = min(max(a.offsets[e], 0), n), hi = min(max(a.offsets[e + 1], 0), n);
    r0 = lo;
    return max(hi - lo, 0);
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ int32_t wave_scan(int32_t v)
{
    const int lane = lane_id();
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int32_t o = __shfl_up(v, off, 64);
        if (lane >= off) v += o;
    }
    return v;
}

// The tile of this workgroup: BM-row tiles of all experts in expert order,
// tiles_n columns each (columns fastest: neighbours share their rows, the next
// ones their weights), dealt to the XCDs in contiguous ranges of the tiles
// there are.  Every wave works it out by itself: lane l counts the tiles of
// experts l, l + 64, .., 64 consecutive experts at a time, prefix sums by a
// wave scan.  The grid is an upper bound of the tiles; -1 past the last one.
template <int BM>
__device__ __forceinline__ ExpertTile expert_tile(const BlockArgs &a)
{
    const int lane = lane_id();
    ExpertTile t = {-1, 0, 0, 0, 0};
    int32_t r0, rows = expert_rows(a, lane, r0);             // the first run, kept for the second pass
    int32_t n = (rows + BM - 1) / BM, sum = wave_scan(n);
    int32_t run = __builtin_amdgcn_readlane(sum, 63), total = run;
    for (int e0 = 64; e0 < a.experts; e0 += 64) {
        int32_t r;
        int32_t m = (expert_rows(a, e0 + lane, r) + BM - 1) / BM;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) m += __shfl_xor(m, off, 64);
        total += __builtin_amdgcn_readfirstlane(m);
    }
    // (offsets that overlap may count more tiles than the grid has; the bound
    // keeps the tile number in the range of the division)
    const int64_t tiles = min((int64_t)total * a.g.tiles_n, (int64_t)gridDim.x);
    if ((int64_t)blockIdx.x >= tiles) return t;
    t.id = (uint32_t)xcd_remap(blockIdx.x, tiles);
    const uint32_t m = fdiv(t.id, a.g.div_per);              // div_per: by tiles_n
    t.column = t.id - m * (uint32_t)a.g.tiles_n;
    int32_t want = (int32_t)m;
    for (int e0 = 0;; ) {
        if (want < run) {
            const int src = __builtin_ctzll(__ballot(want < sum));   // the first expert whose sum passes `want`
            const int32_t k = want - __builtin_amdgcn_readlane(sum - n, src);
            const int32_t first = __builtin_amdgcn_readlane(r0, src);
            t.m0 = (int64_t)first + (int64_t)k * BM;
            t.end = (int64_t)first + __builtin_amdgcn_readlane(rows, src);
            // (false only where offsets that overlap made a sum overflow)
            if (k >= 0 && t.m0 < t.end) t.expert = e0 + src;
            return t;
        }
        want -= run;
        e0 += 64;
        if (e0 >= a.experts) return t;
        rows = expert_rows(a, e0 + lane, r0);
        n = (rows + BM - 1) / BM;
        sum = wave_scan(n);
        run = __builtin_amdgcn_readlane(sum, 63);
    }
}

}  // namespace block
}  // namespace spg
