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
    int64_t m0, end;
};

// Tile of BM rows number `id` of all experts' rows in expert order, and the
// number of such tiles.  Every wave works it out by itself: lane l sums the
// tile counts of experts l, l + 64 (in runs of 64 consecutive experts, so the
// prefix is a wave scan per run).  The offsets are the caller's device data:
// they are clamped to [0, rows] and a decreasing pair is an empty expert, so
// no row outside the output is ever touched.
template <int BM>
__device__ __forceinline__ int32_t expert_rows(const BlockArgs &a, int e, int64_t &r0)
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

template <int BM>
__device__ __forceinline__ int32_t total_tiles(const BlockArgs &a)
{
    const int lane = lane_id();
    int32_t n = 0;
    for (int e = lane; e < a.experts; e += 64) {
        int64_t r0;
        n += (expert_rows<BM>(a, e, r0) + BM - 1) / BM;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) n += __shfl_xor(n, off, 64);
    return __builtin_amdgcn_readfirstlane(n);
}

template <int BM>
__device__ __forceinline__ ExpertTile find_tile(const BlockArgs &a, int32_t id)
{
    const int lane = lane_id();
    int32_t before = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
        int64_t r0;
        const int32_t rows = expert_rows<BM>(a, e0 + lane, r0);
        const int32_t n = (rows + BM - 1) / BM;
        int32_t sum = n;                              // inclusive scan over the wave
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int32_t o = __shfl_up(sum, off, 64);
            if (lane >= off) sum += o;
        }
        const int32_t all = __builtin_amdgcn_readfirstlane(__shfl(sum, 63, 64));
        if (id < before + all) {
            const int32_t want = id - before;
            const uint64_t hit = __ballot(want < sum);   // the first lane whose sum passes `want`
            const int src = __builtin_ctzll(hit);
            const int32_t base = __builtin_amdgcn_readfirstlane(__shfl(sum - n, src, 64));
            const int32_t first = __builtin_amdgcn_readfirstlane(__shfl((int32_t)r0, src, 64));
            const int32_t count = __builtin_amdgcn_readfirstlane(__shfl(rows, src, 64));
            ExpertTile t;
            t.expert = e0 + src;
            t.m0 = (int64_t)first + (int64_t)(want - base) * BM;
            t.end = (int64_t)first + count;
            return t;
        }
        before += all;
    }
    return ExpertTile{-1, 0, 0};
}

}  // namespace block
}  // namespace spg
