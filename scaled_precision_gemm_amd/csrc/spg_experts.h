// Internal declarations of the experts' routing and combining kernels.
#pragma once

#include "spg_common.h"

namespace spg {

struct RouteArgs {
    const void *logits;         // [T, E], row stride ld elements
    int64_t ld;
    const float *bias;          // [E] or null
    const float *grad;          // backward: [T, top]
    void *grad_logits;          // backward: [T, E] contiguous
    float *weights;             // [T, top]
    int32_t *experts;           // [T, top]
    int32_t *offsets;           // [E + 1], or null: no row order
    int32_t *rows;              // [T * top]
    int32_t *slots;             // [T, top]
    int32_t *hist;              // workspace: counts [chunks, E], or null: none
    int32_t chunk, chunks;      // tokens of a chunk, chunks
    int64_t T;
    int32_t E, top, groups, top_groups;
    int32_t score, bf16;        // SPG_SCORE_*; logits (and grad_logits) bf16, else fp32
    int32_t renorm;
    int32_t vec;                // rows of logits 16-byte aligned
    float scale;
    FastDiv div_top, div_group; // by top and by E / groups
};

constexpr int kRouteMaxExperts = 1024, kRouteMaxTop = 32, kRouteMaxGroups = 64;
// Up to this many entries (tokens x places) every workgroup of the row order
// counts them all itself; beyond, the route launch leaves counts per chunk.
constexpr int64_t kRouteSelfCount = 16384;
// Tokens of a chunk; 0: no counts.
int32_t route_chunk(int64_t T, int32_t top);

hipError_t launch_expert_route(const RouteArgs &a, hipStream_t s);
hipError_t launch_expert_sort(const RouteArgs &a, hipStream_t s);
hipError_t launch_expert_route_backward(const RouteArgs &a, hipStream_t s);

struct CombineArgs {
    const uint16_t *y;          // [R, H], row stride ldy
    const float *weights;       // [T, top]
    const int32_t *slots;       // [T, top]
    const uint16_t *residual;   // [T, H] or null, row stride ldr
    const uint16_t *grad;       // backward: [T, H], row stride ldr
    uint16_t *out;              // [T, H], row stride ldo; backward: grad_y [R, H]
    float *grad_weights;        // backward: [T, top]
    int64_t T, R, H, ldy, ldr, ldo;
    int32_t top;
};
hipError_t launch_expert_combine(const CombineArgs &a, hipStream_t s);
hipError_t launch_expert_combine_backward(const CombineArgs &a, hipStream_t s);

}  // namespace spg
