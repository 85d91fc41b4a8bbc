// Internal declarations of the gradients' norm and clipping.
#pragma once

#include "spg_common.h"

namespace spg {

// Tensors of one launch: they travel as kernel arguments (at most 4 KiB), so
// nothing is copied to the device and a captured graph keeps them.
constexpr int kGradTensors = 120;
constexpr int64_t kGradChunk = 16384;          // elements of a workgroup's step
constexpr int64_t kGradWorkgroups = 2048;      // of a launch, each with one partial sum

struct GradTable {
    const void *src[kGradTensors];
    void *dst[kGradTensors];
    int64_t n[kGradTensors];
    uint32_t first[kGradTensors + 1];          // chunks before the tensor
    uint8_t bf16[kGradTensors];                // else fp32
    int32_t count;
};

hipError_t launch_grad_sums(const GradTable &t, double *partials, hipStream_t s);
// norm[0] = the root of the partial sums' sum; factor[0], where given, what scales the gradients
hipError_t launch_grad_norm(const double *partials, int64_t parts, double max_norm, float *norm, float *factor, hipStream_t s);
hipError_t launch_grad_scale(const GradTable &t, const float *factor, hipStream_t s);

inline int64_t grad_parts(int64_t chunks) { return chunks < kGradWorkgroups ? chunks : kGradWorkgroups; }

}  // namespace spg
