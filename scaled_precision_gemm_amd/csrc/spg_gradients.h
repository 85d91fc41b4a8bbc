// Internal declarations of the gradients' norm and clipping.
#pragma once

#include "spg_common.h"

namespace spg {

// Tensors of one launch: they travel as kernel arguments (at most 4 KiB), so
// nothing is copied to the device and a captured graph keeps them.
constexpr int kGradTensors = 120;
constexpr int64_t kGradChunk = 16384;          // elements of a workgroup's step
constexpr int64_t kGradWorkgroups = 2048;      // of a launch, each with one partial sum
// Up to this many partial sums every workgroup of the scaling adds them itself, a
// launch less (one tensor of 1000 elements: 18.4 us with it, 16.0 without).
constexpr int64_t kGradSelfSum = 512;

struct GradTensors {
    const void *src[kGradTensors];
    void *dst[kGradTensors];
    int64_t n[kGradTensors];
    uint32_t first[kGradTensors + 1];          // chunks before the tensor
    uint32_t bf16[kGradTensors];               // else fp32
    int32_t count;
};

// What gradients are scaled by: f 2^e, e = 0 but where that is below fp32's normal
// range (f then in [1/2, 1)).
struct GradFactor {
    float f;
    int32_t e;
};

hipError_t launch_grad_sums(const GradTensors &t, double *partials, hipStream_t s);
// norm[0] = the root of the partial sums' sum; factor[0], where given, what scales the gradients
hipError_t launch_grad_norm(const double *partials, int64_t parts, double max_norm, float *norm, GradFactor *factor,
                            hipStream_t s);
// By *factor; or, partials given, by the factor of their sum (parts of them), and norm[0] where given as above.
hipError_t launch_grad_scale(const GradTensors &t, const GradFactor *factor, const double *partials, int64_t parts, double max_norm,
                             float *norm, hipStream_t s);

inline int64_t grad_parts(int64_t chunks) { return chunks < kGradWorkgroups ? chunks : kGradWorkgroups; }

}  // namespace spg
