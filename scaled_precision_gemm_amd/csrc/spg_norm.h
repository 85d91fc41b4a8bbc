// Internal declarations of the RMS norm kernels.
#pragma once

#include "spg_common.h"

namespace spg {

constexpr int64_t kNormMaxCols = 32768;      // a row stays in the registers of one workgroup

struct NormArgs {
    const uint16_t *x, *residual;            // [R, H], row strides ldx, ldr; residual or null
    const void *weight;                      // [H] fp32 (w32) or bf16
    uint16_t *h;                             // [R, H], ldh: bf16(x + residual), or null
    uint16_t *normed;                        // [R, H], ldn: bf16(y), or null
    uint8_t *q;                              // [R, H], ldq: codes, or null
    float *scale;                            // [R] or [ceil(H / 128), R]
    float *rstd;                             // [R] or null
    int64_t R, H, ldx, ldr, ldh, ldn, ldq;
    double eps;
    float w0;
    int32_t w32, output;                     // SPG_NORM_*
};
hipError_t launch_rms_norm(const NormArgs &a, hipStream_t s);

struct NormGradArgs {
    const uint16_t *dy, *h, *dres;           // [R, H], row strides lddy, ldh, lddr; dres or null
    const void *weight;
    const float *rstd;                       // [R]
    uint16_t *dx;                            // [R, H], lddx
    float *dw;                               // [H] or null
    float *partials;                         // [norm_grad_parts, norm_grad_width] where there is more than one
    int64_t R, H, lddy, ldh, lddr, lddx;
    float w0;
    int32_t w32;
};
// Workgroups of the gradient's launch, each with a partial sum of dw.
int64_t norm_grad_parts(int64_t R, int64_t H);
int64_t norm_grad_width(int64_t H);            // floats of a partial sum, at least H
hipError_t launch_rms_norm_backward(const NormGradArgs &a, hipStream_t s);

}  // namespace spg
