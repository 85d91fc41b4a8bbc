// Exported C ABI (include/spg.h) of the RMS norm and its gradients: argument
// validation and launches.
#include <math.h>
#include <string.h>

#include "spg_api_checks.h"
#include "spg_norm.h"

using namespace spg;

namespace {

// Rows with the team each row length takes: some 2^32 threads.
int64_t max_rows(int64_t H) { return INT64_C(1) << (H <= 2048 ? 26 : H <= 8192 ? 24 : 22); }
// Rows of 64 lanes, four a workgroup: the last one of 2^24 workgroups would make
// 2^32 threads, more than a launch takes.
bool launchable(int64_t R, int64_t H) { return H <= 512 || H > 2048 || R <= (INT64_C(1) << 26) - 4; }

int validate_norm_size(int64_t R, int64_t H)
{
    if (R < 0 || H < 1) return SPG_EINVAL;
    if (H > kNormMaxCols || R >= max_rows(H)) return SPG_EUNSUPPORTED;
    return SPG_OK;
}

// `out` may be the tensor `in` itself, row for row.
bool same_rows(const void *out, int64_t ldo, const void *in, int64_t ldi, int64_t R)
{
    return out == in && (R <= 1 || ldo == ldi);
}
bool clash(const void *out, int64_t ldo, const void *in, int64_t ldi, int64_t R, int64_t H)
{
    return out && in && overlap(out, 2 * extent(R, ldo, H), in, 2 * extent(R, ldi, H)) && !same_rows(out, ldo, in, ldi, R);
}

}  // namespace

SPG_EXPORT int rms_norm(const void *x, const void *residual, const void *weight, void *h, void *normed, uint8_t *q,
                        float *scale, float *rstd, const spg_norm_desc *d, void *stream)
{
    if (!d) return SPG_EINVAL;
    const int v = validate_norm_size(d->R, d->H);
    if (v != SPG_OK) return v;
    const int64_t R = d->R, H = d->H;
    if (!launchable(R, H)) return SPG_EUNSUPPORTED;
    if (d->output != SPG_NORM_BF16 && d->output != SPG_NORM_E4M3_ROW && d->output != SPG_NORM_E4M3_BLOCK128) return SPG_EINVAL;
    if (!(d->eps >= 0.0) || !isfinite(d->eps) || !isfinite(d->weight_offset)) return SPG_EINVAL;
    const bool coded = d->output != SPG_NORM_BF16;
    if (coded && (H % 16)) return SPG_EINVAL;
    if (d->ldx < H || (residual && (d->ldr < H || d->ldh < H)) || (normed && d->ldn < H)) return SPG_EINVAL;
    if (coded && (d->ldq < H || (d->ldq & 15))) return SPG_EINVAL;
    if (!addressable(R, d->ldx) || (residual && (!addressable(R, d->ldr) || !addressable(R, d->ldh))) ||
        (normed && !addressable(R, d->ldn)) || (coded && !addressable(R, d->ldq)))
        return SPG_EUNSUPPORTED;
    if ((residual != nullptr) != (h != nullptr) || coded != (q != nullptr) || coded != (scale != nullptr)) return SPG_EINVAL;
    if (!coded && !normed) return SPG_EINVAL;
    if (R == 0) return SPG_OK;
    if (!x || !weight) return SPG_EINVAL;
    if (!aligned2(x) || !aligned2(residual) || !aligned2(h) || !aligned2(normed) || !aligned16(q) || !aligned4(scale) ||
        !aligned4(rstd) || (d->weight_fp32 ? !aligned4(weight) : !aligned2(weight)))
        return SPG_EINVAL;
    // h and normed may each stand in place of an input; nothing else overlaps
    if (clash(h, d->ldh, x, d->ldx, R, H) || clash(h, d->ldh, residual, d->ldr, R, H) ||
        clash(normed, d->ldn, x, d->ldx, R, H) || clash(normed, d->ldn, residual, d->ldr, R, H))
        return SPG_EINVAL;
    const Range rh = {h, h ? 2 * extent(R, d->ldh, H) : 0}, rn = {normed, normed ? 2 * extent(R, d->ldn, H) : 0};
    const Range rw = {weight, (d->weight_fp32 ? 4 : 2) * H};
    if (overlap(rh.p, rh.bytes, rn.p, rn.bytes) || overlap(rh.p, rh.bytes, rw.p, rw.bytes) ||
        overlap(rn.p, rn.bytes, rw.p, rw.bytes))
        return SPG_EINVAL;
    const int64_t scales = d->output == SPG_NORM_E4M3_BLOCK128 ? cdiv(H, 128) * R : R;
    const Range outs[] = {{q, coded ? extent(R, d->ldq, H) : 0}, {scale, coded ? 4 * scales : 0}, {rstd, rstd ? 4 * R : 0}};
    const Range ins[] = {{x, 2 * extent(R, d->ldx, H)}, {residual, residual ? 2 * extent(R, d->ldr, H) : 0}, rw, rh, rn};
    if (any_overlap(outs, 3, ins, 5)) return SPG_EINVAL;
    NormArgs a;
    memset(&a, 0, sizeof(a));
    a.x = (const uint16_t *)x;
    a.residual = (const uint16_t *)residual;
    a.weight = weight;
    a.h = (uint16_t *)h;
    a.normed = (uint16_t *)normed;
    a.q = q;
    a.scale = scale;
    a.rstd = rstd;
    a.R = R;
    a.H = H;
    a.ldx = d->ldx;
    a.ldr = d->ldr;
    a.ldh = d->ldh;
    a.ldn = d->ldn;
    a.ldq = d->ldq;
    a.eps = d->eps;
    a.w0 = d->weight_offset;
    a.w32 = d->weight_fp32 != 0;
    a.output = d->output;
    return launch_rms_norm(a, (hipStream_t)stream) == hipSuccess ? SPG_OK : SPG_EHIP;
}

SPG_EXPORT size_t rms_norm_backward_workspace_bytes(int64_t R, int64_t H)
{
    if (validate_norm_size(R, H) != SPG_OK || R == 0) return 0;
    const int64_t parts = norm_grad_parts(R, H);
    return parts > 1 ? (size_t)parts * (size_t)norm_grad_width(H) * sizeof(float) : 0;
}

SPG_EXPORT int rms_norm_backward(const void *grad_out, const void *h, const void *grad_residual, const void *weight,
                                 const float *rstd, void *grad_x, float *grad_weight, const spg_norm_grad_desc *d,
                                 void *ws, size_t ws_bytes, void *stream)
{
    if (!d) return SPG_EINVAL;
    const int v = validate_norm_size(d->R, d->H);
    if (v != SPG_OK) return v;
    const int64_t R = d->R, H = d->H;
    if (!isfinite(d->weight_offset)) return SPG_EINVAL;
    if (d->ldg < H || d->ldh < H || d->ldx < H || (grad_residual && d->ldr < H)) return SPG_EINVAL;
    if (!addressable(R, d->ldg) || !addressable(R, d->ldh) || !addressable(R, d->ldx) ||
        (grad_residual && !addressable(R, d->ldr)))
        return SPG_EUNSUPPORTED;
    if (!weight || (R > 0 && (!grad_out || !h || !rstd || !grad_x))) return SPG_EINVAL;
    if (!aligned2(grad_out) || !aligned2(h) || !aligned2(grad_residual) || !aligned2(grad_x) || !aligned4(rstd) ||
        !aligned4(grad_weight) || (d->weight_fp32 ? !aligned4(weight) : !aligned2(weight)))
        return SPG_EINVAL;
    const size_t need = grad_weight ? rms_norm_backward_workspace_bytes(R, H) : 0;
    if (need > 0 && (!ws || ws_bytes < need || !aligned4(ws))) return SPG_EWORKSPACE;
    if (clash(grad_x, d->ldx, grad_out, d->ldg, R, H) || clash(grad_x, d->ldx, h, d->ldh, R, H) ||
        clash(grad_x, d->ldx, grad_residual, d->ldr, R, H))
        return SPG_EINVAL;
    const Range gx = {grad_x, 2 * extent(R, d->ldx, H)}, rw = {weight, (d->weight_fp32 ? 4 : 2) * H}, rr = {rstd, 4 * R};
    if (overlap(gx.p, gx.bytes, rw.p, rw.bytes) || overlap(gx.p, gx.bytes, rr.p, rr.bytes)) return SPG_EINVAL;
    const Range outs[] = {{grad_weight, grad_weight ? 4 * H : 0}, {ws, (int64_t)need}};
    const Range ins[] = {{grad_out, 2 * extent(R, d->ldg, H)}, {h, 2 * extent(R, d->ldh, H)},
                         {grad_residual, grad_residual ? 2 * extent(R, d->ldr, H) : 0}, gx, rw, rr};
    if (any_overlap(outs, 2, ins, 6)) return SPG_EINVAL;
    if (R == 0 && !grad_weight) return SPG_OK;
    NormGradArgs a;
    memset(&a, 0, sizeof(a));
    a.dy = (const uint16_t *)grad_out;
    a.h = (const uint16_t *)h;
    a.dres = (const uint16_t *)grad_residual;
    a.weight = weight;
    a.rstd = rstd;
    a.dx = (uint16_t *)grad_x;
    a.dw = grad_weight;
    a.partials = (float *)ws;
    a.R = R;
    a.H = H;
    a.lddy = d->ldg;
    a.ldh = d->ldh;
    a.lddr = d->ldr;
    a.lddx = d->ldx;
    a.w0 = d->weight_offset;
    a.w32 = d->weight_fp32 != 0;
    return launch_rms_norm_backward(a, (hipStream_t)stream) == hipSuccess ? SPG_OK : SPG_EHIP;
}
