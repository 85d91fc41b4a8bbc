// Exported C ABI (include/spg.h) of the gradients' norm and clipping: argument
// validation and launches.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <new>

#include "spg_api_checks.h"
#include "spg_gradients.h"

using namespace spg;

namespace {

constexpr size_t kHead = 16;                          // the factor, before the partial sums
constexpr int64_t kMaxElements = INT64_C(1) << 44;    // of a tensor: chunks count in 32 bits

int validate_list(const spg_gradient *list, int64_t count, bool clip)
{
    if (count < 0 || (count > 0 && !list)) return SPG_EINVAL;
    if (count > (INT64_C(1) << 24)) return SPG_EUNSUPPORTED;
    for (int64_t i = 0; i < count; ++i) {
        const spg_gradient &g = list[i];
        if (g.n < 0) return SPG_EINVAL;
        if (g.n >= kMaxElements) return SPG_EUNSUPPORTED;
        if (g.n == 0) continue;
        if (!g.src || (clip && !g.dst)) return SPG_EINVAL;
        if (g.bf16 ? !aligned2(g.src) || (clip && !aligned2(g.dst)) : !aligned4(g.src) || (clip && !aligned4(g.dst)))
            return SPG_EINVAL;
    }
    return SPG_OK;
}

int64_t bytes_of(const spg_gradient &g) { return g.n * (g.bf16 ? 2 : 4); }

// Calls f(table) for every launch's tensors (empty ones left out).
template <typename F>
int each_launch(const spg_gradient *list, int64_t count, F &&f)
{
    GradTensors t;
    t.count = 0;
    t.first[0] = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (list[i].n == 0) continue;
        const int64_t chunks = cdiv(list[i].n, kGradChunk);
        if (t.count == kGradTensors || t.first[t.count] + chunks >= (INT64_C(1) << 31)) {
            const int e = f(t);
            if (e != SPG_OK) return e;
            t.count = 0;
        }
        const int k = t.count++;
        t.src[k] = list[i].src;
        t.dst[k] = list[i].dst;
        t.n[k] = list[i].n;
        t.bf16[k] = list[i].bf16 != 0;
        t.first[k + 1] = t.first[k] + (uint32_t)chunks;
    }
    return t.count > 0 ? f(t) : SPG_OK;
}

int64_t all_parts(const spg_gradient *list, int64_t count)
{
    int64_t parts = 0;
    each_launch(list, count, [&](const GradTensors &t) {
        parts += grad_parts(t.first[t.count]);
        return (int)SPG_OK;
    });
    return parts;
}

struct Span {
    uintptr_t lo, hi;
    int64_t owner;         // the tensor, -1: an output of another kind
    bool write;
};

// Whether something written (a dst, norm, the workspace) shares a byte with
// anything but its own tensor's src at the same address.
int overlaps(const spg_gradient *list, int64_t count, bool clip, const Range *outs, int n)
{
    Span *s = new (std::nothrow) Span[2 * count + n];
    if (!s) return SPG_EUNSUPPORTED;
    int64_t m = 0;
    bool sorted = true;
    auto add = [&](const void *p, int64_t bytes, int64_t owner, bool write) {
        if (bytes <= 0) return;
        s[m] = Span{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, owner, write};
        sorted = sorted && (m == 0 || s[m - 1].lo <= s[m].lo);
        ++m;
    };
    for (int64_t i = 0; i < count; ++i) {
        const spg_gradient &g = list[i];
        const bool same = clip && g.src == g.dst;
        add(g.src, bytes_of(g), i, same);
        if (clip && !same) add(g.dst, bytes_of(g), i, true);
    }
    for (int i = 0; i < n; ++i) add(outs[i].p, outs[i].bytes, -1, true);
    if (!sorted) std::sort(s, s + m, [](const Span &a, const Span &b) { return a.lo < b.lo; });
    // the furthest end so far of what is written, and of everything
    uintptr_t written = 0, any = 0;
    int found = SPG_OK;
    for (int64_t i = 0; i < m && found == SPG_OK; ++i) {
        if (s[i].lo < written || (s[i].write && s[i].lo < any)) found = SPG_EINVAL;
        any = std::max(any, s[i].hi);
        if (s[i].write) written = std::max(written, s[i].hi);
    }
    delete[] s;
    return found;
}

int run_gradients(const spg_gradient *list, int64_t count, bool clip, double max_norm, float *norm, void *ws,
                  size_t ws_bytes, void *stream)
{
    const int v = validate_list(list, count, clip);
    if (v != SPG_OK) return v;
    if (!norm || !aligned4(norm)) return SPG_EINVAL;
    const int64_t parts = all_parts(list, count);
    const size_t need = kHead + (size_t)parts * sizeof(double);
    if (!ws || ws_bytes < need || !aligned16(ws)) return SPG_EWORKSPACE;
    const Range outs[] = {{norm, 4}, {ws, (int64_t)need}};
    const int o = overlaps(list, count, clip, outs, 2);
    if (o != SPG_OK) return o;
    GradFactor *const factor = clip ? (GradFactor *)ws : nullptr;
    double *const partials = (double *)((uint8_t *)ws + kHead);
    const hipStream_t s = (hipStream_t)stream;
    int64_t at = 0;
    int e = each_launch(list, count, [&](const GradTensors &t) {
        const hipError_t r = launch_grad_sums(t, partials + at, s);
        at += grad_parts(t.first[t.count]);
        return r == hipSuccess ? SPG_OK : SPG_EHIP;
    });
    if (e != SPG_OK) return e;
    // few partial sums: every workgroup of the scaling adds them itself
    const bool self = clip && parts > 0 && parts <= kGradSelfSum;
    if (!self && launch_grad_norm(partials, parts, max_norm, norm, factor, s) != hipSuccess) return SPG_EHIP;
    if (!clip) return SPG_OK;
    return each_launch(list, count, [&](const GradTensors &t) {
        const hipError_t r = launch_grad_scale(t, factor, self ? partials : nullptr, parts, max_norm, norm, s);
        return r == hipSuccess ? SPG_OK : SPG_EHIP;
    });
}

}  // namespace

SPG_EXPORT size_t gradient_workspace_bytes(const spg_gradient *list, int64_t count)
{
    if (validate_list(list, count, false) != SPG_OK) return 0;
    return kHead + (size_t)all_parts(list, count) * sizeof(double);
}

SPG_EXPORT int gradient_norm(const spg_gradient *list, int64_t count, float *norm, void *ws, size_t ws_bytes, void *stream)
{
    return run_gradients(list, count, false, 0.0, norm, ws, ws_bytes, stream);
}

SPG_EXPORT int clip_gradients(const spg_gradient *list, int64_t count, double max_norm, float *norm, void *ws,
                              size_t ws_bytes, void *stream)
{
    if (!(max_norm >= 0.0) || !isfinite(max_norm)) return SPG_EINVAL;
    return run_gradients(list, count, true, max_norm, norm, ws, ws_bytes, stream);
}
