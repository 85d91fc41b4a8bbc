// Exported C ABI (include/spg.h) of the block-128 quantizer and of the
// experts' layer: argument validation and launches.
#include <math.h>
#include <string.h>

#include "spg_api_checks.h"
#include "spg_experts.h"
#include "spg_gemm_block.h"
#include "spg_grouped_dw.h"

using namespace spg;

namespace {

constexpr int64_t kMaxWords = INT64_C(1) << 29;        // floats within a 31-bit byte range
constexpr int64_t kMaxIndex = INT64_C(1) << 31;        // rows and (token, place) pairs are int32
constexpr int64_t kMaxGrid = INT64_C(1) << 23;         // workgroups: at most 512 threads each, 2^32 in all
constexpr int64_t kMaxGridYZ = 65535;
constexpr int64_t kMaxTokens = INT64_C(1) << 25;       // routed tokens: 64 threads each at most

}  // namespace

SPG_EXPORT int quantize_block128(const void *x, int64_t batch, int64_t rows, int64_t K, int64_t ldx, int64_t bstride,
                                 uint8_t *q, int64_t ldq, int64_t qbstride, float *scale, int tiling, void *stream)
{
    if (tiling != SPG_BLOCK_ROW && tiling != SPG_BLOCK_COLUMN && tiling != SPG_BLOCK_BLOCK) return SPG_EINVAL;
    if (batch < 1 || rows < 0 || K < 0 || (K % 16)) return SPG_EINVAL;
    if (rows == 0) return SPG_OK;
    if (!addressable(rows, ldx) || !addressable(rows, ldq) || !addressable(batch, bstride) || !addressable(batch, qbstride))
        return SPG_EUNSUPPORTED;
    if (K == 0) return SPG_EINVAL;                     // a scale of an empty row is undefined
    if (!x || !q || !scale) return SPG_EINVAL;
    if (ldx < K || ldq < K || (ldx & 7) || (ldq & 15)) return SPG_EINVAL;
    if (batch > 1 && (bstride < extent(rows, ldx, K) || (bstride & 7) || qbstride < extent(rows, ldq, K) ||
                      (qbstride & 15)))
        return SPG_EINVAL;
    if (!aligned16(x) || !aligned16(q) || !aligned4(scale)) return SPG_EINVAL;
    if (batch > kMaxGridYZ) return SPG_EUNSUPPORTED;
    if (tiling == SPG_BLOCK_ROW ? (cdiv(rows, 16) >= kMaxGrid || cdiv(K, 512) > kMaxGridYZ)
                                : (cdiv(K, 128) >= kMaxGrid || cdiv(rows, 128) > kMaxGridYZ))
        return SPG_EUNSUPPORTED;
    {
        const int64_t gr = cdiv(rows, 128), gk = cdiv(K, 128);
        const int64_t words = tiling == SPG_BLOCK_ROW ? gk * rows : tiling == SPG_BLOCK_COLUMN ? gr * K : gr * gk;
        const Range outs[] = {{q, (batch - 1) * qbstride + extent(rows, ldq, K)}, {scale, 4 * batch * words}};
        const Range in = {x, 2 * ((batch - 1) * bstride + extent(rows, ldx, K))};
        if (any_overlap(outs, 2, &in, 1)) return SPG_EINVAL;
    }
    const hipError_t e = launch_quantize_block128((const uint16_t *)x, batch, rows, K, ldx, bstride, q, ldq, qbstride,
                                                  scale, tiling, (hipStream_t)stream);
    return e == hipSuccess ? SPG_OK : SPG_EHIP;
}

// ---------------------------------------------------------------------------
// grouped product
// ---------------------------------------------------------------------------

namespace {

int64_t grouped_nout(const spg_grouped_desc *d, int epi) { return epi == SPG_EPI_SWIGLU ? d->N / 2 : d->N; }

int64_t grouped_columns(const spg_grouped_desc *d, int epi, int bm)
{
    return bm == 16 ? cdiv(grouped_nout(d, epi), narrow_cols(epi))
                    : (epi == SPG_EPI_SWIGLU ? cdiv(d->N / 2, 128) : cdiv(d->N, 256));
}

// Tile rows from the mean rows of an expert.  Tiles of 16 rows stream the
// weights with many small workgroups (decode): up to 4 rows, or up to 8 where
// 128-row tiles would leave compute units idle (of the 256 of an MI355X).  256-row tiles read a weight
// panel half as often (and run an expert's last rows as a 128-row tile): above
// 96 rows, where they still give every compute unit one.  Measured (us, cold
// weights; 16-, 128-, 256-row tiles): 64 experts of 2048 x 2048 with 2 rows 43,
// 46, 46, 4 rows 49, 51, 51, 8 rows 53, 52, 52, 80 rows -, 58, 62, 96 rows -, 59,
// 60, 112 rows -, 74, 66, 176 rows -, 80, 74; 128 experts of 1536 x 2048 with 4
// rows 81, 77, 77, 128 rows -, 111, 105, 192 rows -, 135, 116; 16 experts of 4096 x
// 2048 with 128 rows -, 44, 36; 8 experts of 4096 x 4096 with 8 rows 27, 37, 37, and
// 256-row tiles not for every unit: 192 rows -, 41, 60, 256 rows -, 44, 60, but 512
// rows -, 77, 68.  (32-row tiles were not the fastest of any of these.)
int tile_rows(const spg_grouped_desc *d, int epi)
{
    const double mean = (double)d->rows / d->experts;
    if (mean <= (d->experts * cdiv(d->N, 256) < 256 ? 8 : 4)) return 16;
    if (mean <= 96) return 128;
    return d->experts * cdiv((int64_t)mean, 256) * grouped_columns(d, epi, 256) < 256 ? 128 : 256;
}

// Upper bound of the row tiles: every expert adds at most one partial tile,
// and no tile is empty.
int64_t most_tiles(const spg_grouped_desc *d, int bm)
{
    const int64_t most = d->rows / bm + d->experts;
    return most < d->rows ? most : d->rows;
}

// Checks that do not depend on whether rows are gathered (a_rows is then free,
// but addressed with 31-bit offsets).
int validate_grouped(const spg_grouped_desc *d, int epi)
{
    if (!d) return SPG_EINVAL;
    if (epi != SPG_EPI_STORE && epi != SPG_EPI_ADD && epi != SPG_EPI_SWIGLU) return SPG_EINVAL;
    if (epi == SPG_EPI_ADD) return SPG_EUNSUPPORTED;
    if (d->rows < 0 || d->a_rows < 0 || d->N < 0 || d->K < 0 || (d->K % 16)) return SPG_EINVAL;
    if (d->experts < 1) return SPG_EINVAL;
    if (d->experts > 65536) return SPG_EUNSUPPORTED;
    if (epi == SPG_EPI_SWIGLU && (d->N % 256)) return SPG_EINVAL;
    if (d->lda < d->K || d->ldw < d->K || (d->lda & 15) || (d->ldw & 15)) return SPG_EINVAL;
    if (d->lda > (INT64_C(1) << 23) || d->ldw > (INT64_C(1) << 23)) return SPG_EUNSUPPORTED;
    if (d->stride_w < 0 || (d->stride_w & 15)) return SPG_EINVAL;
    if (!addressable(d->experts, d->stride_w)) return SPG_EUNSUPPORTED;
    if (d->experts > 1 && d->stride_w != 0 && d->stride_w < extent(d->N, d->ldw, d->K)) return SPG_EINVAL;
    if (d->ldo < grouped_nout(d, epi)) return SPG_EINVAL;
    if (d->ldo >= (INT64_C(1) << 26)) return SPG_EUNSUPPORTED;
    if (d->rows >= kMaxWords || d->a_rows >= kMaxWords || d->N >= kMaxWords || d->K >= kMaxWords ||
        cdiv(d->N, 128) * cdiv(d->K, 128) >= kMaxWords)
        return SPG_EUNSUPPORTED;
    const int bm = tile_rows(d, epi);
    if (most_tiles(d, bm) * grouped_columns(d, epi, bm) >= kMaxGrid) return SPG_EUNSUPPORTED;
    return SPG_OK;
}

}  // namespace

SPG_EXPORT int spg_grouped_tile_rows(const spg_grouped_desc *d, int epilogue)
{
    return validate_grouped(d, epilogue) == SPG_OK ? tile_rows(d, epilogue) : 0;
}

SPG_EXPORT int gemm_grouped(void *out, const void *A, const float *sa, const void *W, const float *sw,
                            const int32_t *offsets, const int32_t *row_index, int epilogue, const spg_grouped_desc *d,
                            void *stream)
{
    const int v = validate_grouped(d, epilogue);
    if (v != SPG_OK) return v;
    if (!row_index && d->a_rows < d->rows) return SPG_EINVAL;
    if (row_index && d->a_rows * d->lda >= (INT64_C(1) << 31)) return SPG_EUNSUPPORTED;
    const int64_t nout = grouped_nout(d, epilogue);
    if (d->rows == 0 || nout == 0) return SPG_OK;
    if (!out || !A || !sa || !W || !sw || !offsets) return SPG_EINVAL;
    if (!aligned16(A) || !aligned16(W) || !aligned2(out) || !aligned4(sa) || !aligned4(sw) || !aligned4(offsets) ||
        !aligned4(row_index))
        return SPG_EINVAL;
    const int64_t groups = cdiv(d->K, 128), blocks = cdiv(d->N, 128), E = d->experts;
    const int64_t obytes = 2 * extent(d->rows, d->ldo, nout);
    if (overlap(out, obytes, A, extent(d->a_rows, d->lda, d->K)) ||
        overlap(out, obytes, W, (E - 1) * d->stride_w + extent(d->N, d->ldw, d->K)) ||
        overlap(out, obytes, sa, 4 * groups * d->a_rows) || overlap(out, obytes, sw, 4 * E * blocks * groups) ||
        overlap(out, obytes, offsets, 4 * (E + 1)) || (row_index && overlap(out, obytes, row_index, 4 * d->rows)))
        return SPG_EINVAL;
    BlockArgs a;
    memset(&a, 0, sizeof(a));
    GemmArgs &g = a.g;
    g.out = out;
    g.A = (const uint8_t *)A;
    g.W = (const uint8_t *)W;
    g.sa = sa;
    g.sw = sw;
    g.M = d->rows;
    g.N = d->N;
    g.K = d->K;
    g.batch = 1;
    g.lda = d->lda;
    g.ldw = d->ldw;
    g.ldo = d->ldo;
    g.stride_w = d->stride_w;
    g.sw_bstride = blocks * groups;
    g.format = SPG_FMT_E4M3_BLOCK128;
    g.epilogue = epilogue;
    g.split_k = 1;
    a.a_rows = d->a_rows;
    a.groups = (int32_t)groups;
    a.sw_words = (int32_t)(blocks * groups);
    a.sw_rs = (int32_t)groups;
    a.sw_gs = 1;
    a.offsets = offsets;
    a.row_index = row_index;
    a.experts = d->experts;
    const int bm = tile_rows(d, epilogue);
    g.tiles_n = grouped_columns(d, epilogue, bm);
    g.div_per = make_fastdiv((uint32_t)g.tiles_n);
    const int64_t workgroups = most_tiles(d, bm) * g.tiles_n;
    const hipError_t e = bm == 16 ? launch_gemm_block_narrow(a, bm, workgroups, (hipStream_t)stream)
                                  : launch_gemm_block_tiles(a, bm, workgroups, (hipStream_t)stream);
    return e == hipSuccess ? SPG_OK : SPG_EHIP;
}

// ---------------------------------------------------------------------------
// weight gradient of the grouped product
// ---------------------------------------------------------------------------

namespace {

int validate_dw(const spg_grouped_dw_desc *d, bool gathered, bool add)
{
    if (!d) return SPG_EINVAL;
    if (d->rows < 0 || d->x_rows < 0 || d->N < 0 || d->K < 0 || (d->N % 8) || (d->K % 8) || d->experts < 1) return SPG_EINVAL;
    if (d->ldy < d->N || d->ldx < d->K || (d->ldy & 7) || (d->ldx & 7)) return SPG_EINVAL;
    const int64_t unit = d->out_fp32 ? 4 : 8;               // elements of 16 bytes
    if (d->ldo < d->K || d->ldo % unit || d->stride_o % unit) return SPG_EINVAL;
    if (add && (d->lda < d->K || d->lda % unit || d->stride_a % unit)) return SPG_EINVAL;
    if (d->experts > 65536 || d->rows >= kMaxIndex || d->x_rows >= kMaxIndex || d->N >= kMaxWords || d->K >= kMaxWords ||
        d->ldy > (INT64_C(1) << 24) || d->ldx > (INT64_C(1) << 24))
        return SPG_EUNSUPPORTED;
    if (gathered && extent(d->x_rows, d->ldx, d->K) >= (INT64_C(1) << 30)) return SPG_EUNSUPPORTED;
    if (!addressable(d->N, d->ldo) || !addressable(d->experts, d->stride_o) ||
        (add && (!addressable(d->N, d->lda) || !addressable(d->experts, d->stride_a))))
        return SPG_EUNSUPPORTED;
    // experts' matrices do not overlap
    if (d->experts > 1 && d->stride_o < extent(d->N, d->ldo, d->K)) return SPG_EINVAL;
    if (add && d->experts > 1 && d->stride_a < extent(d->N, d->lda, d->K)) return SPG_EINVAL;
    // tiles are counted in 32 bits
    if ((d->experts * cdiv(d->N, 128) + 64) * cdiv(d->K, kDwTile) >= kMaxIndex / kDwMaxSlices) return SPG_EUNSUPPORTED;
    return SPG_OK;
}

}  // namespace

SPG_EXPORT size_t gemm_grouped_dw_workspace_bytes(const spg_grouped_dw_desc *d)
{
    if (validate_dw(d, false, false) != SPG_OK || d->N == 0 || d->K == 0) return 0;
    GroupedDwArgs a;
    plan_grouped_dw(*d, a);
    const size_t tiles = (size_t)d->experts * a.tiles_n * a.tiles_k;
    return a.slices > 1 ? tiles * a.slices * a.tile_n * kDwTile * sizeof(float) : 0;
}

SPG_EXPORT int gemm_grouped_dw(void *out, const void *dY, const void *X, const int32_t *offsets, const int32_t *row_index,
                               const void *add, const spg_grouped_dw_desc *d, void *ws, size_t ws_bytes, void *stream)
{
    const int v = validate_dw(d, row_index != nullptr, add != nullptr);
    if (v != SPG_OK) return v;
    if (!row_index && d->x_rows < d->rows) return SPG_EINVAL;
    if (d->N == 0 || d->K == 0) return SPG_OK;
    if (!out || !offsets || (d->rows > 0 && (!dY || (d->x_rows > 0 && !X)))) return SPG_EINVAL;
    if (!aligned16(out) || !aligned16(dY) || !aligned16(X) || !aligned16(add) || !aligned4(offsets) || !aligned4(row_index))
        return SPG_EINVAL;
    const size_t need = gemm_grouped_dw_workspace_bytes(d);
    if (need > 0 && (!ws || ws_bytes < need || !aligned16(ws))) return SPG_EWORKSPACE;
    {
        const int64_t size = d->out_fp32 ? 4 : 2, E = d->experts;
        const Range ro = {out, size * ((E - 1) * d->stride_o + extent(d->N, d->ldo, d->K))};
        const Range ra = {add, add ? size * ((E - 1) * d->stride_a + extent(d->N, d->lda, d->K)) : 0};
        const Range outs[] = {ro, {ws, (int64_t)need}};
        const Range ins[] = {{dY, 2 * extent(d->rows, d->ldy, d->N)}, {X, 2 * extent(d->x_rows, d->ldx, d->K)},
                             {offsets, 4 * (E + 1)}, {row_index, row_index ? 4 * d->rows : 0}};
        if (any_overlap(outs, 2, ins, 4) || overlap(ws, (int64_t)need, ra.p, ra.bytes)) return SPG_EINVAL;
        // add may be the output itself
        const bool same = add == out && (d->N <= 1 || d->lda == d->ldo) && (E <= 1 || d->stride_a == d->stride_o);
        if (!same && overlap(ro.p, ro.bytes, ra.p, ra.bytes)) return SPG_EINVAL;
    }
    GroupedDwArgs a;
    memset(&a, 0, sizeof(a));
    a.dy = (const uint16_t *)dY;
    a.x = (const uint16_t *)X;
    a.offsets = offsets;
    a.row_index = row_index;
    a.add = add;
    a.out = out;
    a.partials = (float *)ws;
    a.R = d->rows;
    a.x_rows = d->x_rows;
    a.N = d->N;
    a.K = d->K;
    a.ldy = d->ldy;
    a.ldx = d->ldx;
    a.lda = d->lda;
    a.stride_a = d->stride_a;
    a.ldo = d->ldo;
    a.stride_o = d->stride_o;
    a.E = d->experts;
    a.out_fp32 = d->out_fp32 != 0;
    const int64_t line = d->out_fp32 ? 32 : 64;
    a.lines = ((uintptr_t)out & 127u) == 0 && d->ldo % line == 0 && d->stride_o % line == 0 &&
              (!add || (((uintptr_t)add & 127u) == 0 && d->lda % line == 0 && d->stride_a % line == 0));
    plan_grouped_dw(*d, a);
    return launch_grouped_dw(a, (hipStream_t)stream) == hipSuccess ? SPG_OK : SPG_EHIP;
}

// ---------------------------------------------------------------------------
// routing
// ---------------------------------------------------------------------------

namespace {

int validate_route(const spg_route_desc *d)
{
    if (!d) return SPG_EINVAL;
    if (d->T < 0 || d->E < 1 || d->top < 1 || d->top > d->E || d->ld < d->E) return SPG_EINVAL;
    if (d->groups < 1 || d->top_groups < 1 || d->top_groups > d->groups || d->E % d->groups) return SPG_EINVAL;
    if (d->score != SPG_SCORE_SOFTMAX && d->score != SPG_SCORE_SIGMOID) return SPG_EINVAL;
    if (!isfinite(d->scale)) return SPG_EINVAL;
    if (d->E > kRouteMaxExperts || d->top > kRouteMaxTop || d->groups > kRouteMaxGroups) return SPG_EUNSUPPORTED;
    if (d->T >= kMaxIndex / d->top || d->T >= kMaxTokens || !addressable(d->T, d->ld)) return SPG_EUNSUPPORTED;
    return SPG_OK;
}

// The counts of every chunk of tokens.
size_t order_ws(int64_t T, int32_t top, int32_t E)
{
    const int32_t chunk = route_chunk(T, top);
    return chunk == 0 ? 0 : (size_t)cdiv(T, chunk) * (size_t)E * sizeof(int32_t);
}

RouteArgs route_args(const spg_route_desc *d)
{
    RouteArgs a;
    memset(&a, 0, sizeof(a));
    a.ld = d->ld;
    a.T = d->T;
    a.E = d->E;
    a.top = d->top;
    a.groups = d->groups;
    a.top_groups = d->top_groups;
    a.score = d->score;
    a.bf16 = d->logits_bf16 != 0;
    a.renorm = d->renormalize != 0;
    a.scale = d->scale;
    a.div_top = make_fastdiv((uint32_t)d->top);
    a.div_group = make_fastdiv((uint32_t)(d->E / d->groups));
    return a;
}

}  // namespace

SPG_EXPORT size_t expert_order_workspace_bytes(int64_t T, int32_t top, int32_t E)
{
    if (T <= 0 || top < 1 || E < 1 || E > kRouteMaxExperts || T >= kMaxIndex / top) return 0;
    return order_ws(T, top, E);
}

SPG_EXPORT int expert_route(const void *logits, const float *bias, float *weights, int32_t *experts, int32_t *offsets,
                            int32_t *rows, int32_t *slots, const spg_route_desc *d, void *ws, size_t ws_bytes,
                            void *stream)
{
    const int v = validate_route(d);
    if (v != SPG_OK) return v;
    const bool order = offsets || rows || slots;
    if (order && (!offsets || !rows || !slots)) return SPG_EINVAL;
    if (d->T > 0) {
        if (!logits || !weights || !experts) return SPG_EINVAL;
        if (d->logits_bf16 ? !aligned2(logits) : !aligned4(logits)) return SPG_EINVAL;
    }
    if (!aligned4(bias) || !aligned4(weights) || !aligned4(experts) || !aligned4(offsets) || !aligned4(rows) ||
        !aligned4(slots))
        return SPG_EINVAL;
    RouteArgs a = route_args(d);
    a.vec = aligned16(logits) && d->ld % (d->logits_bf16 ? 8 : 4) == 0;
    a.logits = logits;
    a.bias = bias;
    a.weights = weights;
    a.experts = experts;
    a.offsets = offsets;
    a.rows = rows;
    a.slots = slots;
    if (order && order_ws(d->T, d->top, d->E) > 0) {
        if (!ws || ws_bytes < order_ws(d->T, d->top, d->E) || !aligned4(ws)) return SPG_EWORKSPACE;
        a.hist = (int32_t *)ws;
        a.chunk = route_chunk(d->T, d->top);
        a.chunks = (int32_t)cdiv(d->T, a.chunk);
    }
    {
        const int64_t bytes = 4 * d->T * d->top;
        const Range outs[] = {{weights, bytes}, {experts, bytes}, {offsets, order ? 4 * (int64_t)(d->E + 1) : 0},
                              {rows, order ? bytes : 0}, {slots, order ? bytes : 0},
                              {a.hist, a.hist ? (int64_t)order_ws(d->T, d->top, d->E) : 0}};
        const Range ins[] = {{logits, (d->logits_bf16 ? 2 : 4) * extent(d->T, d->ld, d->E)}, {bias, bias ? 4 * d->E : 0}};
        if (any_overlap(outs, 6, ins, 2)) return SPG_EINVAL;
    }
    // no token: the row order is that of no rows
    if (d->T == 0 && !order) return SPG_OK;
    return launch_expert_route(a, (hipStream_t)stream) == hipSuccess ? SPG_OK : SPG_EHIP;
}

SPG_EXPORT int expert_sort(const int32_t *experts, int64_t T, int32_t top, int32_t E, int32_t *offsets, int32_t *rows,
                           int32_t *slots, void *ws, size_t ws_bytes, void *stream)
{
    if (T < 0 || top < 1 || E < 1) return SPG_EINVAL;
    if (E > kRouteMaxExperts) return SPG_EUNSUPPORTED;
    if (T >= kMaxIndex / top) return SPG_EUNSUPPORTED;
    if (!offsets || (T > 0 && (!experts || !rows || !slots))) return SPG_EINVAL;
    if (!aligned4(experts) || !aligned4(offsets) || !aligned4(rows) || !aligned4(slots)) return SPG_EINVAL;
    const size_t need = order_ws(T, top, E);
    if (need > 0 && (!ws || ws_bytes < need || !aligned4(ws))) return SPG_EWORKSPACE;
    {
        const int64_t bytes = 4 * T * top;
        const Range outs[] = {{offsets, 4 * (int64_t)(E + 1)}, {rows, bytes}, {slots, bytes}, {ws, (int64_t)need}};
        const Range in = {experts, bytes};
        if (any_overlap(outs, 4, &in, 1)) return SPG_EINVAL;
    }
    spg_route_desc d;
    memset(&d, 0, sizeof(d));
    d.T = T;
    d.E = E;
    d.top = top;
    d.groups = d.top_groups = 1;
    RouteArgs a = route_args(&d);
    a.experts = (int32_t *)experts;
    a.offsets = offsets;
    a.rows = rows;
    a.slots = slots;
    if (need > 0) {
        a.hist = (int32_t *)ws;
        a.chunk = route_chunk(T, top);
        a.chunks = (int32_t)cdiv(T, a.chunk);
    }
    return launch_expert_sort(a, (hipStream_t)stream) == hipSuccess ? SPG_OK : SPG_EHIP;
}

SPG_EXPORT int expert_route_backward(const float *grad_weights, const void *logits, const int32_t *experts,
                                     void *grad_logits, const spg_route_desc *d, void *stream)
{
    const int v = validate_route(d);
    if (v != SPG_OK) return v;
    if (d->T == 0) return SPG_OK;
    if (!grad_weights || !logits || !experts || !grad_logits) return SPG_EINVAL;
    if (!aligned4(grad_weights) || !aligned4(experts)) return SPG_EINVAL;
    if (d->logits_bf16 ? !aligned2(logits) || !aligned2(grad_logits) : !aligned4(logits) || !aligned4(grad_logits))
        return SPG_EINVAL;
    const int64_t size = d->logits_bf16 ? 2 : 4;
    const Range out = {grad_logits, size * d->T * d->E};
    const Range ins[] = {{logits, size * extent(d->T, d->ld, d->E)}, {grad_weights, 4 * d->T * d->top},
                         {experts, 4 * d->T * d->top}};
    if (any_overlap(&out, 1, ins, 3)) return SPG_EINVAL;
    RouteArgs a = route_args(d);
    a.logits = logits;
    a.grad = grad_weights;
    a.experts = (int32_t *)experts;
    a.grad_logits = grad_logits;
    return launch_expert_route_backward(a, (hipStream_t)stream) == hipSuccess ? SPG_OK : SPG_EHIP;
}

// ---------------------------------------------------------------------------
// combine
// ---------------------------------------------------------------------------

namespace {

int validate_combine(int64_t T, int64_t R, int32_t top, int64_t H)
{
    if (T < 0 || R < 0 || H < 0 || top < 1) return SPG_EINVAL;
    if (top > kRouteMaxTop) return SPG_EUNSUPPORTED;
    if (T >= kMaxIndex / top || T >= kMaxGrid || R >= kMaxIndex || H >= kMaxGridYZ * 256) return SPG_EUNSUPPORTED;
    return SPG_OK;
}

}  // namespace

SPG_EXPORT int expert_combine(const void *y, int64_t R, int64_t ldy, const float *weights, const int32_t *slots,
                              int64_t T, int32_t top, int64_t H, const void *residual, int64_t ldr, void *out,
                              int64_t ldo, void *stream)
{
    const int v = validate_combine(T, R, top, H);
    if (v != SPG_OK) return v;
    if (ldy < H || ldo < H || (residual && ldr < H)) return SPG_EINVAL;
    if (!addressable(R, ldy) || !addressable(T, ldo) || (residual && !addressable(T, ldr))) return SPG_EUNSUPPORTED;
    if (T == 0 || H == 0) return SPG_OK;
    if ((R > 0 && !y) || !weights || !slots || !out) return SPG_EINVAL;
    if (!aligned2(y) || !aligned2(residual) || !aligned2(out) || !aligned4(weights) || !aligned4(slots))
        return SPG_EINVAL;
    const int64_t obytes = 2 * extent(T, ldo, H);
    if (overlap(out, obytes, y, 2 * extent(R, ldy, H)) || overlap(out, obytes, weights, 4 * T * top) ||
        overlap(out, obytes, slots, 4 * T * top))
        return SPG_EINVAL;
    if (residual && overlap(out, obytes, residual, 2 * extent(T, ldr, H)) && !(residual == out && ldr == ldo))
        return SPG_EINVAL;
    CombineArgs a;
    memset(&a, 0, sizeof(a));
    a.y = (const uint16_t *)y;
    a.weights = weights;
    a.slots = slots;
    a.residual = (const uint16_t *)residual;
    a.out = (uint16_t *)out;
    a.T = T;
    a.R = R;
    a.H = H;
    a.ldy = ldy;
    a.ldr = ldr;
    a.ldo = ldo;
    a.top = top;
    return launch_expert_combine(a, (hipStream_t)stream) == hipSuccess ? SPG_OK : SPG_EHIP;
}

SPG_EXPORT int expert_combine_backward(const void *grad_out, int64_t ldg, const void *y, int64_t R, int64_t ldy,
                                       const float *weights, const int32_t *slots, int64_t T, int32_t top, int64_t H,
                                       void *grad_y, int64_t ldgy, float *grad_weights, void *stream)
{
    const int v = validate_combine(T, R, top, H);
    if (v != SPG_OK) return v;
    if (ldg < H || ldy < H || ldgy < H) return SPG_EINVAL;
    if (!addressable(T, ldg) || !addressable(R, ldy) || !addressable(R, ldgy)) return SPG_EUNSUPPORTED;
    if (T == 0) return SPG_OK;
    if (!weights || !slots || !grad_weights) return SPG_EINVAL;
    if (H > 0 && (!grad_out || (R > 0 && (!y || !grad_y)))) return SPG_EINVAL;
    if (!aligned2(grad_out) || !aligned2(y) || !aligned2(grad_y) || !aligned4(weights) || !aligned4(slots) ||
        !aligned4(grad_weights))
        return SPG_EINVAL;
    {
        const int64_t wbytes = 4 * T * top;
        const Range outs[] = {{grad_y, 2 * extent(R, ldgy, H)}, {grad_weights, wbytes}};
        const Range ins[] = {{y, 2 * extent(R, ldy, H)}, {grad_out, 2 * extent(T, ldg, H)}, {weights, wbytes}, {slots, wbytes}};
        if (any_overlap(outs, 2, ins, 4)) return SPG_EINVAL;
    }
    CombineArgs a;
    memset(&a, 0, sizeof(a));
    a.y = (const uint16_t *)y;
    a.weights = weights;
    a.slots = slots;
    a.grad = (const uint16_t *)grad_out;
    a.out = (uint16_t *)grad_y;
    a.grad_weights = grad_weights;
    a.T = T;
    a.R = R;
    a.H = H;
    a.ldy = ldy;
    a.ldr = ldg;
    a.ldo = ldgy;
    a.top = top;
    return launch_expert_combine_backward(a, (hipStream_t)stream) == hipSuccess ? SPG_OK : SPG_EHIP;
}
