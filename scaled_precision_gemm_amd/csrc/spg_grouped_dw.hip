// Weight gradients of the experts' products, from bf16 operands:
//
//   dW_e[n, k] = add_e[n, k] + sum over the rows r of expert e of dY[r, n] X[row(r), k]
//
// The summed side is the ragged one.  Both operands are stored with it as
// their rows, so the matrix core's fragments, eight consecutive r of one
// column per lane, run across the rows of memory: ds_read_b64_tr_b16 gives
// each of 16 lanes four elements of one column out of four rows of 16
// elements, and the operands need no transposed copy.
//
//  * 256 x 256 tiles of dW_e over eight waves (two a SIMD), each 128 n x 64 k
//    as 4 x 2 blocks of v_mfma_f32_32x32x16_bf16: 128 accumulators a lane.
//    X is the first MFMA operand, so a lane's four consecutive results are
//    four consecutive k of one row n.
//  * A stage is 32 rows of both operands, 32 KiB, copied straight into one of
//    kDepth LDS slots (buffer loads to LDS).  Rows past the expert's last
//    one are out of the buffer's range and read as zeros in both operands, so
//    whatever stands in the rows behind is not multiplied.
//  * LDS row r holds its 16-byte chunk c at c ^ 4 (r % 4): a transposing read
//    takes 64 bytes of four consecutive rows 512 bytes apart, which then lie
//    in four different quarters of the 64 banks.
//  * Experts' rows are read from the offsets on the device, so a captured graph
//    serves any routing.
#include "spg_gemm_common.h"
#include "spg_grouped_dw.h"

namespace spg {

namespace {

using namespace gemm;

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kDwThreads = 512, kDwWaves = 8;
constexpr int kStageRows = 32, kLdsRow = 512;                    // one LDS row: 256 columns
constexpr int kOperand = kStageRows * kLdsRow, kSlotBytes = 2 * kOperand;
constexpr int kDepth = 4;
constexpr int kCopies = 4;                                       // copy instructions of a wave per stage
constexpr int kRegion = 32 * 64 * 4;                             // epilogue: 32 n x 64 k in fp32 per wave
static_assert(kDwWaves * kRegion <= kDepth * kSlotBytes, "the epilogue's LDS fits in the slots");

enum { kOutBf16, kOutFp32, kOutPartial };

// Chunk of 8 (bf16) or 4 (fp32) elements: add + sum, rounded once.
template <int OUT>
__device__ __forceinline__ void store_chunk(const GroupedDwArgs &a, int e, int64_t n, int64_t k, const v4f &lo, const v4f &hi)
{
    const int64_t at = (int64_t)e * a.stride_o + n * a.ldo + k;
    const int64_t from = (int64_t)e * a.stride_a + n * a.lda + k;
    if (OUT == kOutBf16) {
        v4f l = lo, h = hi;
        if (a.add) {
            const uint4 p = *reinterpret_cast<const uint4 *>((const uint16_t *)a.add + from);
            l += v4f{bf16_lo(p.x), bf16_hi(p.x), bf16_lo(p.y), bf16_hi(p.y)};
            h += v4f{bf16_lo(p.z), bf16_hi(p.z), bf16_lo(p.w), bf16_hi(p.w)};
        }
        __builtin_nontemporal_store(v4i{(int)pack_bf16x2(l[0], l[1]), (int)pack_bf16x2(l[2], l[3]),
                                        (int)pack_bf16x2(h[0], h[1]), (int)pack_bf16x2(h[2], h[3])},
                                    reinterpret_cast<v4i *>((uint16_t *)a.out + at));
    } else {
        v4f l = lo;
        if (a.add) l += *reinterpret_cast<const v4f *>((const float *)a.add + from);
        __builtin_nontemporal_store(l, reinterpret_cast<v4f *>((float *)a.out + at));
    }
}

// Rows of expert e: the offsets are the caller's device data, clamped to [0,
// R]; a decreasing pair is an empty expert.
__device__ __forceinline__ void expert_range(const GroupedDwArgs &a, int e, int64_t &lo, int64_t &hi)
{
    const int32_t R = (int32_t)a.R;
    lo = min(max(a.offsets[e], 0), R);
    hi = max((int32_t)lo, min(max(a.offsets[e + 1], 0), R));
}

// Work items in the order expert, slice, row of tiles, tile.  A row of tiles
// (which share their panel of dY) stays on one XCD and the rows are dealt to the
// XCDs in turn, so every XCD gets its share of every expert, however many rows
// that one has.
struct DwWork {
    int e, slice;
    uint32_t tn, tk;
    bool live;
};
__device__ __forceinline__ DwWork dw_work(const GroupedDwArgs &a)
{
    const uint32_t xcd = blockIdx.x & 7u, idx = blockIdx.x >> 3;
    const uint32_t j = fdiv(idx, a.div_k);                        // rows of tiles of this XCD so far
    DwWork w;
    w.tk = idx - j * a.tiles_k;
    const uint32_t row = j * 8u + xcd;
    const uint32_t es = fdiv(row, a.div_n);
    w.tn = row - es * a.tiles_n;
    w.e = (int)fdiv(es, a.div_slice);
    w.slice = (int)(es - (uint32_t)w.e * (uint32_t)a.slices);
    w.live = w.e < a.E;
    return w;
}

template <int OUT, bool GATHER>
__global__ __launch_bounds__(kDwThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void grouped_dw_kernel(
    const GroupedDwArgs a)
{
    __shared__ __attribute__((aligned(2048))) uint8_t lds[kDepth * kSlotBytes];
    const DwWork w = dw_work(a);
    if (!w.live) return;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), ln = lane_id();
    const int wn = wave >> 2, wk = wave & 3;                      // 128 n, 64 k of the tile
    const int64_t n0 = (int64_t)w.tn * kDwTile, k0 = (int64_t)w.tk * kDwTile;
    int64_t r0, r1;
    expert_range(a, w.e, r0, r1);
    int nk = (int)((r1 - r0 + kStageRows - 1) / kStageRows);
    if (OUT == kOutPartial) {
        const int per = (nk + a.slices - 1) / a.slices, first = min(nk, w.slice * per);
        r0 += (int64_t)first * kStageRows;
        nk = min(nk - first, per);
        r1 = min(r1, r0 + (int64_t)nk * kStageRows);
    }

    // ---- copies: wave w takes rows 4 w .. 4 w + 3 of a stage, two per
    // instruction; lane L fetches row L / 32, physical chunk L % 32
    const uint32_t lds_base = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)&lds[0];
    uint32_t cy[2], cx[2];                                        // byte of the row, kOOB past the last column
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t r = (uint32_t)(2 * i) + ((uint32_t)ln >> 5);            // row % 4
        const uint32_t c = ((uint32_t)ln & 31u) ^ (r << 2);
        cy[i] = n0 + c * 8 < a.N ? (uint32_t)(n0 + c * 8) * 2u : kOOB;
        cx[i] = k0 + c * 8 < a.K ? (uint32_t)(k0 + c * 8) * 2u : kOOB;
    }
    const uint32_t ldy = (uint32_t)a.ldy * 2u, ldx = (uint32_t)a.ldx * 2u;
    const v4i rs_all = make_rsrc(a.x, GATHER && a.x_rows > 0 ? (uint32_t)((a.x_rows - 1) * a.ldx + a.K) * 2u : 0u);
    // the stage's row numbers of this wave's four rows, -1 past the last one
    // (scalar loads: they do not enter the count of copies in flight)
    typedef const __attribute__((address_space(4))) int32_t *Indices;
    const Indices row_index = (Indices)(uintptr_t)a.row_index;
    auto indices = [&](int st, int32_t (&idx)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = r0 + (int64_t)st * kStageRows + wave * 4 + i;
            const int32_t v = row_index[r < r1 ? r : r1 - 1];     // (called with r1 > r0)
            idx[i] = r < r1 && v >= 0 && (int64_t)v < a.x_rows ? v : -1;
        }
    };
    auto issue = [&](int st, int slot, const int32_t (&idx)[4]) {
        const uint32_t base =
            (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds_base + (uint32_t)(slot * kSlotBytes + wave * 4 * kLdsRow)));
        const int64_t r = r0 + (int64_t)st * kStageRows;
        const int left = (int)max((int64_t)0, min((int64_t)kStageRows, r1 - r));
        const int64_t rb = left > 0 ? r : 0;
        const v4i rs_y = make_rsrc(a.dy + rb * a.ldy, left > 0 ? (uint32_t)((left - 1) * a.ldy + a.N) * 2u : 0u);
        const v4i rs_x = GATHER ? rs_all
                                : make_rsrc(a.x + rb * a.ldx, left > 0 ? (uint32_t)((left - 1) * a.ldx + a.K) * 2u : 0u);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = wave * 4 + 2 * i + (ln >> 5);
            dma16(base + (uint32_t)(2 * i * kLdsRow), row < left && cy[i] != kOOB ? (uint32_t)row * ldy + cy[i] : kOOB, rs_y, 0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = wave * 4 + 2 * i + (ln >> 5);
            bool ok = row < left && cx[i] != kOOB;
            uint32_t off = (uint32_t)row * ldx;
            if (GATHER) {
                const int32_t v = ln < 32 ? idx[2 * i] : idx[2 * i + 1];
                ok = ok && v >= 0;
                off = (uint32_t)v * ldx;
            }
            dma16(base + (uint32_t)(kOperand + 2 * i * kLdsRow), ok ? off + cx[i] : kOOB, rs_x, 0);
        }
    };

    // ---- fragments: of a 32-column block, lane group l / 16 = (g1 g0) holds
    // columns 16 g0 + l % 16, rows 8 g1 .. 8 g1 + 7 of the 16, in two
    // transposing reads of four rows; lane j of a group points at row j / 4,
    // columns 4 (j % 4) ..
    const uint32_t j = (uint32_t)ln & 15u, g0 = ((uint32_t)ln >> 4) & 1u, g1 = (uint32_t)ln >> 5, jr = j >> 2;
    const uint32_t fbase = (8u * g1 + jr) * kLdsRow + 32u * g0 + 8u * (j & 3u);
    uint32_t fy[4], fx[2];
#pragma unroll
    for (int b = 0; b < 4; ++b) fy[b] = fbase + ((uint32_t)(wn * 4) + ((uint32_t)b ^ jr)) * 64u;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint32_t blk = (uint32_t)(wk * 2 + b);
        fx[b] = kOperand + fbase + ((blk & 4u) + ((blk & 3u) ^ jr)) * 64u;
    }
    auto frag = [&](uint32_t at) -> v8bf {
        typedef __attribute__((address_space(3))) v4s *L;
        const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L)(uintptr_t)(lds_base + at));
        const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L)(uintptr_t)(lds_base + at + 4 * kLdsRow));
        return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };

    v16f acc[2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[x][y][i] = 0.0f;

    if (nk > 0) {
        int32_t idx[4] = {-1, -1, -1, -1};
#pragma unroll
        for (int s = 0; s < kDepth - 1; ++s) {
            if (GATHER) indices(s, idx);
            issue(s, s, idx);
        }
        int slot = 0;
        for (int st = 0; st < nk; ++st) {
            // stage st has landed for every wave, and every wave is done with
            // stage st - 1, whose slot takes stage st + kDepth - 1 (zeros past
            // the last, so that every wait counts the same)
            if (GATHER) indices(st + kDepth - 1, idx);
            wait_vmem<(kDepth - 2) * kCopies>();
            block_barrier();
            issue(st + kDepth - 1, slot == 0 ? kDepth - 1 : slot - 1, idx);
            const uint32_t sb = (uint32_t)(slot * kSlotBytes);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v8bf bx[2], by[4];
#pragma unroll
                for (int b = 0; b < 2; ++b) bx[b] = frag(sb + fx[b] + h * 16 * kLdsRow);
#pragma unroll
                for (int b = 0; b < 4; ++b) by[b] = frag(sb + fy[b] + h * 16 * kLdsRow);
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bx[x], by[y], acc[x][y], 0, 0, 0);
            }
            slot = slot + 1 == kDepth ? 0 : slot + 1;
        }
        wait_vmem<0>();
        wait_lds();
        block_barrier();                                          // the slots become the epilogue's
    }

    // ---- epilogue: lane l of a block holds n = l % 32 and, per register
    // group q, k = 8 q + 4 (l / 32) .. + 3.  32 n x 64 k at a time through
    // the wave's own LDS region (16-byte chunk c of row n at c ^ (n % 16)), so
    // that whole row segments leave.
    float *const region = reinterpret_cast<float *>(&lds[wave * kRegion]);
    const int l32 = ln & 31, kh = ln >> 5;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = x * 8 + q * 2 + kh;
                *reinterpret_cast<v4f *>(region + l32 * 64 + ((c ^ (l32 & 15)) << 2)) =
                    v4f{acc[x][y][4 * q], acc[x][y][4 * q + 1], acc[x][y][4 * q + 2], acc[x][y][4 * q + 3]};
            }
        const int nb = wn * 128 + y * 32, kb = wk * 64;
        if (OUT == kOutPartial) {
            const int64_t tile = ((int64_t)w.e * a.tiles_n + w.tn) * a.tiles_k + w.tk;
            float *const p = a.partials + (tile * a.slices + w.slice) * (kDwTile * kDwTile);
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                const int r = it * 4 + (ln >> 4), c = ln & 15;
                *reinterpret_cast<v4f *>(p + (nb + r) * kDwTile + kb + c * 4) =
                    *reinterpret_cast<const v4f *>(region + r * 64 + ((c ^ (r & 15)) << 2));
            }
        } else if (OUT == kOutBf16) {
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int r = it * 8 + (ln >> 3), c = (ln & 7) * 2;
                const v4f lo = *reinterpret_cast<const v4f *>(region + r * 64 + ((c ^ (r & 15)) << 2));
                const v4f hi = *reinterpret_cast<const v4f *>(region + r * 64 + (((c + 1) ^ (r & 15)) << 2));
                const int64_t n = n0 + nb + r, k = k0 + kb + c * 4;
                if (n < a.N && k < a.K) store_chunk<kOutBf16>(a, w.e, n, k, lo, hi);
            }
        } else {
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                const int r = it * 4 + (ln >> 4), c = ln & 15;
                const v4f lo = *reinterpret_cast<const v4f *>(region + r * 64 + ((c ^ (r & 15)) << 2));
                const int64_t n = n0 + nb + r, k = k0 + kb + c * 4;
                if (n < a.N && k < a.K) store_chunk<kOutFp32>(a, w.e, n, k, lo, lo);
            }
        }
    }
}

// Sums the slices' partial tiles in their order: a workgroup per 16 rows of a
// tile, eight columns of one row per thread and step.
template <int OUT>
__global__ __launch_bounds__(256) void grouped_dw_reduce_kernel(const GroupedDwArgs a)
{
    const uint32_t tile = blockIdx.x >> 4;
    const uint32_t row = fdiv(tile, a.div_k), tk = tile - row * a.tiles_k;
    const uint32_t e = fdiv(row, a.div_n), tn = row - e * a.tiles_n;
    const float *p = a.partials + (int64_t)tile * a.slices * (kDwTile * kDwTile);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = (int)(blockIdx.x & 15u) * 16 + i * 8 + (int)(threadIdx.x >> 5), c = (int)(threadIdx.x & 31u) * 8;
        const int64_t n = (int64_t)tn * kDwTile + r, k = (int64_t)tk * kDwTile + c;
        if (n >= a.N || k >= a.K) continue;
        v4f lo = {}, hi = {};
        for (int s = 0; s < a.slices; ++s) {
            const float *q = p + (int64_t)s * (kDwTile * kDwTile) + r * kDwTile + c;
            lo += __builtin_nontemporal_load(reinterpret_cast<const v4f *>(q));
            hi += __builtin_nontemporal_load(reinterpret_cast<const v4f *>(q + 4));
        }
        store_chunk<OUT>(a, (int)e, n, k, lo, hi);
        if (OUT == kOutFp32) store_chunk<OUT>(a, (int)e, n, k + 4, hi, hi);
    }
}

template <int OUT>
hipError_t launch_out(const GroupedDwArgs &a, unsigned grid, hipStream_t s)
{
    if (a.row_index)
        grouped_dw_kernel<OUT, true><<<grid, kDwThreads, 0, s>>>(a);
    else
        grouped_dw_kernel<OUT, false><<<grid, kDwThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_dw(const GroupedDwArgs &a, hipStream_t s)
{
    // whole rounds of the eight XCDs; workgroups without a row of tiles end at once
    const int64_t rows = (int64_t)a.E * a.slices * a.tiles_n;
    const unsigned grid = (unsigned)((rows + 7) / 8 * 8 * a.tiles_k);
    if (a.slices == 1) return a.out_fp32 ? launch_out<kOutFp32>(a, grid, s) : launch_out<kOutBf16>(a, grid, s);
    hipError_t e = launch_out<kOutPartial>(a, grid, s);
    if (e != hipSuccess) return e;
    const unsigned parts = (unsigned)((int64_t)a.E * a.tiles_n * a.tiles_k * 16);
    if (a.out_fp32)
        grouped_dw_reduce_kernel<kOutFp32><<<parts, 256, 0, s>>>(a);
    else
        grouped_dw_reduce_kernel<kOutBf16><<<parts, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace spg
