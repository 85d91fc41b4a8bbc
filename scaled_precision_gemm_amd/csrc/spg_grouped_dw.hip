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
//  * 256 x 256 tiles of dW_e (128 x 256 where those are few) over eight waves
//    (two a SIMD), each 128 n x 64 k as 4 x 2 blocks of
//    v_mfma_f32_32x32x16_bf16: 128 accumulators a lane.  X is the first MFMA
//    operand, so a lane's four consecutive results are four consecutive k of
//    one row n.
//  * A stage is 32 rows of both operands, 32 KiB, copied straight into one of
//    kDepth LDS slots (buffer loads to LDS).  Rows past the expert's last
//    one are out of the buffer's range and read as zeros in both operands, so
//    whatever stands in the rows behind is not multiplied.
//  * LDS row r holds its 16-byte chunk c at c ^ 4 (r % 4): a transposing read
//    takes 64 bytes of four consecutive rows 512 bytes apart, which then lie
//    in four different quarters of the 64 banks.
//  * Experts' rows are read from the offsets on the device, so a captured graph
//    serves any routing.  Workgroups stay and take tile after tile, copying the
//    next one's first stages under the last one's end.
//
// What bounds it (cycles of the shader clock and that clock, stamped in the same
// launches): long sums the power limit, 32768 rows x 4096 x 4096 840-880 us, 1.3
// PFLOP/s: 1275 cycles a stage, MFMAs 1024 of them, at 1.61 GHz (three, four or
// five slots alike).  64 experts' 2048 x 2048 over 32768 gathered rows, 330 us, its
// stages: a tile takes 37300 cycles at 1.93 GHz, 45 % MFMAs.  Of its 16.5 stages the
// two behind an epilogue take 2190 each, the next two 1820, the others 1740 (with
// copies that all hit the L2 1540); the epilogue 3500 and 1540 waiting before it,
// 2470 to the next tile's first stage.  Equal experts, rows in order: 1410 a stage at
// 1.72 GHz, 290-315 us.  128 x 256 tiles, 4096 x 2048 over 4000 rows: 920 a stage, MFMAs
// 512, at 1.78-1.83 GHz (copies from the L2: 900).  So most of what stages wait for
// lies between LDS and registers.  Added fp32 gradients: the epilogue, 31000-36000
// cycles a tile, the memory's rate.  Few rows an expert: the output at 5.2 TB/s.
// Gathered, added, fp32 tiles of 256 x 256 spill 8 registers (64 x 2048 x 2048 over 32768
// rows 540 us, of which 2.3 GB at the memory's rate are 440).
#include "spg_gemm_common.h"
#include "spg_grouped_dw.h"

#include <type_traits>

namespace spg {

namespace {

using namespace gemm;

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kDwThreads = 512, kDwWaves = 8;
constexpr int kStageRows = 32;
constexpr int kDepth = 4;
constexpr int kRegion = 4096;                                    // epilogue: 32 n x 64 k bf16, 32 n x 32 k fp32

// Tiles of TN n x 256 k.
template <int TN>
struct DwGeometry {
    static constexpr int kRowY = TN * 2, kRowX = 512;            // LDS rows
    static constexpr int kY = kStageRows * kRowY, kX = kStageRows * kRowX;
    static constexpr int kSlot = kY + kX;
    static constexpr int kRowsPerCopy = 1024 / kRowY;            // of dY: a copy instruction moves 1 KiB
    static constexpr int kCopyY = 4 / kRowsPerCopy, kCopyX = 2;  // of a wave per stage: its four rows
    static constexpr int kCopies = kCopyY + kCopyX;
    static constexpr int kWaveN = TN / 2, kBlocksY = kWaveN / 32;   // n of a wave
    // the epilogue's regions: the free slot, and where that is smaller LDS of their own behind the slots
    static constexpr int kOwnRegions = kDwWaves * kRegion > kSlot ? kDwWaves * kRegion : 0;
};
// row numbers of 32 stages of one wave's four rows, two such chunks
constexpr int kChunkStages = 32, kIndexBytes = kChunkStages * 4 * 4;

enum { kOutBf16, kOutFp32, kOutPartial };

// 64 consecutive experts from `base` on, one per lane: their rows (the offsets
// are the caller's device data, clamped to [0, R]; a decreasing pair is an
// empty expert) and their rank among the 64, most rows first.
struct DwExperts {
    int base;
    int32_t first, rows;
    int rank;
};
__device__ __forceinline__ DwExperts dw_experts(const GroupedDwArgs &a, int base)
{
    const int lane = lane_id(), e = base + lane;
    const int32_t R = (int32_t)a.R;
    DwExperts w = {base, 0, -1, 0};
    if (e < a.E) {
        w.first = min(max(a.offsets[e], 0), R);
        w.rows = max(min(max(a.offsets[e + 1], 0), R) - w.first, 0);
    }
    const int n = min(64, a.E - base);
    for (int i = 0; i < n; ++i) {
        const int32_t r = __builtin_amdgcn_readlane(w.rows, i);
        w.rank += r > w.rows || (r == w.rows && i < lane) ? 1 : 0;
    }
    return w;
}

// One tile of an expert's gradient, over rows r0 .. r1 - 1: nk stages, of
// which the pipeline below takes at least MIN (the last ones copy and add
// nothing).
struct DwTile {
    int e, slice;
    uint32_t tn, tk;
    int64_t r0, r1;
    int nk, np;
};

// Tile i of this XCD's list (dw_place).
template <int OUT, int MIN>
__device__ __forceinline__ DwTile dw_tile(const GroupedDwArgs &a, DwExperts &w, uint32_t i)
{
    const DwPlace at = dw_place(a, blockIdx.x & 7u, i);
    const int place = (int)at.place;
    DwTile t;
    t.tk = at.tk;
    t.tn = at.tn;
    t.slice = (int)at.slice;
    t.e = -1;
    t.r0 = t.r1 = 0;
    t.nk = 0;
    if (place < a.E) {
        if ((place & ~63) != w.base) w = dw_experts(a, place & ~63);
        const int src = __builtin_ctzll(__ballot(w.rank == (place & 63) && w.rows >= 0));
        t.e = w.base + src;
        t.r0 = __builtin_amdgcn_readlane(w.first, src);
        t.r1 = t.r0 + __builtin_amdgcn_readlane(w.rows, src);
        t.nk = (int)((t.r1 - t.r0 + kStageRows - 1) / kStageRows);
        if (OUT == kOutPartial) {
            const int per = (t.nk + a.slices - 1) / a.slices, first = min(t.nk, t.slice * per);
            t.r0 += (int64_t)first * kStageRows;
            t.nk = min(t.nk - first, per);
            t.r1 = min(t.r1, t.r0 + (int64_t)t.nk * kStageRows);
        }
    }
    t.np = max(t.nk, MIN);
    return t;
}

template <int TN, int OUT, bool GATHER, bool ADD>
__global__ __launch_bounds__(kDwThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void grouped_dw_kernel(
    const GroupedDwArgs a)
{
    using G = DwGeometry<TN>;
    constexpr int kIndexAt = kDepth * G::kSlot + G::kOwnRegions;
    __shared__ __attribute__((aligned(2048))) uint8_t lds[kIndexAt + (GATHER ? kDwWaves * 2 * kIndexBytes : 0)];
    constexpr int kMin = GATHER ? 7 : 3;                          // (gathered: so that plan() need not wait)
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), ln = lane_id();
    const int wn = wave >> 2, wk = wave & 3;                      // TN / 2 n, 64 k of the tile
    const uint32_t lds_base = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)&lds[0];

    // ---- this workgroup's tiles: one of every `step` of its XCD's, from the
    // front and from the back in turn: with the experts in the order of their
    // rows, all workgroups get about as much
    DwExperts experts = dw_experts(a, 0);
    uint32_t round = 0;
    auto tile = [&](uint32_t k) { return dw_tile<OUT, kMin>(a, experts, dw_item(gridDim.x, blockIdx.x, k)); };
    DwTile cur = tile(0);
    if (cur.e < 0) return;
    DwTile nxt = tile(++round);

    // ---- copies: wave w takes rows 4 w .. 4 w + 3 of a stage, 1 KiB per
    // instruction: X two rows (lane L row L / 32, physical chunk L % 32), dY two
    // or four.  They run kDepth stages ahead, across the border of two tiles.
    constexpr uint32_t kLanesY = G::kRowY / 16;                   // lanes of a row of dY
    const uint32_t ryl = (uint32_t)ln / kLanesY, rxl = (uint32_t)ln >> 5;
    const uint32_t ldy = (uint32_t)a.ldy * 2u, ldx = (uint32_t)a.ldx * 2u;
    const v4i rs_all = make_rsrc(a.x, GATHER && a.x_rows > 0 ? (uint32_t)((a.x_rows - 1) * a.ldx + a.K) * 2u : 0u);
    struct {
        const uint16_t *y, *x;                                    // the next stage's first rows
        int rows;                                                 // of the tile from there on; not above 0: none
        int left, at, buf;                                        // stages left; stage of the tile; index buffer
        uint32_t vy[G::kCopyY], vx[2];                            // byte offsets of the lane's chunks (gathered X: in its row)
        uint32_t most[2];                                         // gathered X: rows that the lane may read, 0 past K
    } cp;
    auto copy_tile = [&](const DwTile &t) {
        cp.y = a.dy + t.r0 * a.ldy;
        cp.x = a.x + (GATHER ? 0 : t.r0 * a.ldx);
        cp.rows = (int)(t.r1 - t.r0);
        cp.left = t.np;
        cp.at = 0;
#pragma unroll
        for (int i = 0; i < G::kCopyY; ++i) {
            const uint32_t r = (uint32_t)(G::kRowsPerCopy * i) + ryl;      // row % 4
            const uint32_t c = t.tn * TN + ((((uint32_t)ln % kLanesY) ^ (r << 2)) << 3);
            cp.vy[i] = c < (uint32_t)a.N ? ((uint32_t)(wave * 4) + r) * ldy + c * 2u : kOOB;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t r = (uint32_t)(2 * i) + rxl;
            const uint32_t c = t.tk * kDwTile + ((((uint32_t)ln & 31u) ^ (r << 2)) << 3);
            cp.most[i] = c < (uint32_t)a.K ? (uint32_t)a.x_rows : 0u;
            cp.vx[i] = c < (uint32_t)a.K ? (GATHER ? 0u : ((uint32_t)(wave * 4) + r) * ldx) + c * 2u : kOOB;
        }
    };
    copy_tile(cur);
    cp.buf = 0;
    const uint32_t index_at = lds_base + (uint32_t)(kIndexAt + wave * 2 * kIndexBytes);
    // row numbers of chunk c of a tile's rows into buffer buf: each wave those
    // of its own rows, read back by itself.  `since` counts the stages copied
    // after them.  A stage's copies are planned ahead of its own wait: four
    // stages after, the waits of the stages before have seen the row numbers
    // land (the first two stages of a tile have none); sooner, plan() waits.
    int since = 0;
    auto copy_indices = [&](int64_t r0, int64_t r1, int c, int buf) {
        const int64_t first = r0 + (int64_t)c * (kChunkStages * kStageRows);
        const int64_t n = max((int64_t)0, min(r1 - first, (int64_t)(kChunkStages * kStageRows)));
        const v4i rs = make_rsrc(a.row_index + (n > 0 ? first : 0), (uint32_t)n * 4u);
        const uint32_t base = (uint32_t)__builtin_amdgcn_readfirstlane((int)(index_at + (uint32_t)(buf * kIndexBytes)));
#pragma unroll
        for (int k = 0; k < 2; ++k)
            dma4(base + 256u * k, (uint32_t)((16 * k + (ln >> 2)) * kStageRows + wave * 4 + (ln & 3)) * 4u, rs, 0);
        since = 0;
    };
    // What the next stage's copies take, worked out ahead of the barrier that
    // frees their slot, in three parts that stand behind MFMAs of their own (in
    // one, the vector instructions of both waves of a SIMD held its matrix core
    // up: 64 x 2048 x 2048 bf16 over 32768 gathered rows 340 us, 333 so); then copy
    // instruction i of the stage's.  Rows past the tile's last one are past the
    // buffers' ranges.
    struct {
        v4i y, x;
        uint32_t live, vx[2];
        int32_t row[2];
    } pl;
    auto plan = [&](int part) {
        if (part == 0) {
            const bool border = cp.left == 0, chunk = cp.at > 0 && cp.at % kChunkStages == 0;
            if (GATHER && (border || chunk)) {
                if (since < 4) wait_vmem<0>();
                cp.buf ^= 1;
            }
            if (border) copy_tile(nxt);
            pl.live = (uint32_t)max(0, min(kStageRows, cp.rows));
            pl.y = make_rsrc(cp.y, pl.live * ldy);
            pl.x = GATHER ? rs_all : make_rsrc(cp.x, pl.live * ldx);
            if (GATHER) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    pl.row[i] = *reinterpret_cast<const int32_t *>(
                        &lds[kIndexAt + (wave * 2 + cp.buf) * kIndexBytes + ((cp.at % kChunkStages) * 4 + 2 * i + (ln >> 5)) * 4]);
            }
        } else {
            const int i = part - 1;
            pl.vx[i] = cp.vx[i];
            if (GATHER) {
                const bool ok = wave * 4 + 2 * i + (ln >> 5) < (int)pl.live && (uint32_t)pl.row[i] < cp.most[i];
                pl.vx[i] = ok ? (uint32_t)pl.row[i] * ldx + cp.vx[i] : kOOB;
            }
        }
    };
    auto issue_one = [&](int slot, int i) {
        const uint32_t base =
            (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds_base + (uint32_t)(slot * G::kSlot)));
        if (i < G::kCopyY)
            dma16(base + (uint32_t)(wave * 4 * G::kRowY + i * 1024), cp.vy[i < G::kCopyY ? i : 0], pl.y, 0);
        else
            dma16(base + (uint32_t)(G::kY + wave * 4 * G::kRowX + (i - G::kCopyY) * 1024), pl.vx[(i - G::kCopyY) & 1], pl.x, 0);
    };
    auto advance = [&]() {
        ++since;
        // the first stage of a later chunk: the chunk after it
        if (GATHER && cp.at > 0 && cp.at % kChunkStages == 0) {
            const int c = cp.at / kChunkStages + 1;
            if (c * kChunkStages < cur.np)
                copy_indices(cur.r0, cur.r1, c, cp.buf ^ 1);
            else
                copy_indices(nxt.r0, nxt.r1, 0, cp.buf ^ 1);
        }
        cp.y += kStageRows * a.ldy;
        if (!GATHER) cp.x += kStageRows * a.ldx;
        cp.rows -= kStageRows;
        ++cp.at;
        --cp.left;
    };
    auto issue = [&](int slot) {
#pragma unroll
        for (int part = 0; part < 3; ++part) plan(part);
#pragma unroll
        for (int i = 0; i < G::kCopies; ++i) issue_one(slot, i);
        advance();
    };

    // ---- fragments: of a 32-column block, lane group l / 16 = (g1 g0) holds
    // columns 16 g0 + l % 16, rows 8 g1 .. 8 g1 + 7 of the 16, in two
    // transposing reads of four rows; lane j of a group points at row j / 4,
    // columns 4 (j % 4) ..
    const uint32_t j = (uint32_t)ln & 15u, g0 = ((uint32_t)ln >> 4) & 1u, g1 = (uint32_t)ln >> 5, jr = j >> 2;
    const uint32_t frow = 8u * g1 + jr, fcol = 32u * g0 + 8u * (j & 3u);
    uint32_t fy[G::kBlocksY], fx[2];
#pragma unroll
    for (int b = 0; b < G::kBlocksY; ++b) {
        const uint32_t blk = (uint32_t)(wn * G::kBlocksY + b);
        fy[b] = frow * G::kRowY + fcol + ((blk & 4u) + ((blk & 3u) ^ jr)) * 64u;
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint32_t blk = (uint32_t)(wk * 2 + b);
        fx[b] = G::kY + frow * G::kRowX + fcol + ((blk & 4u) + ((blk & 3u) ^ jr)) * 64u;
    }
    auto frag = [&](uint32_t at, uint32_t four_rows) -> v8bf {
        typedef __attribute__((address_space(3))) v4s *L;
        const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L)(uintptr_t)(lds_base + at));
        const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L)(uintptr_t)(lds_base + at + four_rows));
        return __builtin_bit_cast(v8bf, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    constexpr int kYB = G::kBlocksY, kFrags = 2 + kYB, kMfma = 2 * kYB;   // of a step
    v8bf bx[2][2], by[2][kYB];
    auto read_frag = [&](uint32_t sb, int h, int i) {             // i: 0, 1 X blocks, then Y blocks
        if (i < 2)
            bx[h][i & 1] = frag(sb + (uint32_t)(h * 16 * G::kRowX) + fx[i & 1], 4 * G::kRowX);
        else
            by[h][(i - 2) & (kYB - 1)] = frag(sb + (uint32_t)(h * 16 * G::kRowY) + fy[(i - 2) & (kYB - 1)], 4 * G::kRowY);
    };

    // ---- the pipeline.  One stage is two steps of 16 rows, each 8 MFMAs (128
    // n: 4), m = 2 y + x; the next step's fragments are read under this step's MFMAs.
    // Before the second step all of the stage's fragments are in registers
    // and this wave's copies of the next stage have landed -> barrier: the
    // slot is free, the next stage is published, and under the second step the
    // copies of stage st + kDepth go into the slot.  The scheduling barriers
    // pin that order (the compiler otherwise reads each fragment right before
    // its MFMA); hazards and the waits of LDS reads are the compiler's.
    //
    // A tile's last kDepth stages copy the next tile's first ones, but for the
    // very last: its slot is the epilogue's.  Before the epilogue all copies
    // in flight have landed (stages 0 .. 2 of the next tile), so that the
    // first two stages after it need no wait: one would wait for the
    // epilogue's stores as well, which share the counter.
    v16f acc[2][kYB];
    int slot = 0;
    auto stage = [&](auto real_c, int st) {
        constexpr bool REAL = decltype(real_c)::value;
        const int next = slot + 1 == kDepth ? 0 : slot + 1;
        const uint32_t sb = (uint32_t)(slot * G::kSlot), nb = (uint32_t)(next * G::kSlot);
        const bool more = st != cur.np - 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h == 1) {
                wait_lds();
                if (st >= 2) wait_vmem<(kDepth - 2) * G::kCopies>();
                block_barrier();
            }
#pragma unroll
            for (int m = 0; m < kMfma; ++m) {
                const int y = m >> 1, x = m & 1;
                if (REAL) acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bx[h][x], by[h][y], acc[x][y], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
                constexpr int kPer = (kFrags + kMfma - 1) / kMfma;      // fragments read per MFMA
#pragma unroll
                for (int i = m * kPer; i < (m + 1) * kPer && i < kFrags; ++i)
                    if (REAL || h == 1) read_frag(h == 0 ? sb : nb, h ^ 1, i);
                if (h == 0 && m >= kMfma - 4 && m < kMfma - 1 && more) plan(m - (kMfma - 4));
                if (h == 1 && m < G::kCopies && more) issue_one(slot, m);
                if (h == 1 && m == kMfma - 1 && more) advance();
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        slot = next;
    };

    if (GATHER) {
        copy_indices(cur.r0, cur.r1, 0, 0);
        wait_vmem<0>();
    }
#pragma unroll
    for (int s = 0; s < kDepth - 1; ++s) issue(s);
    wait_vmem<0>();
    block_barrier();
#pragma unroll
    for (int i = 0; i < kFrags; ++i) read_frag(0, 0, i);
    for (;;) {
        // the slot behind the three stages that have landed; the row numbers
        // behind the chunk that the copies are in (the first)
        if (GATHER) {
            if (cur.np > kChunkStages)
                copy_indices(cur.r0, cur.r1, 1, cp.buf ^ 1);
            else
                copy_indices(nxt.r0, nxt.r1, 0, cp.buf ^ 1);
        }
        issue(slot == 0 ? kDepth - 1 : slot - 1);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < kYB; ++y)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[x][y][i] = 0.0f;
        for (int st = 0; st < cur.nk; ++st) stage(std::true_type{}, st);
        for (int st = cur.nk; st < cur.np; ++st) stage(std::false_type{}, st);
        // ---- epilogue: lane l of a block holds n = l % 32 and, per register
        // group q, k = 8 q + 4 (l / 32) .. + 3.  128-byte rows of the output
        // go through the wave's own region (16-byte chunk c of row n at c ^
        // (n / 2 % 8)), so that whole lines leave: passes of 32 n x 64 k (bf16)
        // or x 32 k (fp32).  Where rows begin on lines nothing is read or written
        // twice and both go past the caches (ordinary stores of 64 x 2048 x 2048
        // bf16 with 512 rows an expert 358 us, 323 so); elsewhere neighbouring
        // waves meet in a line, which the L2 has to put together (64 x 1000 x 792
        // bf16, few rows: 54 us past the caches, 28 through them).  What is added is
        // loaded a pass ahead (two passes ahead would spill registers; as the
        // accumulators' first values it came to 290 us where this takes 275: 64
        // experts of 2048 x 1024 in fp32 over 32768 rows).
        const int l32 = ln & 31, kh = ln >> 5, r8 = ln >> 3, c8 = ln & 7;
        const int64_t n0 = (int64_t)cur.tn * TN + wn * G::kWaveN, k0 = (int64_t)cur.tk * kDwTile + wk * 64;
        constexpr int kPasses = OUT == kOutBf16 ? kYB : 2 * kYB, kSize = OUT == kOutBf16 ? 2 : 4;
        // element (pass row it * 8 + r8, 16-byte chunk c8): its n and k
        auto row_of = [&](int p, int it) { return n0 + (OUT == kOutBf16 ? p : p >> 1) * 32 + it * 8 + r8; };
        auto col_of = [&](int p) { return k0 + (OUT == kOutBf16 ? c8 * 8 : (p & 1) * 32 + c8 * 4); };
        v4i ad[2][ADD ? 4 : 1];
        auto load_add = [&](int p) {
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int64_t n = row_of(p, it), k = col_of(p);
                const int64_t at = (int64_t)cur.e * a.stride_a + n * a.lda + k;
                ad[p & 1][ADD ? it : 0] = v4i{0, 0, 0, 0};
                const v4i *const from = reinterpret_cast<const v4i *>((const uint8_t *)a.add + at * kSize);
                if (n < a.N && k < a.K) ad[p & 1][ADD ? it : 0] = a.lines ? __builtin_nontemporal_load(from) : *from;
            }
        };
        if constexpr (ADD) load_add(0);
        wait_vmem<0>();
        uint8_t *const region =
            &lds[(G::kOwnRegions > 0 ? kDepth : slot == 0 ? kDepth - 1 : slot - 1) * G::kSlot + wave * kRegion];
        auto place = [&](int row, int c) { return region + row * 128 + ((c ^ ((row >> 1) & 7)) << 4); };
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (ADD)
                if (p + 1 < kPasses) load_add(p + 1);
            if constexpr (OUT == kOutBf16) {
                if (ADD) {
#pragma unroll
                    for (int it = 0; it < 4; ++it) *reinterpret_cast<v4i *>(place(it * 8 + r8, c8)) = ad[p & 1][ADD ? it : 0];
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint2 *const at = reinterpret_cast<uint2 *>(place(l32, x * 4 + q) + kh * 8);
                        float v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = acc[x][p][4 * q + i];
                        if (ADD) {
                            const uint2 r = *at;
                            v[0] += bf16_lo(r.x);
                            v[1] += bf16_hi(r.x);
                            v[2] += bf16_lo(r.y);
                            v[3] += bf16_hi(r.y);
                        }
                        *at = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                    }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<v4f *>(place(l32, q * 2 + kh)) =
                        v4f{acc[p & 1][p >> 1][4 * q], acc[p & 1][p >> 1][4 * q + 1], acc[p & 1][p >> 1][4 * q + 2],
                            acc[p & 1][p >> 1][4 * q + 3]};
            }
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                v4i v = *reinterpret_cast<const v4i *>(place(it * 8 + r8, c8));
                const int64_t n = row_of(p, it), k = col_of(p);
                if constexpr (OUT == kOutPartial) {
                    const int64_t tile = ((int64_t)cur.e * a.tiles_n + cur.tn) * a.tiles_k + cur.tk;
                    float *const to = a.partials + (tile * a.slices + cur.slice) * (TN * kDwTile);
                    *reinterpret_cast<v4i *>(to + (n - (int64_t)cur.tn * TN) * kDwTile + (k - (int64_t)cur.tk * kDwTile)) = v;
                } else {
                    if (n >= a.N || k >= a.K) continue;
                    if (OUT == kOutFp32 && ADD)
                        v = __builtin_bit_cast(v4i, __builtin_bit_cast(v4f, v) + __builtin_bit_cast(v4f, ad[p & 1][ADD ? it : 0]));
                    const int64_t at = (int64_t)cur.e * a.stride_o + n * a.ldo + k;
                    v4i *const to = reinterpret_cast<v4i *>((uint8_t *)a.out + at * kSize);
                    if (a.lines)
                        __builtin_nontemporal_store(v, to);
                    else
                        *to = v;
                }
            }
        }
        if (nxt.e < 0) break;
        cur = nxt;
        nxt = tile(++round);
        // every wave's copies of the next tile's first three stages have landed,
        // and every wave is done with the epilogue's slot
        wait_lds();
        block_barrier();
    }
}

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

// Sums the slices' partial tiles in their order: a workgroup per 4 rows of a
// tile, eight columns of one row per thread, kBatch slices' loads in flight.
constexpr int kReduceRows = 4, kBatch = 4;
template <int TN, int OUT>
__global__ __launch_bounds__(32 * kReduceRows) void grouped_dw_reduce_kernel(const GroupedDwArgs a)
{
    constexpr uint32_t kParts = TN / kReduceRows;
    const uint32_t tile = blockIdx.x / kParts;
    const uint32_t row = fdiv(tile, a.div_k), tk = tile - row * a.tiles_k;
    const uint32_t e = fdiv(row, a.div_n), tn = row - e * a.tiles_n;
    const int r = (int)(blockIdx.x % kParts) * kReduceRows + (int)(threadIdx.x >> 5), c = (int)(threadIdx.x & 31u) * 8;
    const int64_t n = (int64_t)tn * TN + r, k = (int64_t)tk * kDwTile + c;
    if (n >= a.N || k >= a.K) return;
    const float *p = a.partials + (int64_t)tile * a.slices * (TN * kDwTile) + r * kDwTile + c;
    v4f lo = {}, hi = {};
    for (int s0 = 0; s0 < a.slices; s0 += kBatch) {
        v4f l[kBatch], h[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float *q = p + (int64_t)min(s0 + i, a.slices - 1) * (TN * kDwTile);
            l[i] = *reinterpret_cast<const v4f *>(q);
            h[i] = *reinterpret_cast<const v4f *>(q + 4);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (s0 + i < a.slices) {
                lo += l[i];
                hi += h[i];
            }
    }
    store_chunk<OUT>(a, (int)e, n, k, lo, hi);
    if (OUT == kOutFp32) store_chunk<OUT>(a, (int)e, n, k + 4, hi, hi);
}

template <int TN, int OUT>
hipError_t launch_out(const GroupedDwArgs &a, unsigned grid, hipStream_t s)
{
    if constexpr (OUT != kOutPartial) {
        if (a.add) {
            if (a.row_index)
                grouped_dw_kernel<TN, OUT, true, true><<<grid, kDwThreads, 0, s>>>(a);
            else
                grouped_dw_kernel<TN, OUT, false, true><<<grid, kDwThreads, 0, s>>>(a);
            return hipGetLastError();
        }
    }
    if (a.row_index)
        grouped_dw_kernel<TN, OUT, true, false><<<grid, kDwThreads, 0, s>>>(a);
    else
        grouped_dw_kernel<TN, OUT, false, false><<<grid, kDwThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <int TN>
hipError_t launch_tiles(const GroupedDwArgs &a, hipStream_t s)
{
    const unsigned grid = dw_grid(a);
    if (a.slices == 1) return a.out_fp32 ? launch_out<TN, kOutFp32>(a, grid, s) : launch_out<TN, kOutBf16>(a, grid, s);
    hipError_t e = launch_out<TN, kOutPartial>(a, grid, s);
    if (e != hipSuccess) return e;
    const unsigned parts = (unsigned)((int64_t)a.E * a.tiles_n * a.tiles_k * (TN / kReduceRows));
    if (a.out_fp32)
        grouped_dw_reduce_kernel<TN, kOutFp32><<<parts, 32 * kReduceRows, 0, s>>>(a);
    else
        grouped_dw_reduce_kernel<TN, kOutBf16><<<parts, 32 * kReduceRows, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_dw(const GroupedDwArgs &a, hipStream_t s)
{
    return a.tile_n == 256 ? launch_tiles<256>(a, s) : launch_tiles<128>(a, s);
}

}  // namespace spg
