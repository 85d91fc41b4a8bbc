// Block-scaled FP8 product over tiles, dense and per expert (see
// spg_gemm_block_common.h for the arithmetic).
//
// Design for CDNA4:
//  * Tiles of BM x 256 (BM = 256 or 128 token rows, 256 weight rows) over
//    eight waves, four token strips x two weight halves, two waves per SIMD:
//    while one wave waits (for LDS, a barrier, its own results) the other
//    feeds the matrix core.  A wave holds BM / 4 tokens x 128 weight rows,
//    at most 128 accumulators per lane: the vector unit adds into them, so
//    they must sit in vector registers, where the 256 accumulators of the
//    row-scaled kernel's 128 x 128 wave tiles would leave no room.
//  * v_mfma_f32_16x16x128_f8f6f4: one instruction per 16 x 16 block and
//    group, so a partial product P is four registers.  (32 x 32 blocks need
//    two instructions and sixteen registers per P; with the fragments read
//    ahead that spilled 60 registers.)
//  * W fragments are the first MFMA operand, so a lane holds one token of a
//    block and its factor sa[token] sw[block] is one register for all four
//    values of P.
//  * K advances one group (128 bytes) per stage.  Codes and scales go
//    straight into LDS (buffer loads to LDS), DEPTH slots, one barrier per
//    stage (see the schedule below).
//  * What bounds it: the matrix core at the clock that the card's power
//    allows.  4096 x 34816 x 5120 SWIGLU: 590 us in a burst, 617 - 656
//    us (2.3 PFLOP/s) sustained; the row-scaled kernel 552.  MFMAs are busy 55 -
//    58 % of the cycles (row-scaled 64 %) and the vector unit, whose four
//    multiply-adds of a partial product take half of a 16 x 16 x 128 MFMA's
//    cycles, 50 %; a tile's fill and epilogue take 6.8 us beside 1.57 us a
//    stage.  4096 x 5120 x 6144 ADD 129 us, 8192^3 417 - 428 us (2.6 PFLOP/s).
//    128-row tiles take 0.92 us a stage, half the work, with MFMAs busy 36 % and
//    the vector unit 32 % (1111 x 7168 x 5120): neither is what they wait for.
//  * Experts' products: a workgroup finds its (expert, rows) tile from the
//    offsets in device memory, and gathers A rows by index with per-lane copy
//    addresses; the grid is the largest that the row count allows, and
//    workgroups past the last tile end at once.
#include "spg_gemm_block_common.h"

namespace spg {

namespace {

using namespace block;

constexpr int kBK = 128;

template <int BM>
struct Geometry {
    static constexpr int kWaves = 8, kThreads = 64 * kWaves;
    static constexpr int kStrip = BM / 4;                   // token rows of a wave
    static constexpr int kY = kStrip / 16;                  // 16-token blocks of a wave
    static constexpr int kA = BM * kBK;                     // code bytes of a slot: A
    static constexpr int kW = 256 * kBK;                    // and W
    static constexpr int kScales = kWaves * 256;            // per wave one 256-byte line of token scales, one of
    static constexpr int kSlot = kA + kW + 2 * kScales;     // weight scales
    static constexpr int kDepth = BM == 256 ? 2 : 3;
    static constexpr int kCopyA = BM / kWaves / 8;          // copy instructions of a wave per stage: A
    static constexpr int kCopyW = 256 / kWaves / 8;         // W
    static constexpr int kCopies = kCopyA + kCopyW + 2;     // and the two scale lines
    // weight blocks read ahead: one block is kY MFMAs, and two of kY == 2 are
    // less than an LDS read takes (128-row tiles: 41.9 us a call with two
    // blocks ahead, 39.9 with four, 128 x 34816 x 5120 SWIGLU); four of kY == 4
    // would need 32 more registers than there are
    static constexpr int kAhead = kY == 4 ? 2 : 4;
    static constexpr int kLds = kDepth * kSlot;
    // after the main loop: a staging region of kY 4 KiB passes per wave and
    // the biases
    static constexpr int kRegion = kY * 4096, kBias = kWaves * kRegion;
    static_assert(kBias + kWaves * 512 <= kLds, "the epilogue's LDS fits in the slots");
    static_assert(kSlot % 256 == 0, "a slot starts on LDS bank 0");
};

// One tile: rows T.m0 .. m_end - 1 (at most BM) x 256 weight rows, K slice
// `split`.
template <int EPI, int BM, bool EXPERTS, bool SPLIT, bool SO>
__device__ __forceinline__ void block_tile(const BlockArgs &a, const Tile &T, int64_t m_end, int split, uint8_t *lds)
{
    using G = Geometry<BM>;
    constexpr bool SW = EPI == SPG_EPI_SWIGLU;
    const GemmArgs &g = a.g;
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int ln = lane_id();
    const int k0g = SPLIT ? split * (int)(g.k_chunk / kBK) : 0;                    // first group
    const int nk = SPLIT ? min(a.groups - k0g, (int)(g.k_chunk / kBK)) : a.groups;
    const int64_t Nh = g.N / 2;

    // ---- copies -------------------------------------------------------------
    // Wave w copies tile rows [w * 8 kCopyA, ..) of A and [w * 8 kCopyW, ..)
    // of W, eight rows (1 KiB) per instruction: lane L fetches for LDS row
    // L / 8, physical chunk L % 8, i.e. logical chunk (L % 8) ^ ((row >> 1) & 7).
    const uint32_t rib = (uint32_t)ln >> 3, pch = (uint32_t)ln & 7;
    const uint32_t c_even = pch ^ (((uint32_t)ln >> 4) & 7u);
    const uint32_t c_odd = pch ^ ((4u + ((uint32_t)ln >> 4)) & 7u);
    const uint8_t *Ab = g.A + ((!EXPERTS && g.stride_a) ? T.b * g.stride_a : 0);
    const uint8_t *Wb = g.W + (g.stride_w ? T.b * g.stride_w : 0);
    const bool gather = EXPERTS && a.row_index != nullptr;
    const int64_t a_rows = min((int64_t)BM, m_end - T.m0);
    const v4i rs_a = gather ? make_rsrc(Ab, (uint32_t)(a.a_rows * g.lda))
                            : make_rsrc(Ab + T.m0 * g.lda, (uint32_t)(a_rows * g.lda));
    uint32_t va[G::kCopyA];
#pragma unroll
    for (int i = 0; i < G::kCopyA; ++i) {
        const uint32_t r = (uint32_t)(wave * 8 * G::kCopyA + 8 * i) + rib;
        uint32_t src = r;
        bool ok = (int64_t)r < a_rows;
        if (gather) {
            const int32_t x = ok ? a.row_index[T.m0 + r] : -1;
            ok = x >= 0 && (int64_t)x < a.a_rows;
            src = (uint32_t)x;
        }
        va[i] = ok ? src * (uint32_t)g.lda + ((i & 1) ? c_odd : c_even) * 16u : kOOB;
    }
    // W rows of this wave: 128-row halves (SWIGLU: gate rows n0 .., up rows
    // N / 2 + n0 ..), each with its own range
    constexpr int kWRows = 8 * G::kCopyW;                  // rows per wave, a divisor of 128
    const int w_half = (wave * kWRows) >> 7, w_in = (wave * kWRows) & 127;
    const int64_t w_first = SW ? (w_half ? Nh : 0) + T.n0 : T.n0 + w_half * 128;
    const int64_t w_rows = max((int64_t)0, min((int64_t)128, SW ? Nh - T.n0 : g.N - w_first));
    const v4i rs_w = make_rsrc(Wb + w_first * g.ldw, (uint32_t)(w_rows * g.ldw));
    uint32_t vw[2];
    vw[0] = (uint32_t)(w_in + (int)rib) * (uint32_t)g.ldw + c_even * 16u;
    vw[1] = (uint32_t)(w_in + (int)rib) * (uint32_t)g.ldw + c_odd * 16u;
    // scales: lane l the token scale of the wave's row l, lanes 0 .. 3 the
    // weight scales of its four 32-row blocks
    const float *sa = (const float *)g.sa + T.b * g.sa_bstride;
    const float *sw = (const float *)g.sw + T.b * g.sw_bstride;
    uint32_t vsa, vsw = kOOB;
    {
        const uint32_t r = (uint32_t)(wm * G::kStrip + ln);
        uint32_t src = r;
        bool ok = ln < G::kStrip && (int64_t)r < a_rows;
        if (gather) {
            const int32_t x = ok ? a.row_index[T.m0 + r] : -1;
            ok = x >= 0 && (int64_t)x < a.a_rows;
            src = (uint32_t)x;
        }
        vsa = ok ? src * 4u : kOOB;
        if (ln < 4) {
            const int tr = wtile_row0<EPI>(wn, ln);        // tile row of the lane's block
            const int64_t row = SW ? (tr < 128 ? T.n0 + tr : Nh + T.n0 + tr - 128) : T.n0 + tr;
            if (SW ? T.n0 + (tr & 127) < Nh : row < g.N) vsw = (uint32_t)(row >> 7) * (uint32_t)a.sw_rs * 4u;
        }
    }
    const float *sa_tile = gather ? sa : sa + T.m0;
    const uint32_t sa_bytes = (uint32_t)((gather ? a.a_rows : a_rows) * 4);
    const v4i rs_sw = make_rsrc(sw, (uint32_t)a.sw_words * 4u);

    const uint32_t lds_base = (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)&lds[0];
    // Copies of stage kt (0 .. nk - 1; others copy zeros, so that every wait
    // counts the same): the lane conditions and scalar offsets, then copy
    // instruction idx (A, W, token scales, weight scales) into slot `slot`.
    struct StageCopy {
        uint32_t soff, sw_off;
        bool live, in_e, in_o;
        v4i rs_sa;
    };
    auto plan = [&](int kt) -> StageCopy {
        StageCopy c;
        c.live = kt < nk;
        const int64_t kg = c.live ? k0g + kt : 0;
        const uint32_t left = c.live ? (uint32_t)min(g.K - kg * kBK, (int64_t)kBK) : 0;   // bytes of the group
        c.in_e = c_even * 16 < left;
        c.in_o = c_odd * 16 < left;
        c.soff = (uint32_t)kg * kBK;
        c.sw_off = (uint32_t)kg * (uint32_t)a.sw_gs * 4u;
        c.rs_sa = make_rsrc(sa_tile + kg * a.a_rows, sa_bytes);
        return c;
    };
    auto issue_one = [&](const StageCopy &c, int slot, int idx) {
        const uint32_t base = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds_base + (uint32_t)(slot * G::kSlot)));
        if (idx < G::kCopyA)
            dma16(base + (uint32_t)((wave * 8 * G::kCopyA + 8 * idx) * kBK),
                  ((idx & 1) ? c.in_o : c.in_e) ? va[idx < G::kCopyA ? idx : 0] : kOOB, rs_a, c.soff);
        else if (idx < G::kCopyA + G::kCopyW) {
            const int i = idx - G::kCopyA;
            dma16(base + (uint32_t)(G::kA + (wave * kWRows + 8 * i) * kBK),
                  ((i & 1) ? c.in_o : c.in_e) ? vw[i & 1] + (uint32_t)(8 * i) * (uint32_t)g.ldw : kOOB, rs_w, c.soff);
        } else if (idx == G::kCopyA + G::kCopyW)
            dma4(base + (uint32_t)(G::kA + G::kW + wave * 256), c.live ? vsa : kOOB, c.rs_sa, 0);
        else
            dma4(base + (uint32_t)(G::kA + G::kW + G::kScales + wave * 256), c.live ? vsw : kOOB, rs_sw, c.sw_off);
    };

    // ---- fragments ------------------------------------------------------------
    // v_mfma_f32_16x16x128_f8f6f4: lane l holds row l % 16 and 32 bytes of
    // the group, the same ones in both operands; which ones is free.  LDS
    // serves a 16-byte read for lanes 0-3, 12-15, 20-27 (then 4-11, 16-19,
    // 28-31, ...) at once, rows 0-3 and 12-15 of one lane group with rows
    // 4-11 of the next: with chunks q and q ^ 2 for lane group l / 16 = (q1
    // q0), q = 4 q1 + q0, the sixteen lanes touch all banks once (chunks 2 q,
    // 2 q + 1 met every bank twice: 68 of 148 M LDS cycles were conflicts).
    // Weight rows are taken with bits 2 and 3 of the row swapped, which makes
    // the results of two token blocks one lane exchange away from the 32 x 32
    // layout that the epilogue takes (below).
    const uint32_t r16 = (uint32_t)ln & 15, kq = (uint32_t)ln >> 4;
    const uint32_t q0 = (kq & 1u) | ((kq & 2u) << 1);
    const uint32_t wr16 = (r16 & 3u) | ((r16 & 4u) << 1) | ((r16 & 8u) >> 1);
    const uint32_t foa = r16 * kBK + ((q0 ^ ((r16 >> 1) & 7u)) << 4);      // second half: chunk ^ 2
    const uint32_t fow = wr16 * kBK + ((q0 ^ ((wr16 >> 1) & 7u)) << 4);
    auto frag = [&](const uint8_t *rows, uint32_t off) -> v8i {
        const uint4 lo = *reinterpret_cast<const uint4 *>(rows + off);
        const uint4 hi = *reinterpret_cast<const uint4 *>(rows + (off ^ 32u));
        return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };

    v4f acc4[8][G::kY];                                    // [16 weight rows][16 tokens]
#pragma unroll
    for (int x = 0; x < 8; ++x)
#pragma unroll
        for (int y = 0; y < G::kY; ++y) acc4[x][y] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    // One stage is 8 kY MFMAs, m = kY X + Y: weight block X (16 rows) times
    // token block Y.  The partial product of MFMA m joins its accumulators -
    // four multiply-adds - under MFMA m + 3, so neither unit waits for the
    // other, and weight fragments are read kAhead blocks ahead:
    //   block X, first MFMA : weight block X + kAhead (X < 8 - kAhead)
    //   before block 8 - kAhead : all of this stage's weight fragments are in
    //                   registers and this wave's copies of the next stage
    //                   have landed -> barrier: the slot is free, the next
    //                   stage is published
    //   from there on : the copies of stage kt + DEPTH into the freed slot, one
    //                   every kSpread / kCopies MFMAs and on into the next stage
    //                   (the copy path takes 64 bytes a cycle: the waves' 64 or
    //                   48 KiB issued in the MFMAs left of the stage, eight
    //                   each, held them up.  Over 8 | 12 | 16 | 20 | 28 MFMAs,
    //                   us: 4096 x 34816 x 5120 SWIGLU 618 | 605 | 597 | 605 |
    //                   612, later copies landing too late for the barrier;
    //                   128-row tiles, 128 x 34816 x 5120 SWIGLU, 8 | 10 | 12 |
    //                   14 | 16: 40.3 | 39.5 | 36.5 | 35.4 | 35.8);
    //                   the next stage's first weight blocks; its token block Y
    //                   once the last MFMA has taken this stage's; its scales
    // Empty assembly statements pin the order (the compiler otherwise gathers
    // MFMAs and multiply-adds into runs that wait for each other); hazards and
    // waits are still the compiler's.
    constexpr int Y_ = G::kY, kM = 8 * Y_, kBar = (8 - G::kAhead) * Y_, kBufs = 2 * G::kAhead;
    constexpr int kSpread = 16;
    constexpr auto copy_at = [](int idx) { return kBar + idx * kSpread / G::kCopies; };   // >= kM: in the next stage
    // copies issued in the stage itself
    constexpr int kNow = kM - kBar >= kSpread ? G::kCopies : ((kM - kBar) * G::kCopies + kSpread - 1) / kSpread;
    static_assert(copy_at(kNow - 1) < kM && (kNow == G::kCopies || copy_at(kNow) >= kM) &&
                      copy_at(G::kCopies - 1) - kM < kBar,
                  "all copies of a stage are out before the next barrier");
    v8i fa[Y_], fw[kBufs];
    v4f P[4];
    float sv[Y_], fy[Y_], sw_lo, sw_hi;                    // token scales, factors, weight scales (SWIGLU: gate, up)
    auto read_a = [&](int slot, int y) {
        fa[y] = frag(&lds[slot * G::kSlot] + (wm * G::kStrip + y * 16) * kBK, foa);
    };
    auto read_w = [&](int slot, int x) {
        fw[x % kBufs] = frag(&lds[slot * G::kSlot] + G::kA + (wtile_row0<EPI>(wn, x >> 1) + (x & 1) * 16) * kBK, fow);
    };
    auto read_s = [&](int slot) {
        const float *ls = reinterpret_cast<const float *>(&lds[slot * G::kSlot] + G::kA + G::kW + wave * 256);
#pragma unroll
        for (int y = 0; y < Y_; ++y) sv[y] = ls[y * 16 + r16];
        sw_lo = ls[G::kScales / 4];
        sw_hi = SW ? ls[G::kScales / 4 + 2] : 0.0f;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) P[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};   // before stage 0: nothing to add
#pragma unroll
    for (int y = 0; y < Y_; ++y) fy[y] = 0.0f;
    if (nk > 0) {
#pragma unroll
        for (int i = 0; i < G::kDepth; ++i) {
            const StageCopy c = plan(i);
#pragma unroll
            for (int idx = 0; idx < G::kCopies; ++idx)
                if (i < G::kDepth - 1 || idx < kNow) issue_one(c, i, idx);
        }
        wait_vmem<(G::kDepth - 2) * G::kCopies + kNow>();
        wait_lds();
        block_barrier();
#pragma unroll
        for (int x = 0; x < G::kAhead; ++x) read_w(0, x);
#pragma unroll
        for (int y = 0; y < Y_; ++y) read_a(0, y);
        read_s(0);
    }
    auto add = [&](int m) {                                // MFMA m's product into its accumulators
        v4f &c = acc4[m / Y_][m % Y_];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = __builtin_fmaf(P[m & 3][e], fy[m % Y_], c[e]);
        asm volatile("" : "+v"(c));
    };
    // a strip past the tile's last row only copies and waits with the others:
    // a tile of at most BM / 2 rows has one wave per SIMD at work
    const bool busy = wm * G::kStrip < (int)a_rows;
    int slot = 0, prev = G::kDepth - 1;
    StageCopy old = plan(G::kDepth - 1);                   // whose last copies, into slot prev, are not out yet
    for (int kt = 0; kt < (busy ? nk : 0); ++kt) {
        const int next = slot + 1 == G::kDepth ? 0 : slot + 1;
        const StageCopy c = plan(kt + G::kDepth);
#pragma unroll
        for (int m = 0; m < kM; ++m) {
            const int X = m / Y_, Y = m % Y_;
            if (m == kBar) {
                wait_lds();
                wait_vmem<(G::kDepth - 2) * G::kCopies>();
                block_barrier();
            }
            P[m & 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[X % kBufs], fa[Y], v4f{0.0f, 0.0f, 0.0f, 0.0f},
                                                                        0, 0, 0, 0, 0, 0);
            asm volatile("" : "+v"(P[m & 3]));
            __builtin_amdgcn_sched_barrier(0);
            if (Y == 0 && X + G::kAhead < 8) read_w(slot, X + G::kAhead);
            if (Y == 0 && X + G::kAhead >= 8) read_w(next, X + G::kAhead - 8);
            if (X == 7) read_a(next, Y);
#pragma unroll
            for (int idx = 0; idx < G::kCopies; ++idx)
                if (copy_at(idx) == m) issue_one(c, slot, idx);
                else if (copy_at(idx) - kM == m) issue_one(old, prev, idx);
            add((m + kM - 3) % kM);                        // MFMA m - 3
            // the factors change once the last product that takes the old
            // ones is added: here for the weight rows' first half and, gate
            // and up rows having their own, for the second
            if (m == 2 || (SW && m == 4 * Y_ + 2)) {
#pragma unroll
                for (int y = 0; y < Y_; ++y) fy[y] = sv[y] * (m == 2 ? sw_lo : sw_hi);
            }
            if (m == kM - 1) read_s(next);
            __builtin_amdgcn_sched_barrier(0);
        }
        prev = slot;
        slot = next;
        old = c;
    }
    if (nk > 0 && busy) {
        add(kM - 3);
        add(kM - 2);
        add(kM - 1);
    }
    if (nk > 0 && !busy)
#pragma unroll
        for (int idx = kNow; idx < G::kCopies; ++idx) issue_one(old, prev, idx);
    for (int kt = 0; kt < (busy ? 0 : nk); ++kt) {
        const StageCopy c = plan(kt + G::kDepth);
        wait_vmem<(G::kDepth - 2) * G::kCopies>();
        block_barrier();
#pragma unroll
        for (int idx = 0; idx < G::kCopies; ++idx) issue_one(c, slot, idx);
        slot = slot + 1 == G::kDepth ? 0 : slot + 1;
    }
    wait_vmem<0>();
    wait_lds();
    block_barrier();                                        // the slots become the epilogue's

    // Lane l of a 16 x 16 result holds token l % 16 and weight rows 4 (l / 16)
    // + e as taken; exchanging the odd 16-lane rows of token block 2 y with
    // the even rows of block 2 y + 1 leaves, with the rows' swapped bits, lane
    // l with token l % 32 and rows 8 q + 4 (l / 32) + e: the 32 x 32 layout.
    Acc acc;
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < Y_ / 2; ++y)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const auto t = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc4[2 * x + h][2 * y][e]),
                                                                    __float_as_uint(acc4[2 * x + h][2 * y + 1][e]), false, false);
                    acc[x][y][8 * h + e] = __uint_as_float(t[0]);
                    acc[x][y][8 * h + 4 + e] = __uint_as_float(t[1]);
                }

    if constexpr (SPLIT) {
        // partial tile: float4 q of block 4 y + x of thread i at
        // ((y * 4 + x) * 4 + q) * threads * 4 + 4 i, whole lines per store
        float *base = g.partials + ((T.global * g.split_k + split) * (int64_t)(BM * 256)) + tid * 4;
#pragma unroll
        for (int y = 0; y < Y_ / 2; ++y) {
            if (T.m0 + wm * G::kStrip + y * 32 + (ln & 31) >= g.M) continue;
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<v4f *>(base + ((y * 4 + x) * 4 + q) * (G::kThreads * 4)) =
                        v4f{acc[x][y][4 * q], acc[x][y][4 * q + 1], acc[x][y][4 * q + 2], acc[x][y][4 * q + 3]};
        }
    } else {
        GemmArgs ge = g;
        ge.M = m_end;
        if (EXPERTS) ge.stride_o = 0;
        epilogue<EPI, Y_ / 2, true, true, SO, true>(ge, T, acc, nullptr, nullptr,
                                                    reinterpret_cast<float *>(&lds[G::kBias]), &lds[wave * G::kRegion], wave);
    }
}

template <int EPI, int BM, bool EXPERTS, bool SPLIT, bool SO>
__global__ __launch_bounds__(Geometry<BM>::kThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) void gemm_block_kernel(
    const BlockArgs a)
{
    constexpr bool SW = EPI == SPG_EPI_SWIGLU;
    // an expert's last tile of at most 128 rows runs as a 128-row tile, whose
    // rows spread over all eight waves and whose copies have three slots (64
    // experts of 2048 x 2048, us: 256 rows 121 as 256-row tiles, 109 so; 512 rows
    // 176 and 168; 128 rows, where most tiles are whole 128-row ones, 70 and 72)
    constexpr bool LIGHT = EXPERTS && BM == 256;
    constexpr int kLds = LIGHT && Geometry<128>::kLds > Geometry<BM>::kLds ? Geometry<128>::kLds : Geometry<BM>::kLds;
    __shared__ __attribute__((aligned(2048))) uint8_t lds[kLds];
    const GemmArgs &g = a.g;
    clock_mark(g.clocks, 0);

    // ---- the tile -----------------------------------------------------------
    Tile T;
    int64_t m_end = g.M;
    int split = 0;
    if (EXPERTS) {
        const ExpertTile t = expert_tile<BM>(a);
        if (t.expert < 0) return;
        T.global = t.id;
        T.b = t.expert;
        T.m0 = t.m0;
        T.tn = t.column;
        T.n0 = T.tn * (SW ? 128 : 256);
        T.c0 = T.n0;
        m_end = t.end;
    } else {
        if (BM == 128 && !SPLIT && !g.rows128) {
            // the tail of a product in 256-row tiles: half v % 2 of tile
            // tile_begin + v / 2 (neighbouring halves share their W panel)
            const uint32_t v = (uint32_t)xcd_remap(blockIdx.x, 2 * g.tile_count);
            T = tile_from_id<EPI, 256>(g, g.tile_begin + (v >> 1));
            T.m0 += (int64_t)(v & 1u) * 128;
            if (T.m0 >= g.M) return;
        } else {
            const WorkItem wi = work_item(g);
            split = wi.split;
            T = tile_from_id<EPI, BM>(g, g.tile_begin + wi.tile);
        }
    }
    if (LIGHT && m_end - T.m0 <= 128)
        block_tile<EPI, 128, EXPERTS, SPLIT, SO>(a, T, m_end, split, lds);
    else
        block_tile<EPI, BM, EXPERTS, SPLIT, SO>(a, T, m_end, split, lds);
    clock_mark(g.clocks, 1);
}

// Sums the K slices' partial tiles and applies the epilogue: one workgroup
// per (tile, block x, block y) of every wave (SWIGLU: a gate block and its up
// block), each thread the 16 accumulators that it held in the product.
template <int EPI, int BM>
__global__ __launch_bounds__(Geometry<BM>::kThreads) void gemm_block_reduce_kernel(const BlockArgs a)
{
    using G = Geometry<BM>;
    constexpr bool SW = EPI == SPG_EPI_SWIGLU;
    constexpr int kYB = G::kY / 2;
    __shared__ __attribute__((aligned(16))) float lds_one[256];
    const GemmArgs &g = a.g;
    const int tid = threadIdx.x;
    if (tid < 256) lds_one[tid] = 1.0f;
    __syncthreads();
    const Tile T = tile_from_id<EPI, BM>(g, blockIdx.x);
    const int x = (int)blockIdx.y / kYB, y = (int)blockIdx.y % kYB;
    const int wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
    if (T.m0 + wm * G::kStrip + y * 32 + (tid & 31) >= g.M) return;
    const float *base = g.partials + (int64_t)blockIdx.x * g.split_k * (BM * 256) + tid * 4;
    v16f sum = {}, up = {};
    for (int s = 0; s < g.split_k; ++s) {
        const float *p = base + (int64_t)s * (BM * 256);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const v4f v = __builtin_nontemporal_load(
                reinterpret_cast<const v4f *>(p + ((y * 4 + x) * 4 + q) * (G::kThreads * 4)));
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[4 * q + j] += v[j];
            if (SW) {
                const v4f u = __builtin_nontemporal_load(
                    reinterpret_cast<const v4f *>(p + ((y * 4 + x + 2) * 4 + q) * (G::kThreads * 4)));
#pragma unroll
                for (int j = 0; j < 4; ++j) up[4 * q + j] += u[j];
            }
        }
    }
    // epilogue_block places 32-row block y of strip wm at row 128 wm + 32 y
    // of the tile; strips here are kStrip rows
    epilogue_block<EPI>(g, T, epi_out<EPI>(g, T), wtile_row0<EPI>(wn, x), y - wm * (128 - G::kStrip) / 32, sum, up,
                        lds_one, lds_one);
}

template <int EPI, int BM>
hipError_t launch_geometry(const BlockArgs &a, int64_t workgroups, hipStream_t s)
{
    const dim3 grid((unsigned)workgroups), threads(Geometry<BM>::kThreads);
    if (a.experts > 0) {
        if constexpr (EPI != SPG_EPI_ADD)
            gemm_block_kernel<EPI, BM, true, false, false><<<grid, threads, 0, s>>>(a);
        else
            return hipErrorInvalidValue;
    } else if (a.g.split_k > 1) {
        gemm_block_kernel<EPI, BM, false, true, false><<<grid, threads, 0, s>>>(a);
    } else if (a.g.nseg != 0) {
        gemm_block_kernel<EPI, BM, false, false, true><<<grid, threads, 0, s>>>(a);
    } else {
        gemm_block_kernel<EPI, BM, false, false, false><<<grid, threads, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <int EPI>
hipError_t launch_epi(const BlockArgs &a, int bm, int64_t workgroups, hipStream_t s)
{
    return bm == 256 ? launch_geometry<EPI, 256>(a, workgroups, s) : launch_geometry<EPI, 128>(a, workgroups, s);
}

template <int EPI, int BM>
hipError_t launch_reduce(const BlockArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)a.g.tile_count, (EPI == SPG_EPI_SWIGLU ? 2u : 4u) * (Geometry<BM>::kY / 2));
    gemm_block_reduce_kernel<EPI, BM><<<grid, Geometry<BM>::kThreads, 0, s>>>(a);
    return hipGetLastError();
}

template <int EPI>
hipError_t launch_reduce_epi(const BlockArgs &a, int bm, hipStream_t s)
{
    return bm == 256 ? launch_reduce<EPI, 256>(a, s) : launch_reduce<EPI, 128>(a, s);
}

}  // namespace

hipError_t launch_gemm_block_tiles(const BlockArgs &a, int bm, int64_t workgroups, hipStream_t s)
{
    switch (a.g.epilogue) {
    case SPG_EPI_STORE: return launch_epi<SPG_EPI_STORE>(a, bm, workgroups, s);
    case SPG_EPI_ADD: return launch_epi<SPG_EPI_ADD>(a, bm, workgroups, s);
    default: return launch_epi<SPG_EPI_SWIGLU>(a, bm, workgroups, s);
    }
}

hipError_t launch_gemm_block_reduce(const BlockArgs &a, int bm, hipStream_t s)
{
    switch (a.g.epilogue) {
    case SPG_EPI_STORE: return launch_reduce_epi<SPG_EPI_STORE>(a, bm, s);
    case SPG_EPI_ADD: return launch_reduce_epi<SPG_EPI_ADD>(a, bm, s);
    default: return launch_reduce_epi<SPG_EPI_SWIGLU>(a, bm, s);
    }
}

}  // namespace spg
