// Block-scaled FP8 product over tiles, dense and per expert (see
// spg_gemm_block_common.h for the arithmetic).
//
// Design for CDNA4:
//  * Tiles of BM x 256 (BM = 256 or 128 token rows, 256 weight rows), waves
//    2 (weight halves) x BM / 64 (token strips): each wave holds 64 tokens x
//    128 weight rows = 2 x 4 blocks of v_mfma_f32_32x32x64_f8f6f4, 128
//    accumulators per lane.  With BM = 256 that is two waves per SIMD, so one
//    wave's multiply-adds (acc += P s) run under the other's MFMAs; the 128 x
//    128 wave tiles of the row-scaled kernel would need 256 accumulators in
//    vector registers (the vector unit cannot add into accumulation
//    registers), which leaves no room for P.
//  * W fragments are the first MFMA operand, so a lane holds one token's
//    column of a block: its factor sa[token] sw[block] is one register per
//    block, the same for all 16 of its accumulators.
//  * K advances one group (128 bytes) per stage.  Codes and scales go
//    straight into LDS (buffer loads to LDS), DEPTH slots, one barrier per
//    stage: behind it stage s has landed for all waves and every wave is done
//    with stage s - 1, whose slot takes the copies of stage s + DEPTH - 1.
//  * Experts' products: a workgroup finds its (expert, rows) tile from the
//    offsets in device memory, and gathers A rows by index with per-lane copy
//    addresses; the grid is the largest that the row count allows, and
//    workgroups past the last tile end at once.
#include "spg_gemm_block_common.h"

namespace spg {

namespace {

using namespace block;

constexpr int kBK = 128;

template <int WM>
struct Geometry {
    static constexpr int kRows = 64 * WM;                   // token rows of a tile
    static constexpr int kWaves = 2 * WM;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr int kA = kRows * kBK;                  // code bytes of a slot: A
    static constexpr int kW = 256 * kBK;                    // and W
    static constexpr int kSa = kRows * 4;                   // token scales
    static constexpr int kSw = kWaves * 256;                // one 256-byte row of weight scales per wave
    static constexpr int kSlot = kA + kW + kSa + kSw;
    static constexpr int kDepth = WM == 4 ? 2 : 3;
    static constexpr int kCopyA = kRows / kWaves / 8;       // copy instructions of a wave per stage: A
    static constexpr int kCopyW = 256 / kWaves / 8;         // and W
    static constexpr int kCopies = kCopyA + kCopyW + 2;     // and the two scale copies
    static_assert(kSlot % 256 == 0, "a slot starts on LDS bank 0");
};

template <int EPI, int WM, bool EXPERTS, bool SPLIT, bool SO>
__global__ __launch_bounds__(Geometry<WM>::kThreads) void gemm_block_kernel(const BlockArgs a)
{
    using G = Geometry<WM>;
    constexpr int BM = G::kRows;
    constexpr bool SW = EPI == SPG_EPI_SWIGLU;
    __shared__ __attribute__((aligned(2048))) uint8_t lds[G::kDepth * G::kSlot];
    __shared__ __attribute__((aligned(16))) float lds_one[256];
    __shared__ __attribute__((aligned(16))) float lds_bias[EPI == SPG_EPI_ADD ? G::kWaves * 128 : 4];
    const GemmArgs &g = a.g;
    clock_mark(g.clocks, 0);

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int ln = lane_id();

    // ---- the tile -----------------------------------------------------------
    Tile T;
    int64_t m_end = g.M;
    int split = 0;
    if (EXPERTS) {
        const int32_t mt = total_tiles<BM>(a);
        const int64_t n = (int64_t)mt * g.tiles_n;
        if ((int64_t)blockIdx.x >= n) return;
        const uint32_t v = (uint32_t)xcd_remap(blockIdx.x, n);
        const uint32_t m = fdiv(v, g.div_per);            // div_per: by tiles_n
        const ExpertTile t = find_tile<BM>(a, (int32_t)m);
        if (t.expert < 0) return;
        T.global = v;
        T.b = t.expert;
        T.m0 = t.m0;
        T.tn = v - m * (uint32_t)g.tiles_n;
        T.n0 = T.tn * (SW ? 128 : 256);
        T.c0 = T.n0;
        m_end = t.end;
    } else {
        const WorkItem wi = work_item(g);
        split = wi.split;
        T = tile_from_id<EPI, BM>(g, wi.tile);
    }
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
    // scales: lane l the token scale of row 64 wm + l (both waves of a strip
    // copy it: the same values to the same place), lanes 0 .. 3 the weight
    // scales of the wave's four 32-row blocks
    const float *sa = (const float *)g.sa + ((!EXPERTS && g.stride_a) ? T.b * g.sa_bstride : 0);
    const float *sw = (const float *)g.sw + (g.stride_w ? T.b * g.sw_bstride : 0);
    uint32_t vsa, vsw = kOOB;
    {
        const uint32_t r = (uint32_t)(wm * 64 + ln);
        uint32_t src = r;
        bool ok = (int64_t)r < a_rows;
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
    // stage kt (0 .. nk - 1; others copy zeros, so that every wait counts the
    // same) into slot `slot`
    auto issue = [&](int kt, int slot) {
        const bool live = kt < nk;
        const int64_t k0 = live ? (int64_t)(k0g + kt) * kBK : 0;
        const bool in_e = live && k0 + (int64_t)c_even * 16 < g.K;
        const bool in_o = live && k0 + (int64_t)c_odd * 16 < g.K;
        const uint32_t soff = (uint32_t)k0;
        const uint32_t base = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds_base + (uint32_t)(slot * G::kSlot)));
#pragma unroll
        for (int i = 0; i < G::kCopyA; ++i)
            dma16(base + (uint32_t)((wave * 8 * G::kCopyA + 8 * i) * kBK), ((i & 1) ? in_o : in_e) ? va[i] : kOOB, rs_a, soff);
#pragma unroll
        for (int i = 0; i < G::kCopyW; ++i)
            dma16(base + (uint32_t)(G::kA + (wave * kWRows + 8 * i) * kBK),
                  ((i & 1) ? in_o : in_e) ? vw[i & 1] + (uint32_t)(8 * i) * (uint32_t)g.ldw : kOOB, rs_w, soff);
        const int64_t kg = live ? k0g + kt : 0;
        dma4(base + (uint32_t)(G::kA + G::kW + wm * 256), live ? vsa : kOOB,
             make_rsrc(sa_tile + kg * a.a_rows, sa_bytes), 0);
        dma4(base + (uint32_t)(G::kA + G::kW + G::kSa + wave * 256), live ? vsw : kOOB, rs_sw,
             (uint32_t)kg * (uint32_t)a.sw_gs * 4u);
    };

    // ---- fragments ------------------------------------------------------------
    const uint32_t l32 = (uint32_t)ln & 31, khalf = (uint32_t)ln >> 5, fx = (l32 >> 1) & 7u;
    uint32_t foff[2][2];
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            foff[ks][h] = l32 * kBK + ((((uint32_t)ks * 4 + khalf * 2 + (uint32_t)h) ^ fx) << 4);
    auto frag = [&](const uint8_t *rows, int ks) -> v8i {
        const uint4 lo = *reinterpret_cast<const uint4 *>(rows + foff[ks][0]);
        const uint4 hi = *reinterpret_cast<const uint4 *>(rows + foff[ks][1]);
        return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };

    Acc acc;                                               // blocks acc[x][0..1]
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[x][y][e] = 0.0f;

    auto compute = [&](int slot) {
        const uint8_t *la = &lds[slot * G::kSlot + wm * 64 * kBK];
        const uint8_t *lw = &lds[slot * G::kSlot + G::kA];
        const float *ls = reinterpret_cast<const float *>(&lds[slot * G::kSlot + G::kA + G::kW]);
        v8i fa[2][2];
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) fa[y][ks] = frag(la + y * 32 * kBK, ks);
        const float s0 = ls[wm * 64 + l32], s1 = ls[wm * 64 + 32 + l32];
        const v4f swv = *reinterpret_cast<const v4f *>(ls + G::kRows + wave * 64);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint8_t *rows = lw + wtile_row0<EPI>(wn, x) * kBK;
            const v8i f0 = frag(rows, 0), f1 = frag(rows, 1);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                v16f p = {};
                p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f0, fa[y][0], p, 0, 0, 0, 0, 0, 0);
                p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f1, fa[y][1], p, 0, 0, 0, 0, 0, 0);
                const float f = (y ? s1 : s0) * swv[x];
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[x][y][e] = __builtin_fmaf(p[e], f, acc[x][y][e]);
            }
        }
    };

    if (tid < 256) lds_one[tid] = 1.0f;
    if (G::kThreads < 256)
        for (int i = tid + G::kThreads; i < 256; i += G::kThreads) lds_one[i] = 1.0f;
#pragma unroll
    for (int i = 0; i < G::kDepth - 1; ++i) issue(i, i);
    int slot = 0;
    for (int kt = 0; kt < nk; ++kt) {
        wait_vmem<(G::kDepth - 2) * G::kCopies>();         // stage kt landed (this wave's copies)
        wait_lds();
        block_barrier();                                    // ... and all waves'; stage kt - 1 is done with
        const int free_slot = slot == 0 ? G::kDepth - 1 : slot - 1;
        issue(kt + G::kDepth - 1, free_slot);
        compute(slot);
        slot = slot + 1 == G::kDepth ? 0 : slot + 1;
    }
    wait_vmem<0>();
    wait_lds();
    block_barrier();                                        // the slots become the epilogue's staging regions

    if constexpr (SPLIT) {
        // partial tile: float4 q of block 4 y' + x of thread i at
        // ((y' * 4 + x) * 4 + q) * threads * 4 + 4 i, whole lines per store
        float *base = g.partials + ((T.global * g.split_k + split) * (int64_t)(BM * 256)) + tid * 4;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            if (T.m0 + wm * 64 + y * 32 + l32 >= g.M) continue;
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
        epilogue<EPI, 2, true, true, SO>(ge, T, acc, lds_one, lds_one, lds_bias, &lds[wave * 16384], wave);
    }
    clock_mark(g.clocks, 1);
}

// Sums the K slices' partial tiles and applies the epilogue: one workgroup
// per (tile, block x, block y) of every wave (SWIGLU: a gate block and its up
// block), each thread the 16 accumulators that it held in the product.
template <int EPI, int WM>
__global__ __launch_bounds__(Geometry<WM>::kThreads) void gemm_block_reduce_kernel(const BlockArgs a)
{
    using G = Geometry<WM>;
    constexpr bool SW = EPI == SPG_EPI_SWIGLU;
    __shared__ __attribute__((aligned(16))) float lds_one[256];
    const GemmArgs &g = a.g;
    const int tid = threadIdx.x;
    for (int i = tid; i < 256; i += G::kThreads) lds_one[i] = 1.0f;
    __syncthreads();
    const Tile T = tile_from_id<EPI, G::kRows>(g, blockIdx.x);
    const int x = (int)blockIdx.y >> 1, y = (int)blockIdx.y & 1;
    const int wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
    if (T.m0 + wm * 64 + y * 32 + (tid & 31) >= g.M) return;
    const float *base = g.partials + (int64_t)blockIdx.x * g.split_k * (G::kRows * 256) + tid * 4;
    v16f sum = {}, up = {};
    for (int s = 0; s < g.split_k; ++s) {
        const float *p = base + (int64_t)s * (G::kRows * 256);
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
    // epilogue_block places wave strip wm at 128 wm + 32 y: shift y by -2 wm
    // for strips of 64 rows.  Its own wm is the same thread index >> 7.
    epilogue_block<EPI>(g, T, epi_out<EPI>(g, T), wtile_row0<EPI>(wn, x), y - 2 * wm, sum, up, lds_one, lds_one);
}

template <int EPI, int WM>
hipError_t launch_geometry(const BlockArgs &a, int64_t workgroups, hipStream_t s)
{
    const dim3 grid((unsigned)workgroups), threads(Geometry<WM>::kThreads);
    if (a.experts > 0) {
        if constexpr (EPI != SPG_EPI_ADD)
            gemm_block_kernel<EPI, WM, true, false, false><<<grid, threads, 0, s>>>(a);
        else
            return hipErrorInvalidValue;
    } else if (a.g.split_k > 1) {
        gemm_block_kernel<EPI, WM, false, true, false><<<grid, threads, 0, s>>>(a);
    } else if (a.g.nseg != 0) {
        gemm_block_kernel<EPI, WM, false, false, true><<<grid, threads, 0, s>>>(a);
    } else {
        gemm_block_kernel<EPI, WM, false, false, false><<<grid, threads, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <int EPI>
hipError_t launch_epi(const BlockArgs &a, int bm, int64_t workgroups, hipStream_t s)
{
    return bm == 256 ? launch_geometry<EPI, 4>(a, workgroups, s) : launch_geometry<EPI, 2>(a, workgroups, s);
}

template <int EPI>
hipError_t launch_reduce(const BlockArgs &a, int bm, hipStream_t s)
{
    const dim3 grid((unsigned)a.g.tile_count, EPI == SPG_EPI_SWIGLU ? 4u : 8u);
    if (bm == 256)
        gemm_block_reduce_kernel<EPI, 4><<<grid, Geometry<4>::kThreads, 0, s>>>(a);
    else
        gemm_block_reduce_kernel<EPI, 2><<<grid, Geometry<2>::kThreads, 0, s>>>(a);
    return hipGetLastError();
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
    case SPG_EPI_STORE: return launch_reduce<SPG_EPI_STORE>(a, bm, s);
    case SPG_EPI_ADD: return launch_reduce<SPG_EPI_ADD>(a, bm, s);
    default: return launch_reduce<SPG_EPI_SWIGLU>(a, bm, s);
    }
}

}  // namespace spg
