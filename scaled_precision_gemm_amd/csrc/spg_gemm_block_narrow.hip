// Block-scaled FP8 product for few rows per tile: dense products of at most
// 32 tokens and experts with a handful of rows each.
//
// Such a product is a stream over the weights, so the kernel is shaped like
// the decode-width kernel of the other formats (spg_gemm_narrow.hip): one
// workgroup per 16- or 32-row tile and 32 output columns (SWIGLU: 16), its
// four waves take contiguous quarters of K, each through a private LDS ring
// of direct copies, and the quarters are summed through LDS in a fixed order.
// A ring chunk is 128 K-elements of every row - one scale group - so each
// v_mfma_f32_16x16x128_f8f6f4 yields one group's partial product, which joins
// the accumulator times sa sw (sa: one token per lane; sw: one per weight
// block).
//
// Bound by the weight stream: 16 x 8192 x 8192 14.4 us (4.7 TB/s), 16 x 5120 x
// 17408 ADD 23 us with weights from HBM (3.9 TB/s; 160 workgroups, row-scaled
// 21.6), 128 rows over 64 experts of 2048 x 2048 43 us (5.5 TB/s).  16
// columns a workgroup where 32 leave compute units idle took longer (16 x 5120
// x 17408 29.8 us for 24.5: A is copied twice as often), and so did rings of
// 32 KiB a wave (16 x 8192 x 8192 20.6 us for 14.3).
#include "spg_gemm_block_common.h"

namespace spg {

namespace {

using namespace block;

constexpr int kWaves = 4;
constexpr int kNarrowThreads = 64 * kWaves;
constexpr int kChunk = 128;
constexpr int kWaveLds = 16384;       // ring bytes per wave (as the decode-width kernel)

template <int EPI, int TB, int RB, bool EXPERTS>
__global__ __launch_bounds__(kNarrowThreads) void gemm_block_narrow_kernel(const BlockArgs a)
{
    constexpr bool SW = EPI == SPG_EPI_SWIGLU;
    constexpr int NB = (SW ? 2 : 1) * RB;                // 16-row weight blocks
    constexpr int kCols = 16 * RB;
    constexpr int ROWS = 16 * (NB + TB);
    constexpr int SLOT = ROWS * kChunk + 512;            // codes, token scales, weight scales
    constexpr int DEPTH = kWaveLds / SLOT < 2 ? 2 : kWaveLds / SLOT;
    constexpr int IPC = 2 * (NB + TB) + 2;               // copy instructions per chunk
    static_assert((DEPTH - 1) * IPC <= 63, "vmcnt range");
    constexpr int kRingBytes = kWaves * DEPTH * SLOT;
    static_assert(kWaves * NB * TB * 64 * 16 <= kRingBytes, "the partial sums fit in the ring");
    __shared__ __attribute__((aligned(2048))) uint8_t lds[kRingBytes];
    auto ring = reinterpret_cast<uint8_t (*)[DEPTH][SLOT]>(lds);
    auto red = reinterpret_cast<float (*)[NB * TB][64 * 4]>(lds);

    const GemmArgs &g = a.g;
    clock_mark(g.clocks, 0);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t nout = SW ? g.N / 2 : g.N;
    const int r = lane & 15, kq = lane >> 4;

    // ---- the tile: token rows m0 .. m_end - 1 (at most 16 TB), columns j0 ..
    int64_t b, m0 = 0, m_end = g.M, j0;
    if (EXPERTS) {
        const ExpertTile t = expert_tile<16 * TB>(a);
        if (t.expert < 0) return;
        b = t.expert;
        m0 = t.m0;
        m_end = t.end;
        j0 = (int64_t)t.column * kCols;
    } else {
        b = (int64_t)blockIdx.x / g.tiles_n;
        j0 = ((int64_t)blockIdx.x - b * g.tiles_n) * kCols;
    }
    const int64_t a_rows = min((int64_t)(16 * TB), m_end - m0);

    const int nch = a.groups, per = (nch + kWaves - 1) / kWaves;
    const int c_begin = min(nch, wave * per), c_end = min(nch, c_begin + per);

    // ---- copies: lane L fetches row 8 i + L / 8 of a 16-row block (i = 0, 1),
    // 16-byte piece gj[i], landing at LDS piece L % 8
    const int crow = lane >> 3, cj = lane & 7;
    uint32_t gj[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) gj[i] = (uint32_t)(cj ^ ((4 * i + (crow >> 1)) & 7));

    const int64_t cols = min((int64_t)kCols, nout - j0);
    auto wrow0 = [&](int nb) -> int64_t { return (nb >= RB ? g.N / 2 : 0) + j0 + 16 * (nb % RB); };
    auto brows = [&](int nb) -> int64_t { return max((int64_t)0, min((int64_t)16, cols - 16 * (nb % RB))); };
    const uint8_t *wbase = g.W + (g.stride_w ? b * g.stride_w : 0);
    v4i rw[NB];
    uint32_t woff[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        rw[nb] = make_rsrc(wbase + wrow0(nb) * g.ldw, (uint32_t)(brows(nb) * g.ldw));
#pragma unroll
        for (int i = 0; i < 2; ++i)
            woff[nb][i] = 8 * i + crow < brows(nb) ? (uint32_t)(8 * i + crow) * (uint32_t)g.ldw + 16 * gj[i] : kOOB;
    }
    const bool gather = EXPERTS && a.row_index != nullptr;
    const uint8_t *abase = g.A + ((!EXPERTS && g.stride_a) ? b * g.stride_a : 0);
    const v4i ra = gather ? make_rsrc(abase, (uint32_t)(a.a_rows * g.lda))
                          : make_rsrc(abase + m0 * g.lda, (uint32_t)(a_rows * g.lda));
    auto source = [&](int row, bool &ok) -> uint32_t {   // A row of tile row `row`
        ok = row < a_rows;
        if (!gather) return (uint32_t)row;
        const int32_t x = ok ? a.row_index[m0 + row] : -1;
        ok = x >= 0 && (int64_t)x < a.a_rows;
        return (uint32_t)x;
    };
    uint32_t aoff[TB][2];
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bool ok;
            const uint32_t src = source(16 * t + 8 * i + crow, ok);
            aoff[t][i] = ok ? src * (uint32_t)g.lda + 16 * gj[i] : kOOB;
        }
    // scales of a chunk: lane l the token scale of tile row l, lane nb the
    // weight scale of block nb
    const float *sa = (const float *)g.sa + b * g.sa_bstride + (gather ? 0 : m0);
    const uint32_t sa_bytes = (uint32_t)((gather ? a.a_rows : a_rows) * 4);
    const v4i rsw = make_rsrc((const float *)g.sw + b * g.sw_bstride, (uint32_t)a.sw_words * 4u);
    uint32_t vsa, vsw = kOOB;
    {
        bool ok;
        const uint32_t src = source(lane, ok);
        vsa = ok ? src * 4u : kOOB;
        const int64_t row = wrow0(lane < NB ? lane : 0);
        if (lane < NB && brows(lane) > 0) vsw = (uint32_t)(row >> 7) * (uint32_t)a.sw_rs * 4u;
    }

    auto slot_addr = [&](int s) -> uint32_t {
        return (uint32_t)__builtin_amdgcn_readfirstlane(
            (int)(uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)&ring[wave][s][0]);
    };
    // copies of chunk c into slot s (chunks past the wave's range and pieces
    // past K read as zero: no memory traffic)
    auto issue = [&](int s, int c) {
        const uint32_t base = slot_addr(s);
        const bool live = c < c_end;
        const uint32_t soff = live ? (uint32_t)c * kChunk : 0u;
        const bool kin = live && (int64_t)c * kChunk + 16 * gj[0] < g.K;
        const bool kin1 = live && (int64_t)c * kChunk + 16 * gj[1] < g.K;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            dma16(base + (uint32_t)(nb * 16) * kChunk, kin ? woff[nb][0] : kOOB, rw[nb], soff);
            dma16(base + (uint32_t)(nb * 16 + 8) * kChunk, kin1 ? woff[nb][1] : kOOB, rw[nb], soff);
        }
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            dma16(base + (uint32_t)((NB + t) * 16) * kChunk, kin ? aoff[t][0] : kOOB, ra, soff);
            dma16(base + (uint32_t)((NB + t) * 16 + 8) * kChunk, kin1 ? aoff[t][1] : kOOB, ra, soff);
        }
        const int64_t cg = live ? c : 0;
        dma4(base + ROWS * kChunk, live ? vsa : kOOB, make_rsrc(sa + cg * a.a_rows, sa_bytes), 0);
        dma4(base + ROWS * kChunk + 256, live ? vsw : kOOB, rsw, (uint32_t)cg * (uint32_t)a.sw_gs * 4u);
    };

    // chunks of a lane's 32 bytes chosen against bank conflicts (see
    // spg_gemm_block.hip)
    const uint32_t fsw = (uint32_t)((r >> 1) & 7), q0 = (uint32_t)((kq & 1) | ((kq & 2) << 1));
    const uint32_t fo0 = (uint32_t)r * kChunk + ((q0 ^ fsw) << 4), fo1 = fo0 ^ 32u;
    auto frag = [&](const uint8_t *rows) -> v8i {
        const uint4 lo = *reinterpret_cast<const uint4 *>(rows + fo0);
        const uint4 hi = *reinterpret_cast<const uint4 *>(rows + fo1);
        return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };

    v4f acc[NB][TB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int t = 0; t < TB; ++t) acc[nb][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    // chunk c_begin + i sits in slot i % DEPTH; a slot is read when at most
    // the later chunks' copies are outstanding, and refilled once its reads
    // have completed
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) issue(i, c_begin + i);
    for (int c = c_begin; c < c_end; c += DEPTH) {
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            wait_vmem<(DEPTH - 1) * IPC>();
            const uint8_t *sl = &ring[wave][i][0];
            const float *ss = reinterpret_cast<const float *>(sl + ROWS * kChunk);
            v8i w[NB], x[TB];
            float fs[TB], fw[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) w[nb] = frag(sl + nb * 16 * kChunk);
#pragma unroll
            for (int t = 0; t < TB; ++t) x[t] = frag(sl + (NB + t) * 16 * kChunk);
#pragma unroll
            for (int t = 0; t < TB; ++t) fs[t] = ss[t * 16 + r];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) fw[nb] = ss[64 + nb];
            wait_lds();
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    const v4f p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        w[nb], x[t], v4f{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
                    const float f = fs[t] * fw[nb];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[nb][t][e] = __builtin_fmaf(p[e], f, acc[nb][t][e]);
                }
            issue(i, c + DEPTH + i);
        }
    }
    wait_vmem<0>();

    // ---- the four K quarters, summed in a fixed order
    __syncthreads();
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int t = 0; t < TB; ++t) *reinterpret_cast<v4f *>(&red[wave][nb * TB + t][lane * 4]) = acc[nb][t];
    __syncthreads();
    if (tid >= 64 * TB * RB) return;
    const int q = tid >> 6, t = q % TB, rb = q / TB;
    constexpr int NH = SW ? 2 : 1;
    v4f v[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
        const int slot = (h * RB + rb) * TB + t;
        v[h] = *reinterpret_cast<const v4f *>(&red[0][slot][lane * 4]);
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v[h] += *reinterpret_cast<const v4f *>(&red[w][slot][lane * 4]);
    }

    // ---- epilogue: lane l, register e hold output column 4 (l / 16) + e of
    // the block and token l % 16 of token block t
    const int64_t m = m0 + t * 16 + (lane & 15);
    const int64_t col = j0 + 16 * rb + (lane >> 4) * 4;
    if (m < m_end && m < m0 + a_rows && col < nout) {
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = SW ? swiglu_f32(v[0][e], v[NH - 1][e]) : v[0][e];
        const int nv = (int)min((int64_t)4, nout - col);
        if (EPI == SPG_EPI_ADD) {
            if (g.bias_mode != 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < nv) o[e] += bias_at(g, b, col + e);
            } else {
                const uint16_t *rrow = g.residual + (g.stride_r ? b * g.stride_r : 0) + m * g.ldr + col;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (e < nv) o[e] += __uint_as_float((uint32_t)rrow[e] << 16);
            }
        }
        const uint2 pk = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
        int64_t ld;
        uint16_t *const dst = g.nseg ? out_at(g, b, m, col, ld)   // a 4-column group never straddles segments
                                     : (uint16_t *)g.out + ((!EXPERTS && g.stride_o) ? b * g.stride_o : 0) + m * g.ldo + col;
        (void)ld;
        if (nv == 4 && (((uintptr_t)dst) & 7) == 0) {
            *reinterpret_cast<uint2 *>(dst) = pk;
        } else {
            const uint32_t wd[2] = {pk.x, pk.y};
            for (int e = 0; e < nv; ++e) dst[e] = (uint16_t)(wd[e >> 1] >> (16 * (e & 1)));
        }
    }
    clock_mark(g.clocks, 1);
}

template <int EPI, bool EXPERTS>
hipError_t launch_epi(const BlockArgs &a, int bm, int64_t workgroups, hipStream_t s)
{
    constexpr int RB = narrow_cols(EPI) / 16;
    if (bm == 16) {
        gemm_block_narrow_kernel<EPI, 1, RB, EXPERTS><<<dim3((unsigned)workgroups), kNarrowThreads, 0, s>>>(a);
        return hipGetLastError();
    }
    if constexpr (!EXPERTS) {                            // experts take 16 or at least 128 rows
        gemm_block_narrow_kernel<EPI, 2, RB, false><<<dim3((unsigned)workgroups), kNarrowThreads, 0, s>>>(a);
        return hipGetLastError();
    }
    return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_gemm_block_narrow(const BlockArgs &a, int bm, int64_t workgroups, hipStream_t s)
{
    const bool x = a.experts > 0;
    switch (a.g.epilogue) {
    case SPG_EPI_ADD: return x ? hipErrorInvalidValue : launch_epi<SPG_EPI_ADD, false>(a, bm, workgroups, s);
    case SPG_EPI_SWIGLU:
        return x ? launch_epi<SPG_EPI_SWIGLU, true>(a, bm, workgroups, s)
                 : launch_epi<SPG_EPI_SWIGLU, false>(a, bm, workgroups, s);
    default:
        return x ? launch_epi<SPG_EPI_STORE, true>(a, bm, workgroups, s)
                 : launch_epi<SPG_EPI_STORE, false>(a, bm, workgroups, s);
    }
}

}  // namespace spg
