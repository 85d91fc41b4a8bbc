// RMS norm with the residual's addition in front and an 8-bit output behind,
// and its gradients.
//
//   h = bf16(x + residual)        the residual stream, stored as it is normed
//   rstd = 1 / sqrt(mean(h^2) + eps)
//   y = (h rstd) (w + w0)
//   out: bf16(y), or E4M3 codes of y / s with s = fl32(max |y| / 448) over the
//   row or over 128 elements of it
//
// The squares are summed in 64 bits: they are exact there and bf16's largest
// values do not overflow, so rstd is a correctly rounded fp32 number but for a
// last bit in some 2^-20 of the rows.  y is fp32 and is rounded once, to the
// output's type (not to bf16 in between).
//
// A stream: 2 to 4 bytes in, 1 to 5 out per element.  A row is read once and
// stays in the registers of its team of 16, 64, 256 or 1024 lanes, each with V
// vectors of eight elements; a lane's loads are all in flight before the first
// square.
#include "spg_gemm_common.h"
#include "spg_norm.h"
#include "spg_quant_common.h"

namespace spg {

namespace {

using namespace quant;

// Eight bf16 values at any address that a bf16 may have: the hardware takes
// 16-byte accesses at 2-byte alignment, so rows of odd length or odd stride
// move as vectors too; the row's last, partial vector moves by elements.
struct __attribute__((packed, aligned(2))) Vec8 {
    uint32_t w[4];
};
__device__ __forceinline__ uint4 load8(const uint16_t *p, int n)
{
    if (n >= 8) {
        const Vec8 v = *reinterpret_cast<const Vec8 *>(p);
        return make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    }
    uint32_t h[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int i = 0; i < 7; ++i)
        if (i < n) h[i] = p[i];
    return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6]);
}
__device__ __forceinline__ void store8(uint16_t *p, const uint4 &v, int n)
{
    if (n >= 8) {
        *reinterpret_cast<Vec8 *>(p) = Vec8{{v.x, v.y, v.z, v.w}};
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    for (int i = 0; i < 7; ++i)
        if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
}
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(gemm::pack_bf16x2(f[0], f[1]), gemm::pack_bf16x2(f[2], f[3]), gemm::pack_bf16x2(f[4], f[5]),
                      gemm::pack_bf16x2(f[6], f[7]));
}
// Eight weights + w0 (w0 past the row, where nothing but zeros is weighted).
struct __attribute__((packed, aligned(4))) Vec8f {
    float f[8];
};
__device__ __forceinline__ void weights8(const void *weight, int w32, float w0, int64_t col, int n, float (&f)[8])
{
    if (w32) {
        const float *p = (const float *)weight + col;
        Vec8f v = {};
        if (n >= 8)
            v = *reinterpret_cast<const Vec8f *>(p);
        else
            for (int i = 0; i < 7; ++i)
                if (i < n) v.f[i] = p[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = v.f[i] + w0;
    } else {
        unpack8(n > 0 ? load8((const uint16_t *)weight + col, n) : make_uint4(0, 0, 0, 0), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += w0;
    }
}

// E4M3 codes of eight fp32 values by their group's scale (see RowScale).
__device__ __forceinline__ uint2 encode8_f32(const float (&y)[8], const RowScale &t)
{
    uint32_t out[2];
    if (t.fast) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int d = __builtin_amdgcn_cvt_pk_fp8_f32(quot<true>(y[4 * h], t), quot<true>(y[4 * h + 1], t), 0, false);
            d = __builtin_amdgcn_cvt_pk_fp8_f32(quot<true>(y[4 * h + 2], t), quot<true>(y[4 * h + 3], t), d, true);
            out[h] = (uint32_t)d;
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            out[h] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float v = y[4 * h + i];
                out[h] |= (t.s > 0.0f ? encode_e4m3(v / t.s) : (__float_as_uint(v) >> 24) & 0x80u) << (8 * i);
            }
        }
    }
    return make_uint2(out[0], out[1]);
}

// Sums and maxima over the TEAM lanes of a row, a power of two: inside a wave
// by exchange, then over the workgroup's waves in LDS, in a fixed order.
template <int TEAM, typename T, typename F>
__device__ __forceinline__ T wave_fold(T v, F &&f)
{
#pragma unroll
    for (int off = (TEAM < 64 ? TEAM : 64) / 2; off >= 1; off >>= 1) v = f(v, __shfl_xor(v, off, 64));
    return v;
}
template <int TEAM, int U, typename T, typename F>
__device__ __forceinline__ void team_fold(T (&v)[U], T (*lds)[U], F &&f)
{
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = wave_fold<TEAM>(v[u], f);
    if constexpr (TEAM > 64) {
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int u = 0; u < U; ++u) lds[threadIdx.x >> 6][u] = v[u];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = lds[0][u];
            for (int w = 1; w < TEAM / 64; ++w) v[u] = f(v[u], lds[w][u]);
        }
    }
}

// 1 / sqrt(m) for m >= 0: the hardware's estimate and two steps of Newton's
// method in 64 bits.  m = 0 gives infinity, infinity 0, NaN NaN.
__device__ __forceinline__ float inverse_root(double m)
{
    const double y = __builtin_amdgcn_rsq(m);
    double z = y;
#pragma unroll
    for (int i = 0; i < 2; ++i) z = __builtin_fma(0.5 * z, __builtin_fma(-m * z, z, 1.0), z);
    return (float)(m > 0.0 && m < __builtin_inf() ? z : y);
}

// One team of TEAM lanes per row, U rows a team at once; lane t holds the
// vectors t + TEAM v of its row, so the 16 lanes of a 128-element group are
// neighbours.
template <int TEAM, int V, int U, int OUTPUT>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void rms_norm_kernel(const NormArgs a)
{
    constexpr int THREADS = TEAM < 256 ? 256 : TEAM, TEAMS = THREADS / TEAM;
    __shared__ double lds_sum[THREADS / 64][U];
    __shared__ uint32_t lds_max[THREADS / 64][U];
    const int t = (int)threadIdx.x % TEAM, team = (int)threadIdx.x / TEAM;
    const int64_t row0 = (int64_t)blockIdx.x * (TEAMS * U) + team;      // rows row0 + u TEAMS
    const int H = (int)a.H;
    uint4 hv[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t row = row0 + u * TEAMS;
            const int col = (t + v * TEAM) * 8;
            hv[u][v] = make_uint4(0, 0, 0, 0);
            if (row < a.R && col < H) hv[u][v] = load8(a.x + row * a.ldx + col, H - col);
        }
    if (a.residual) {
        uint4 rv[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int64_t row = row0 + u * TEAMS;
                const int col = (t + v * TEAM) * 8;
                rv[u][v] = make_uint4(0, 0, 0, 0);
                if (row < a.R && col < H) rv[u][v] = load8(a.residual + row * a.ldr + col, H - col);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float f[8], r[8];
                unpack8(hv[u][v], f);
                unpack8(rv[u][v], r);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] += r[i];
                hv[u][v] = pack8(f);
            }
    }
    // the weights' round trip: in front of the sum for short rows, whose time
    // is latency; behind it for others, where their registers hold more waves
    // back than the trip costs
    constexpr bool EARLY = U * V == 1;
    float w[V][8];
    auto load_weights = [&]() {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (t + v * TEAM) * 8;
            weights8(a.weight, a.w32, a.w0, col, H - col, w[v]);
        }
    };
    if (EARLY) load_weights();
    double ss[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        ss[u] = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float f[8];
            unpack8(hv[u][v], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss[u] = __builtin_fma((double)f[i], (double)f[i], ss[u]);
        }
    }
    if (!EARLY) {
        __builtin_amdgcn_sched_barrier(0);
        load_weights();
    }
    team_fold<TEAM>(ss, lds_sum, [](double p, double q) { return p + q; });
    float rstd[U];
    uint32_t amax[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = row0 + u * TEAMS;
        rstd[u] = inverse_root(ss[u] / (double)H + a.eps);
        if (a.rstd && t == 0 && row < a.R) a.rstd[row] = rstd[u];
        amax[u] = 0;
        if (a.residual) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int col = (t + v * TEAM) * 8;
                if (row < a.R && col < H) store8(a.h + row * a.ldh + col, hv[u][v], H - col);
            }
        }
    }
    auto values = [&](int u, int v, float (&y)[8]) {
        unpack8(hv[u][v], y);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = (y[i] * rstd[u]) * w[v][i];
    };
    auto largest = [](const float (&y)[8]) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
        return m;
    };
    if constexpr (OUTPUT == SPG_NORM_E4M3_ROW) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float y[8];
                values(u, v, y);
                if ((t + v * TEAM) * 8 < H) amax[u] = max(amax[u], largest(y));
            }
        team_fold<TEAM>(amax, lds_max, [](uint32_t p, uint32_t q) { return p > q ? p : q; });
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t row = row0 + u * TEAMS;
        RowScale rs;
        if constexpr (OUTPUT == SPG_NORM_E4M3_ROW) {
            rs = row_scale(__uint_as_float(amax[u]));
            if (t == 0 && row < a.R) a.scale[row] = rs.s;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (t + v * TEAM) * 8;
            float y[8];
            values(u, v, y);
            const bool in = row < a.R && col < H;
            if constexpr (OUTPUT == SPG_NORM_E4M3_BLOCK128) {
                rs = row_scale(__uint_as_float(wave_fold<16>(in ? largest(y) : 0u, [](uint32_t p, uint32_t q) { return p > q ? p : q; })));
                if (in && (t & 15) == 0) a.scale[(int64_t)(col >> 7) * a.R + row] = rs.s;
            }
            if (!in) continue;
            if constexpr (OUTPUT != SPG_NORM_BF16)
                *reinterpret_cast<uint2 *>(a.q + row * a.ldq + col) = encode8_f32(y, rs);    // H % 16 == 0
            if (OUTPUT == SPG_NORM_BF16 || a.normed) store8(a.normed + row * a.ldn + col, pack8(y), H - col);
        }
    }
}

template <int TEAM, int V, int U>
hipError_t launch_team(const NormArgs &a, hipStream_t s)
{
    constexpr int THREADS = TEAM < 256 ? 256 : TEAM, ROWS = THREADS / TEAM * U;
    const unsigned grid = (unsigned)((a.R + ROWS - 1) / ROWS);
    if (a.output == SPG_NORM_BF16)
        rms_norm_kernel<TEAM, V, U, SPG_NORM_BF16><<<grid, THREADS, 0, s>>>(a);
    else if (a.output == SPG_NORM_E4M3_ROW)
        rms_norm_kernel<TEAM, V, U, SPG_NORM_E4M3_ROW><<<grid, THREADS, 0, s>>>(a);
    else
        rms_norm_kernel<TEAM, V, U, SPG_NORM_E4M3_BLOCK128><<<grid, THREADS, 0, s>>>(a);
    return hipGetLastError();
}

// ---- gradients -----------------------------------------------------------------
//   g = dy (w + w0), xh = h rstd, m = mean(g xh)
//   dx = rstd (g - xh m) + dres        one rounding to bf16
//   dw = sum over the rows of dy xh    fp32
//
// A workgroup walks over rows, U a team at once (all of their loads in flight
// before the first product); a lane keeps its columns' weights and sums of dw
// in registers.  Every workgroup leaves one partial sum of dw, which a second
// launch adds in the workgroups' order.  Partial sums lie as the lanes hold
// them: element i of vector t + TEAM v at (i V + v) TEAM + t.
template <int TEAM, int V, int U>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void rms_norm_backward_kernel(const NormGradArgs a)
{
    constexpr int THREADS = TEAM < 256 ? 256 : TEAM, TEAMS = THREADS / TEAM, WIDTH = TEAM * V * 8;
    __shared__ float lds_sum[2][THREADS / 64][U];
    __shared__ float lds_dw[TEAMS > 1 ? TEAMS : 1][TEAMS > 1 ? WIDTH : 1];
    const int t = (int)threadIdx.x % TEAM, team = (int)threadIdx.x / TEAM;
    const int H = (int)a.H;
    // (the longest rows' weights would not fit beside the rest: read again per row)
    constexpr bool KEEP = TEAM * V < 4096;
    float w[KEEP ? V : 1][8], dw[V][8];
    auto weights = [&](int v) {
        const int col = (t + v * TEAM) * 8;
        weights8(a.weight, a.w32, a.w0, col, H - col, w[KEEP ? v : 0]);
    };
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (KEEP) weights(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
    }
    int parity = 0;
    for (int64_t first = (int64_t)blockIdx.x * (TEAMS * U); first < a.R; first += (int64_t)gridDim.x * (TEAMS * U), parity ^= 1) {
        uint4 cd[U][V], ch[U][V], cr[U][V];
        float rstd[U], dot[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = first + team + u * TEAMS;
            rstd[u] = row < a.R ? a.rstd[row] : 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int col = (t + v * TEAM) * 8;
                cd[u][v] = ch[u][v] = cr[u][v] = make_uint4(0, 0, 0, 0);
                if (row < a.R && col < H) {
                    cd[u][v] = load8(a.dy + row * a.lddy + col, H - col);
                    ch[u][v] = load8(a.h + row * a.ldh + col, H - col);
                    if (a.dres) cr[u][v] = load8(a.dres + row * a.lddr + col, H - col);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            dot[u] = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float d[8], h[8];
                unpack8(cd[u][v], d);
                unpack8(ch[u][v], h);
                if (!KEEP) weights(v);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = d[i] * (h[i] * rstd[u]);
                    dot[u] = __builtin_fmaf(p, w[KEEP ? v : 0][i], dot[u]);
                    dw[v][i] += p;
                }
            }
        }
        team_fold<TEAM>(dot, lds_sum[parity], [](float p, float q) { return p + q; });
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = first + team + u * TEAMS;
            const float m = dot[u] / (float)H;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int col = (t + v * TEAM) * 8;
                float d[8], h[8], r[8];
                unpack8(cd[u][v], d);
                unpack8(ch[u][v], h);
                unpack8(cr[u][v], r);
                if (!KEEP) weights(v);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[i] = __builtin_fmaf(__builtin_fmaf(-(h[i] * rstd[u]), m, d[i] * w[KEEP ? v : 0][i]), rstd[u], r[i]);
                if (row < a.R && col < H) store8(a.dx + row * a.lddx + col, pack8(r), H - col);
            }
        }
    }
    if (!a.dw) return;
    // one workgroup: its sums are the result
    float *const part = a.partials + (int64_t)blockIdx.x * WIDTH;
    auto leave = [&](int at, float s) {
        if (gridDim.x > 1)
            part[at] = s;
        else if (const int col = (at % (TEAM * V)) * 8 + at / (TEAM * V); col < H)
            a.dw[col] = s;
    };
    if constexpr (TEAMS > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) lds_dw[team][(i * V + v) * TEAM + t] = dw[v][i];
        __syncthreads();
        for (int at = (int)threadIdx.x; at < WIDTH; at += THREADS) {
            float s = lds_dw[0][at];
            for (int k = 1; k < TEAMS; ++k) s += lds_dw[k][at];
            leave(at, s);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) leave((i * V + v) * TEAM + t, dw[v][i]);
    }
}

// Sum of the partial sums [parts, width]: 16 places a workgroup, 64 runs of at
// most kRun parts side by side (each run's loads all in flight), joined eight by
// eight in order.
constexpr int kRun = 8;
__global__ __launch_bounds__(1024) void norm_dw_reduce_kernel(const float *partials, int parts, int width, int64_t H, float *dw)
{
    __shared__ float lds[64][16], lds8[8][16];
    const int c = (int)threadIdx.x & 15, k = (int)threadIdx.x >> 4;
    const int at = (int)blockIdx.x * 16 + c;
    const int per = (parts + 63) / 64;
    float s = 0.0f;
    for (int p0 = 0; p0 < per; p0 += kRun) {
        float v[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            const int p = k * per + p0 + i;
            v[i] = p0 + i < per && p < parts ? partials[(int64_t)p * width + at] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kRun; ++i) s += v[i];
    }
    lds[k][c] = s;
    __syncthreads();
    if (k < 8) {
        s = lds[8 * k][c];
        for (int i = 1; i < 8; ++i) s += lds[8 * k + i][c];
        lds8[k][c] = s;
    }
    __syncthreads();
    if (k == 0) {
        s = lds8[0][c];
        for (int i = 1; i < 8; ++i) s += lds8[i][c];
        const int vecs = width / 8, col = (at % vecs) * 8 + at / vecs;
        if (col < H) dw[col] = s;
    }
}

constexpr int64_t kGradWorkgroups = 512;

// Calls f(team, vectors, rows at once) for rows of H elements.
template <int N>
using Int = std::integral_constant<int, N>;
template <typename F>
auto with_grad_shape(int64_t H, F &&f)
{
    if (H <= 128) return f(Int<16>{}, Int<1>{}, Int<4>{});
    if (H <= 256) return f(Int<16>{}, Int<2>{}, Int<2>{});
    if (H <= 512) return f(Int<16>{}, Int<4>{}, Int<2>{});
    if (H <= 1024) return f(Int<64>{}, Int<2>{}, Int<2>{});
    if (H <= 2048) return f(Int<64>{}, Int<4>{}, Int<2>{});
    if (H <= 4096) return f(Int<256>{}, Int<2>{}, Int<2>{});
    if (H <= 6144) return f(Int<256>{}, Int<3>{}, Int<2>{});
    if (H <= 8192) return f(Int<256>{}, Int<4>{}, Int<2>{});
    if (H <= 16384) return f(Int<1024>{}, Int<2>{}, Int<1>{});
    return f(Int<1024>{}, Int<4>{}, Int<1>{});
}

}  // namespace

int64_t norm_grad_parts(int64_t R, int64_t H)
{
    const int64_t rows = with_grad_shape(H, [](auto team, auto, auto u) { return (team < 256 ? 256 / team : 1) * u; });
    const int64_t n = (R + rows - 1) / rows;
    return n < 1 ? 1 : n < kGradWorkgroups ? n : kGradWorkgroups;     // no rows: one, which writes zeros
}

int64_t norm_grad_width(int64_t H)
{
    return with_grad_shape(H, [](auto team, auto v, auto) { return 8 * team * v; });
}

hipError_t launch_rms_norm(const NormArgs &a, hipStream_t s)
{
    const int64_t H = a.H;
    if (H <= 128) return launch_team<16, 1, 4>(a, s);
    if (H <= 256) return launch_team<16, 2, 2>(a, s);
    if (H <= 512) return launch_team<16, 4, 1>(a, s);
    if (H <= 1024) return launch_team<64, 2, 1>(a, s);
    if (a.R <= 256 && H <= 2048) return launch_team<256, 1, 1>(a, s);
    if (H <= 2048) return launch_team<64, 4, 1>(a, s);
    if (a.R <= 256 && H <= 8192) return launch_team<1024, 1, 1>(a, s);
    if (H <= 4096) return launch_team<256, 2, 1>(a, s);
    if (H <= 6144) return launch_team<256, 3, 1>(a, s);
    if (H <= 8192) return launch_team<256, 4, 1>(a, s);
    if (H <= 16384) return launch_team<1024, 2, 1>(a, s);
    return launch_team<1024, 4, 1>(a, s);
}

hipError_t launch_rms_norm_backward(const NormGradArgs &a, hipStream_t s)
{
    const int64_t parts = norm_grad_parts(a.R, a.H);
    const hipError_t e = with_grad_shape(a.H, [&](auto team, auto v, auto u) {
        constexpr int TEAM = decltype(team)::value;
        rms_norm_backward_kernel<TEAM, decltype(v)::value, decltype(u)::value>
            <<<(unsigned)parts, TEAM < 256 ? 256 : TEAM, 0, s>>>(a);
        return hipGetLastError();
    });
    if (e != hipSuccess || !a.dw || parts == 1) return e;
    const int64_t width = norm_grad_width(a.H);
    norm_dw_reduce_kernel<<<(unsigned)(width / 16), 1024, 0, s>>>(a.partials, (int)parts, (int)width, a.H, a.dw);
    return hipGetLastError();
}

}  // namespace spg
