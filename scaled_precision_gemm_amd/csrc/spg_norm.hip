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
    float w[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int col = (t + v * TEAM) * 8;
        weights8(a.weight, a.w32, a.w0, col, H - col, w[v]);
    }
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
// A workgroup walks over rows blockIdx.x, + gridDim.x, ...; a lane keeps its
// columns' weights and sums of dw in registers, and the next row's loads are
// in flight while this row is summed.  Every workgroup leaves one partial sum
// of dw, which a second launch adds in the workgroups' order.
template <int TEAM, int V>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void rms_norm_backward_kernel(const NormGradArgs a)
{
    constexpr int THREADS = TEAM < 256 ? 256 : TEAM, TEAMS = THREADS / TEAM;
    __shared__ float lds_sum[2][THREADS / 64][1];
    __shared__ float lds_dw[TEAMS > 1 ? TEAMS : 1][TEAMS > 1 ? TEAM * V * 8 : 1];
    const int t = (int)threadIdx.x % TEAM, team = (int)threadIdx.x / TEAM;
    const int H = (int)a.H;
    float w[V][8], dw[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int col = (t + v * TEAM) * 8;
        weights8(a.weight, a.w32, a.w0, col, H - col, w[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
    }
    uint4 nd[V], nh[V], nr[V];
    float ns = 0.0f;
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (t + v * TEAM) * 8;
            nd[v] = nh[v] = nr[v] = make_uint4(0, 0, 0, 0);
            if (row < a.R && col < H) {
                nd[v] = load8(a.dy + row * a.lddy + col, H - col);
                nh[v] = load8(a.h + row * a.ldh + col, H - col);
                if (a.dres) nr[v] = load8(a.dres + row * a.lddr + col, H - col);
            }
        }
        ns = row < a.R ? a.rstd[row] : 0.0f;
    };
    const int64_t step = (int64_t)gridDim.x * TEAMS;
    fetch((int64_t)blockIdx.x * TEAMS + team);
    int parity = 0;
    for (int64_t first = (int64_t)blockIdx.x * TEAMS; first < a.R; first += step, parity ^= 1) {
        const int64_t row = first + team;
        uint4 cd[V], ch[V], cr[V];
        const float rstd = ns;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            cd[v] = nd[v];
            ch[v] = nh[v];
            cr[v] = nr[v];
        }
        fetch(row + step);
        float dot[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float d[8], h[8];
            unpack8(cd[v], d);
            unpack8(ch[v], h);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = d[i] * (h[i] * rstd);
                dot[0] = __builtin_fmaf(p, w[v][i], dot[0]);
                dw[v][i] += p;
            }
        }
        team_fold<TEAM>(dot, lds_sum[parity], [](float p, float q) { return p + q; });
        const float m = dot[0] / (float)H;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (t + v * TEAM) * 8;
            float d[8], h[8], r[8];
            unpack8(cd[v], d);
            unpack8(ch[v], h);
            unpack8(cr[v], r);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r[i] = __builtin_fmaf(__builtin_fmaf(-(h[i] * rstd), m, d[i] * w[v][i]), rstd, r[i]);
            if (row < a.R && col < H) store8(a.dx + row * a.lddx + col, pack8(r), H - col);
        }
    }
    if (!a.dw) return;
    float *out = gridDim.x > 1 ? a.partials + (int64_t)blockIdx.x * a.H : a.dw;
    if constexpr (TEAMS > 1) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) lds_dw[team][(t + v * TEAM) * 8 + i] = dw[v][i];
        __syncthreads();
        for (int c = (int)threadIdx.x; c < H; c += THREADS) {
            float s = lds_dw[0][c];
            for (int k = 1; k < TEAMS; ++k) s += lds_dw[k][c];
            out[c] = s;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (t + v * TEAM) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i < H) out[col + i] = dw[v][i];
        }
    }
}

// dw[c] = sum of the partial sums [parts, H]: 32 columns a workgroup, eight
// runs of parts side by side, joined in order.
__global__ __launch_bounds__(256) void norm_dw_reduce_kernel(const float *partials, int parts, int64_t H, float *dw)
{
    __shared__ float lds[8][32];
    const int c = (int)threadIdx.x & 31, k = (int)threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + c;
    const int per = (parts + 7) / 8, end = min(parts, (k + 1) * per);
    float s = 0.0f;
    if (col < H)
        for (int p = k * per; p < end; ++p) s += partials[(int64_t)p * H + col];
    lds[k][c] = s;
    __syncthreads();
    if (k == 0 && col < H) {
        for (int i = 1; i < 8; ++i) s += lds[i][c];
        dw[col] = s;
    }
}

constexpr int64_t kGradWorkgroups = 512;

int grad_team(int64_t H) { return H <= 512 ? 16 : H <= 2048 ? 64 : H <= 8192 ? 256 : 1024; }

template <int TEAM, int V>
hipError_t launch_grad(const NormGradArgs &a, hipStream_t s)
{
    rms_norm_backward_kernel<TEAM, V><<<(unsigned)norm_grad_parts(a.R, a.H), TEAM < 256 ? 256 : TEAM, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

int64_t norm_grad_parts(int64_t R, int64_t H)
{
    const int team = grad_team(H), teams = team < 256 ? 256 / team : 1;
    const int64_t n = (R + teams - 1) / teams;
    return n < 1 ? 1 : n < kGradWorkgroups ? n : kGradWorkgroups;     // no rows: one, which writes zeros
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
    const int64_t H = a.H;
    const hipError_t e = H <= 128     ? launch_grad<16, 1>(a, s)
                         : H <= 256   ? launch_grad<16, 2>(a, s)
                         : H <= 512   ? launch_grad<16, 4>(a, s)
                         : H <= 1024  ? launch_grad<64, 2>(a, s)
                         : H <= 2048  ? launch_grad<64, 4>(a, s)
                         : H <= 4096  ? launch_grad<256, 2>(a, s)
                         : H <= 6144  ? launch_grad<256, 3>(a, s)
                         : H <= 8192  ? launch_grad<256, 4>(a, s)
                         : H <= 16384 ? launch_grad<1024, 2>(a, s)
                                      : launch_grad<1024, 4>(a, s);
    if (e != hipSuccess || !a.dw) return e;
    const int64_t parts = norm_grad_parts(a.R, a.H);
    if (parts > 1) {
        norm_dw_reduce_kernel<<<(unsigned)((H + 31) / 32), 256, 0, s>>>(a.partials, (int)parts, H, a.dw);
        return hipGetLastError();
    }
    return hipSuccess;
}

}  // namespace spg
