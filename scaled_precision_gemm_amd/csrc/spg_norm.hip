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
// stays in the registers of its team of 8 to 1024 lanes, each with V
// vectors of eight elements; a lane's loads are all in flight before the first
// square.  With a residual and row scales 4096 x 5120 (147 MB) takes 30 us, 4.9
// TB/s, and 500000 x 128 82 us, 5.4 TB/s: the memory's rate.  44440 x 128 in bf16
// (23 MB) takes 8 us, half of it start and drain; up to 256 rows take 2.5 to 5.9
// us, a load's, a reduction's and a store's latency.
#include "spg_gemm_common.h"
#include "spg_norm.h"
#include "spg_quant_common.h"

#include <type_traits>

namespace spg {

namespace {

using namespace quant;

// Eight bf16 values at any address that a bf16 may have: the hardware takes
// 16-byte accesses at 2-byte alignment, so rows of odd length or odd stride
// move as vectors too; the row's last, partial vector moves by elements.
struct __attribute__((packed, aligned(2))) Vec8 {
    uint32_t w[4];
};
// The vectors at columns (t + v TEAM) 8 of the rows row[u] of a matrix, zeros
// past its last row and column.  No branch stands between the vectors' loads,
// so that all are in flight at once: lanes without a whole vector read the
// matrix's first one.  (With a branch around each the compiler waited for every
// load: 4096 x 5120 with row scales 42 us, 35 without; its gradients 62 and 53.)
template <int TEAM, int V, int U>
__device__ __forceinline__ void load_rows(uint4 (&out)[U][V], const uint16_t *p, int64_t ld, const int64_t (&row)[U], int64_t R,
                                          int H, int t)
{
    if (H >= 8) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int col = (t + v * TEAM) * 8;
                const bool in = row[u] < R && col + 8 <= H;
                const Vec8 x = *reinterpret_cast<const Vec8 *>(p + (in ? row[u] * ld + col : 0));
                out[u][v] = make_uint4(in ? x.w[0] : 0, in ? x.w[1] : 0, in ? x.w[2] : 0, in ? x.w[3] : 0);
            }
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int v = 0; v < V; ++v) out[u][v] = make_uint4(0, 0, 0, 0);
    }
    if (H & 7) {
        // one vector of the row is partial: lane (H / 8) % TEAM's number H / 8 / TEAM
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int col = (t + v * TEAM) * 8, n = H - col;
                if (row[u] < R && n > 0 && n < 8) {
                    const uint16_t *q = p + row[u] * ld + col;
                    uint32_t h[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                    for (int i = 0; i < 7; ++i)
                        if (i < n) h[i] = q[i];
                    out[u][v] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6]);
                }
            }
    }
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
// Keeps the vectors packed here: the compiler otherwise holds the values that
// it unpacked before a reduction over it, twice the registers.
template <int U, int V>
__device__ __forceinline__ void keep_packed(uint4 (&x)[U][V])
{
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int v = 0; v < V; ++v) asm volatile("" : "+v"(x[u][v].x), "+v"(x[u][v].y), "+v"(x[u][v].z), "+v"(x[u][v].w));
}

// The weights + w0 of a lane's columns (w0 past the row, where nothing but
// zeros is weighted), loaded like the rows.
struct __attribute__((packed, aligned(4))) Vec8f {
    float f[8];
};
template <int TEAM, int V>
__device__ __forceinline__ void load_weights(float (&w)[V][8], const void *weight, int w32, float w0, int H, int t)
{
    if (w32) {
        const float *p = (const float *)weight;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (t + v * TEAM) * 8;
            Vec8f x = {};
            if (H >= 8) x = *reinterpret_cast<const Vec8f *>(p + (col + 8 <= H ? col : 0));
#pragma unroll
            for (int i = 0; i < 8; ++i) w[v][i] = col + 8 <= H ? x.f[i] : 0.0f;
        }
        if (H & 7) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int col = (t + v * TEAM) * 8;
#pragma unroll
                for (int i = 0; i < 7; ++i)
                    if (col + i < H && col + 8 > H) w[v][i] = p[col + i];
            }
        }
    } else {
        uint4 x[1][V];
        const int64_t row[1] = {0};
        load_rows<TEAM>(x, (const uint16_t *)weight, 0, row, 1, H, t);
#pragma unroll
        for (int v = 0; v < V; ++v) unpack8(x[0][v], w[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) w[v][i] += w0;
}

// A group's scale s = fl32(amax / 448), amax = max |y| = max |y0| m.  m falls
// out of a quotient by the unrounded scale, y0 (448 / max |y0|), whose factor is
// held as a sum of two numbers: the codes' quotients are within a last bit (the
// products of bf16 weights y0 are exact).  Scales far from 1, zero and those
// that are not finite take IEEE division of y by s.
struct GroupScale {
    float s, f, f2;
    bool plain;
};
__device__ __forceinline__ GroupScale group_scale(uint32_t amax0, float m)
{
    GroupScale t;
    const float a = __uint_as_float(amax0);
    t.s = a * m / 448.0f;          // rounding keeps the order: max |y0| m is max |y|
    t.plain = t.s > 0x1p-100f && t.s < 0x1p100f;
    const float r = __builtin_amdgcn_rcpf(a);
    t.f = 448.0f * r;
    t.f = __builtin_fmaf(__builtin_fmaf(-t.f, a, 448.0f), r, t.f);
    t.f2 = __builtin_fmaf(-t.f, a, 448.0f) * r;
    if (t.f2 < 0.0f) {             // both of one sign: y0 = -0 stays -0
        t.f = __uint_as_float(__float_as_uint(t.f) - 1);
        t.f2 = __builtin_fmaf(-t.f, a, 448.0f) * r;
    }
    return t;
}
// The same with y0 and its largest value in 64 bits, where products of fp32
// weights, or of weights + w0, are exact as well: of 53 million codes of such rows
// 19 are not the nearest ones, 28 with products in 32 bits, 33 where y and y / s
// are formed one after the other (4096 x 2048 17.1 us, in 32 bits 15.8).
struct WideScale {
    float s;
    double f;
    bool plain;
};
__device__ __forceinline__ WideScale group_scale(double amax0, float m)
{
    WideScale t;
    t.s = (float)amax0 * m / 448.0f;
    t.plain = t.s > 0x1p-100f && t.s < 0x1p100f;
    double r = __builtin_amdgcn_rcp(amax0);
    r = __builtin_fma(__builtin_fma(-amax0, r, 1.0), r, r);
    t.f = 448.0 * r;
    return t;
}
__device__ __forceinline__ float quotient(float y0, const GroupScale &t) { return __builtin_fmaf(y0, t.f, y0 * t.f2); }
__device__ __forceinline__ float quotient(double y0, const WideScale &t) { return (float)(y0 * t.f); }
template <typename Y, typename S>
__device__ __forceinline__ uint2 encode8(const Y (&y0)[8], float m, const S &t)
{
    uint32_t out[2];
    if (t.plain) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = __builtin_amdgcn_fmed3f(quotient(y0[4 * h + i], t), -448.0f, 448.0f);
            const int d = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
            out[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], d, true);
        }
        return make_uint2(out[0], out[1]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        out[h] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = (float)y0[4 * h + i] * m;
            out[h] |= (t.s > 0.0f ? encode_e4m3(v / t.s) : (__float_as_uint(v) >> 24) & 0x80u) << (8 * i);
        }
    }
    return make_uint2(out[0], out[1]);
}

// Sums and maxima over the TEAM lanes of a row, a power of two: inside a wave
// by moves within 16 lanes and exchanges of 16- and 32-lane halves, all in
// the vector unit, then over the workgroup's waves in LDS, in a fixed order.
template <int CTRL>
__device__ __forceinline__ uint32_t move16(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ double move16(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)move16<CTRL>((uint32_t)u) | (uint64_t)move16<CTRL>((uint32_t)(u >> 32)) << 32);
}
template <int CTRL>
__device__ __forceinline__ float move16(float v)
{
    return __uint_as_float(move16<CTRL>(__float_as_uint(v)));
}
// The values of the two halves (of 32 lanes where HALF is 16, else of 64), each
// in both: first, second.
template <int HALF>
__device__ __forceinline__ void halves(uint32_t v, uint32_t &p, uint32_t &q)
{
    if (HALF == 16) {
        const auto t = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        p = t[0];
        q = t[1];
    } else {
        const auto t = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        p = t[0];
        q = t[1];
    }
}
template <int HALF>
__device__ __forceinline__ void halves(float v, float &p, float &q)
{
    uint32_t a, b;
    halves<HALF>(__float_as_uint(v), a, b);
    p = __uint_as_float(a);
    q = __uint_as_float(b);
}
template <int HALF>
__device__ __forceinline__ void halves(double v, double &p, double &q)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    uint32_t a, b, c, d;
    halves<HALF>((uint32_t)u, a, b);
    halves<HALF>((uint32_t)(u >> 32), c, d);
    p = __builtin_bit_cast(double, (uint64_t)a | (uint64_t)c << 32);
    q = __builtin_bit_cast(double, (uint64_t)b | (uint64_t)d << 32);
}
template <int TEAM, typename T, typename F>
__device__ __forceinline__ T wave_fold(T v, F &&f)
{
    v = f(v, move16<0xB1>(v));                           // lanes 1 0 3 2 of a quad
    v = f(v, move16<0x4E>(v));                           // 2 3 0 1
    v = f(v, move16<0x141>(v));                          // 7 .. 0 of eight
    if (TEAM > 8) v = f(v, move16<0x140>(v));            // 15 .. 0 of sixteen
    if (TEAM > 16) {
        T p, q;
        halves<16>(v, p, q);
        v = f(p, q);
        halves<32>(v, p, q);
        v = f(p, q);
    }
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
#pragma unroll
            for (int w = 1; w < TEAM / 64; ++w) v[u] = f(v[u], lds[w][u]);
        }
    }
}

// 1 / sqrt(m) for m >= 0: the hardware's estimate and two steps of Newton's
// method in 64 bits.  m = 0 gives infinity, infinity 0, NaN NaN.
__device__ __forceinline__ double inverse_root(double m)
{
    const double y = __builtin_amdgcn_rsq(m);
    double z = y;
#pragma unroll
    for (int i = 0; i < 2; ++i) z = __builtin_fma(0.5 * z, __builtin_fma(-m * z, z, 1.0), z);
    return m > 0.0 && m < __builtin_inf() ? z : y;
}

// One team of TEAM lanes per row, U rows a team at once; lane t holds the
// vectors t + TEAM v of its row, so the 16 lanes of a 128-element group are
// neighbours.
template <int TEAM, int V, int U, int OUTPUT, bool WIDE>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void rms_norm_kernel(const NormArgs a)
{
    constexpr int THREADS = TEAM < 256 ? 256 : TEAM, TEAMS = THREADS / TEAM;
    __shared__ double lds_sum[THREADS / 64][U];
    using Y = std::conditional_t<WIDE, double, float>;           // y0
    using Max = std::conditional_t<WIDE, double, uint32_t>;      // |y0|: its bits, whose order is that of the values
    using Scale = std::conditional_t<WIDE, WideScale, GroupScale>;
    __shared__ Max lds_max[THREADS / 64][U];
    const int t = (int)threadIdx.x % TEAM, team = (int)threadIdx.x / TEAM;
    const int64_t row0 = (int64_t)blockIdx.x * (TEAMS * U) + team;      // rows row0 + u TEAMS
    const int H = (int)a.H;
    int64_t row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) row[u] = row0 + u * TEAMS;
    uint4 hv[U][V];
    load_rows<TEAM>(hv, a.x, a.ldx, row, a.R, H, t);
    if (a.residual) {
        uint4 rv[U][V];
        load_rows<TEAM>(rv, a.residual, a.ldr, row, a.R, H, t);
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
    if (EARLY) load_weights<TEAM>(w, a.weight, a.w32, a.w0, H, t);
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
        load_weights<TEAM>(w, a.weight, a.w32, a.w0, H, t);
    }
    team_fold<TEAM>(ss, lds_sum, [](double p, double q) { return p + q; });
    keep_packed(hv);
    // rstd = c m with a power of two c: h c is exact and near 1 whatever the
    // row's size, y0 = (h c) w, y = y0 m
    float c[U], m[U];
    Max amax[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const double rstd = inverse_root(ss[u] / (double)H + a.eps);
        if (a.rstd && t == 0 && row[u] < a.R) a.rstd[row[u]] = (float)rstd;
        const int e = min(max((int)((__builtin_bit_cast(uint64_t, rstd) >> 52) & 0x7FF) - 1023, -126), 127);
        const bool ordinary = rstd > 0.0 && rstd < __builtin_inf();
        c[u] = ordinary ? __uint_as_float((uint32_t)(e + 127) << 23) : (float)rstd;
        m[u] = ordinary ? (float)(rstd * __builtin_bit_cast(double, (uint64_t)(1023 - e) << 52)) : 1.0f;
        amax[u] = 0;
        if (a.residual) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int col = (t + v * TEAM) * 8;
                if (row[u] < a.R && col < H) store8(a.h + row[u] * a.ldh + col, hv[u][v], H - col);
            }
        }
    }
    auto values = [&](int u, int v, Y (&y)[8]) {
        float f[8];
        unpack8(hv[u][v], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = (Y)(f[i] * c[u]) * (Y)w[v][i];
    };
    // (64 bits: a NaN, which maxima drop, counts as infinity)
    auto largest = [](const Y (&y)[8]) {
        Max m = 0;
        if constexpr (WIDE) {
            bool nan = false;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                m = __builtin_fmax(m, __builtin_fabs(y[i]));
                nan |= y[i] != y[i];
            }
            return nan ? __builtin_inf() : m;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
            return m;
        }
    };
    auto larger = [](Max p, Max q) { return p > q ? p : q; };
    if constexpr (OUTPUT == SPG_NORM_E4M3_ROW) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                Y y[8];
                values(u, v, y);
                if ((t + v * TEAM) * 8 < H) amax[u] = larger(amax[u], largest(y));
            }
        team_fold<TEAM>(amax, lds_max, larger);
        keep_packed(hv);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        Scale rs;
        if constexpr (OUTPUT == SPG_NORM_E4M3_ROW) {
            rs = group_scale(amax[u], m[u]);
            if (t == 0 && row[u] < a.R) a.scale[row[u]] = rs.s;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int col = (t + v * TEAM) * 8;
            Y y[8];
            values(u, v, y);
            const bool in = row[u] < a.R && col < H;
            if constexpr (OUTPUT == SPG_NORM_E4M3_BLOCK128) {
                rs = group_scale(wave_fold<16>(in ? largest(y) : (Max)0, larger), m[u]);
                if (in && (t & 15) == 0) a.scale[(int64_t)(col >> 7) * a.R + row[u]] = rs.s;
            }
            if (!in) continue;
            if constexpr (OUTPUT != SPG_NORM_BF16)
                *reinterpret_cast<uint2 *>(a.q + row[u] * a.ldq + col) = encode8(y, m[u], rs);    // H % 16 == 0
            if (OUTPUT == SPG_NORM_BF16 || a.normed) {
                float n[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) n[i] = (float)y[i] * m[u];
                store8(a.normed + row[u] * a.ldn + col, pack8(n), H - col);
            }
        }
    }
}

template <int TEAM, int V, int U>
hipError_t launch_team(const NormArgs &a, hipStream_t s)
{
    constexpr int THREADS = TEAM < 256 ? 256 : TEAM, ROWS = THREADS / TEAM * U;
    const unsigned grid = (unsigned)((a.R + ROWS - 1) / ROWS);
    // products of bf16 weights are exact in 32 bits
    const bool wide = a.w32 || a.w0 != 0.0f;
    auto launch = [&](auto output) {
        constexpr int O = decltype(output)::value;
        if (O != SPG_NORM_BF16 && wide)
            rms_norm_kernel<TEAM, V, U, O, O != SPG_NORM_BF16><<<grid, THREADS, 0, s>>>(a);
        else
            rms_norm_kernel<TEAM, V, U, O, false><<<grid, THREADS, 0, s>>>(a);
    };
    if (a.output == SPG_NORM_BF16)
        launch(std::integral_constant<int, SPG_NORM_BF16>{});
    else if (a.output == SPG_NORM_E4M3_ROW)
        launch(std::integral_constant<int, SPG_NORM_E4M3_ROW>{});
    else if constexpr (TEAM >= 16)
        launch(std::integral_constant<int, SPG_NORM_E4M3_BLOCK128>{});
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
// them: element i of vector t + TEAM v at (i V + v) TEAM + t.  4096 x 2048 (67 MB)
// takes 15.4 us, 4.4 TB/s, and its partial sums (512 of 2048, in the caches) 3.9.
template <int TEAM, int V, int U>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void rms_norm_backward_kernel(const NormGradArgs a)
{
    constexpr int THREADS = TEAM < 256 ? 256 : TEAM, TEAMS = THREADS / TEAM, WIDTH = TEAM * V * 8;
    __shared__ float lds_sum[2][THREADS / 64][U];
    __shared__ float lds_dw[TEAMS > 1 ? TEAMS : 1][TEAMS > 1 ? WIDTH : 1];
    const int t = (int)threadIdx.x % TEAM, team = (int)threadIdx.x / TEAM;
    const int H = (int)a.H;
    // (the longest rows' weights and added gradients would not fit beside the
    // rest: they are read where they are used, the weights twice a row)
    constexpr bool KEEP = TEAM * V < 4096;
    float w[V][8], dw[V][8];
    if (KEEP) load_weights<TEAM>(w, a.weight, a.w32, a.w0, H, t);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
    int parity = 0;
    for (int64_t first = (int64_t)blockIdx.x * (TEAMS * U); first < a.R; first += (int64_t)gridDim.x * (TEAMS * U), parity ^= 1) {
        uint4 cd[U][V], ch[U][V], cr[U][V] = {};
        int64_t row[U];
        float rstd[U], dot[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            row[u] = first + team + u * TEAMS;
            rstd[u] = a.rstd[row[u] < a.R ? row[u] : 0];
        }
        load_rows<TEAM>(cd, a.dy, a.lddy, row, a.R, H, t);
        load_rows<TEAM>(ch, a.h, a.ldh, row, a.R, H, t);
        if (KEEP && a.dres) load_rows<TEAM>(cr, a.dres, a.lddr, row, a.R, H, t);
#pragma unroll
        for (int u = 0; u < U; ++u) rstd[u] = row[u] < a.R ? rstd[u] : 0.0f;
        if (!KEEP) load_weights<TEAM>(w, a.weight, a.w32, a.w0, H, t);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            dot[u] = 0.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float d[8], h[8];
                unpack8(cd[u][v], d);
                unpack8(ch[u][v], h);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = d[i] * (h[i] * rstd[u]);
                    dot[u] = __builtin_fmaf(p, w[v][i], dot[u]);
                    dw[v][i] += p;
                }
            }
        }
        team_fold<TEAM>(dot, lds_sum[parity], [](float p, float q) { return p + q; });
        keep_packed(cd);
        keep_packed(ch);
        if (!KEEP) {
            load_weights<TEAM>(w, a.weight, a.w32, a.w0, H, t);
            if (a.dres) load_rows<TEAM>(cr, a.dres, a.lddr, row, a.R, H, t);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float m = dot[u] / (float)H;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int col = (t + v * TEAM) * 8;
                float d[8], h[8], r[8];
                unpack8(cd[u][v], d);
                unpack8(ch[u][v], h);
                unpack8(cr[u][v], r);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[i] = __builtin_fmaf(__builtin_fmaf(-(h[i] * rstd[u]), m, d[i] * w[v][i]), rstd[u], r[i]);
                if (row[u] < a.R && col < H) store8(a.dx + row[u] * a.lddx + col, pack8(r), H - col);
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

// Calls f(team, vectors, rows at once) for rows of H elements: one vector a
// lane from 1024 to 8192 elements, where the registers leave room for rows at once
// and waves (us, 4096 x 2048: 64 lanes x 4 vectors x 2 rows 24.8, 256 x 1 x 4 19.1;
// 1111 x 8192: 256 x 4 x 2 35.7, 1024 x 1 x 2 25.3, four rows at once spill; 4096
// x 4096: 512 x 1 x 2 32.0, x 4 37.5, 256 x 2 x 2 33.1; 4096 x 5120: 256 x 3 x 2
// 43.4, 1024 x 1 x 2 43.5).  Shorter rows, with added gradients, in a captured graph:
// 500000 x 64: 8 x 1 x 4 53, x 2 55, 16 x 1 x 2 86; 500000 x 128: 16 x 1 x 4 97, x 2 101,
// 8 x 2 x 2 98; 100000 x 256: 16 x 2 x 2 44, x 1 45, 64 x 1 x 4 55; 32768 x 1024: 64 x 2 x 2
// 53.5, x 1 56, x 4 62.5, 256 x 1 x 4 74; 32768 x 512: 16 x 4 x 2, which takes 296 registers
// and leaves one wave a SIMD, 38, x 1 30.5, 64 x 1 x 4 30.  Rows past 16384 elements
// spill registers: 1024 x 32768 207, 1024 x 16384 40.
template <int N>
using Int = std::integral_constant<int, N>;
template <typename F>
auto with_grad_shape(int64_t H, F &&f)
{
    if (H <= 64) return f(Int<8>{}, Int<1>{}, Int<4>{});
    if (H <= 128) return f(Int<16>{}, Int<1>{}, Int<4>{});
    if (H <= 256) return f(Int<16>{}, Int<2>{}, Int<2>{});
    if (H <= 512) return f(Int<16>{}, Int<4>{}, Int<2>{});
    if (H <= 1024) return f(Int<64>{}, Int<2>{}, Int<2>{});
    if (H <= 2048) return f(Int<256>{}, Int<1>{}, Int<4>{});
    if (H <= 4096) return f(Int<512>{}, Int<1>{}, Int<2>{});
    if (H <= 8192) return f(Int<1024>{}, Int<1>{}, Int<2>{});
    if (H <= 16384) return f(Int<1024>{}, Int<2>{}, Int<1>{});
    return f(Int<1024>{}, Int<4>{}, Int<1>{});
}

}  // namespace

int64_t norm_grad_parts(int64_t R, int64_t H)
{
    const int64_t rows = with_grad_shape(H, [](auto team, auto, auto u) { return (team < 256 ? 256 / team : 1) * u; });
    const int64_t most = with_grad_shape(H, [](auto team, auto, auto) { return team < 1024 ? 512 : 256; });
    const int64_t n = (R + rows - 1) / rows;
    // one workgroup for up to four of its steps (1 us each; a second launch and
    // its workspace take 8), and for no rows, where it writes zeros
    return n <= 4 ? 1 : n < most ? n : most;
}

int64_t norm_grad_width(int64_t H)
{
    return with_grad_shape(H, [](auto team, auto v, auto) { return 8 * team * v; });
}

hipError_t launch_rms_norm(const NormArgs &a, hipStream_t s)
{
    const int64_t H = a.H;
    // Few lanes a row where rows are short; a lane's vectors side by side where
    // they are long, until a row's lanes stand in the way of other rows' loads
    // (us in a captured graph, a residual added, row scales / 128-element scales):
    //   44440 x 128   16 lanes, 4 rows at once 13.0 / 12.5, 2 12.6 / 12.2, 1 11.3 / 10.9
    //   500000 x 128  84.5 / 83.5, 84.5 / 82.6, 89.1 / 87.2
    //   4096 x 2048   64 x 4 vectors 14.4 / 14.3, 256 x 1 14.4 / 14.1
    //   4096 x 4096   256 x 2 26.5 / 27.2, 512 x 1 29.2 / 28.5, 1024 x 1 42.7 / 41.3
    //   4096 x 5120   256 x 3 32.6 / 34.0, 512 x 2 34.7 / 35.8, 1024 x 1 46.0 / 45.6
    //   4096 x 8192   256 x 4 47.7 / 49.6, 512 x 2 47.4 / 49.4, 1024 x 1 53.8 / 53.1
    // Few rows leave compute units idle, and one vector a lane has the shortest
    // way: 16 x 2048 64 x 4 4.8 / 5.1, 256 x 1 3.5 / 3.4 (1024 rows 6.2 / 6.4, 5.8 / 5.7;
    // 2048 rows 9.2 / 9.6, 10.0 / 9.8); 16 x 5120 256 x 3 4.6 / 4.6, 1024 x 1 4.3 / 4.1
    // (512 rows 6.8 / 7.0, 7.9 / 7.6); 16 x 8192 256 x 4 5.3 / 5.4, 1024 x 1 4.7 / 4.6.  Up to
    // 4096 elements half of those 1024 lanes hold nothing, and the way is no shorter:
    // 16 x 4096 256 x 2 4.1 / 4.1, 512 x 1 3.7 / 3.7, 1024 x 1 4.3 / 4.0.
    if (H <= 64 && a.output != SPG_NORM_E4M3_BLOCK128) return launch_team<8, 1, 4>(a, s);    // (a group is 16 lanes)
    if (H <= 128) return launch_team<16, 1, 2>(a, s);
    if (H <= 256) return launch_team<16, 2, 1>(a, s);
    if (H <= 512) return launch_team<16, 4, 1>(a, s);
    if (H <= 1024) return launch_team<64, 2, 1>(a, s);
    if (a.R <= 1024 && H <= 2048) return launch_team<256, 1, 1>(a, s);
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
