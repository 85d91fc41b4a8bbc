// Device helpers shared by the quantizer kernels: maxima of bf16 vectors and
// the E4M3 encode of a group of elements that share one fp32 scale.
#pragma once

#include "spg_common.h"

#include <type_traits>

namespace spg {
namespace quant {

constexpr int kThreads = 256;

// max(|bf16|) over the 8 values of a 16-byte vector, as a bit pattern.
__device__ __forceinline__ uint32_t amax8(const uint4 &v)
{
    uint32_t m = 0;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
        m = max(m, max(lo, hi));
    }
    return m;
}

// Division by a row's scale, made cheap.  The E4M3 code of fl32(x / s) is
// needed for every element; s = fl32(amax / 448) is fixed per row (per
// matrix for the per-tensor format).  Instead of an IEEE division per element:
//   xs = x k, ss = s k        (k = 2^100 when amax < 2^-40, else 1: exact)
//   r  = fl32(1 / ss)         (once per row)
//   q0 = fl32(xs r);  e = fma(-q0, ss, xs);  q = copysign(fma(e, r, q0), x)
// then q is clamped to [-448, 448] and converted with v_cvt_pk_fp8_f32
// (E4M3FN, round to nearest even).  q can differ from fl32(x / s) by an ulp
// only where the code cannot change; the scaling keeps the residual e from
// underflowing for tiny rows.  Checked exhaustively on the GPU against IEEE
// division followed by the reference RNE encoder: every positive finite bf16
// amax with every bf16 x, |x| <= amax, gives the same code (and the clamped
// conversion matches the reference encoder for every finite binary32).
// Rows whose scale is zero, infinite or NaN keep the exact slow path.
struct RowScale {
    float s, k, ss, r;
    bool fast;
};

__device__ __forceinline__ RowScale row_scale(float amax)
{
    RowScale t;
    t.s = amax / 448.0f;
    t.fast = t.s > 0.0f && t.s <= 3.40282347e38f;
    t.k = amax < 0x1p-40f ? 0x1p100f : 1.0f;
    t.ss = t.s * t.k;
    t.r = 1.0f / t.ss;
    return t;
}

// SCALED: the row needs the 2^100 scaling (k != 1); the common case skips
// the multiplications by k (exact either way: k = 1 makes them identities).
// The clamp is one v_med3_f32.
template <bool SCALED>
__device__ __forceinline__ float quot(float x, const RowScale &t)
{
    const float xs = SCALED ? x * t.k : x;
    const float q0 = xs * t.r;
    const float e = __builtin_fmaf(-q0, t.ss, xs);
    const float q = __builtin_copysignf(__builtin_fmaf(e, t.r, q0), x);
    return __builtin_amdgcn_fmed3f(q, -448.0f, 448.0f);
}

// Encode 8 bf16 values (one 16-byte vector) to 8 E4M3 codes.  MODE (the
// same for a whole row or matrix): 0 the exact slow path (zero, infinite or
// NaN scale: IEEE division or signed zeros), 1 the fast path, 2 the fast path
// with the 2^100 scaling of tiny rows.
template <int MODE>
__device__ __forceinline__ uint2 encode8_e4m3(const uint4 &v, const RowScale &t)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t out[2];
    if (MODE > 0) {
        constexpr bool SC = MODE == 2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int d = __builtin_amdgcn_cvt_pk_fp8_f32(quot<SC>(bf16_lo(w[2 * h]), t), quot<SC>(bf16_hi(w[2 * h]), t),
                                                    0, false);
            d = __builtin_amdgcn_cvt_pk_fp8_f32(quot<SC>(bf16_lo(w[2 * h + 1]), t),
                                                quot<SC>(bf16_hi(w[2 * h + 1]), t), d, true);
            out[h] = (uint32_t)d;
        }
    } else {
        const float s = t.s;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t c0, c1, c2, c3;
            if (s > 0.0f) {
                c0 = encode_e4m3(bf16_lo(w[2 * h]) / s);
                c1 = encode_e4m3(bf16_hi(w[2 * h]) / s);
                c2 = encode_e4m3(bf16_lo(w[2 * h + 1]) / s);
                c3 = encode_e4m3(bf16_hi(w[2 * h + 1]) / s);
            } else {   // zero scale: signed zeros
                c0 = (w[2 * h] >> 8) & 0x80u;
                c1 = (w[2 * h] >> 24) & 0x80u;
                c2 = (w[2 * h + 1] >> 8) & 0x80u;
                c3 = (w[2 * h + 1] >> 24) & 0x80u;
            }
            out[h] = c0 | (c1 << 8) | (c2 << 16) | (c3 << 24);
        }
    }
    return make_uint2(out[0], out[1]);
}

// Calls f(std::integral_constant<int, MODE>) with the encode mode of scale t.
template <typename F>
__device__ __forceinline__ void with_encode_mode(const RowScale &t, F &&f)
{
    if (!t.fast)
        f(std::integral_constant<int, 0>{});
    else if (t.k == 1.0f)
        f(std::integral_constant<int, 1>{});
    else
        f(std::integral_constant<int, 2>{});
}

// Block-wide max of a per-thread value (256 threads = 4 waves).
__device__ __forceinline__ uint32_t block_max_u32(uint32_t v, uint32_t *lds4)
{
    v = wave_max_u32(v);
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) lds4[wave] = v;
    __syncthreads();
    uint32_t r = max(max(lds4[0], lds4[1]), max(lds4[2], lds4[3]));
    __syncthreads();
    return r;
}

__device__ __forceinline__ uint4 ld16(const uint16_t *p) { return *reinterpret_cast<const uint4 *>(p); }

}  // namespace quant
}  // namespace spg
