// Routing of tokens to experts, the row order of the experts' products, and
// the weighted sum of their rows.
//
// Routing.  For a token with logits l (E of them):
//   p_e = softmax(l)_e or 1 / (1 + exp(-l_e)),  c_e = p_e + bias_e
//   groups of E / groups consecutive experts: a group's score is the sum of
//   its two largest c; only the top_groups best groups stay
//   experts = the top largest c, ties to the lowest index
//   w_j = scale p_j / sum_i p_i, or scale p_j
// Experts next to the border of the top must not depend on how an exp is
// rounded, so p and c are computed and compared in 64 bits; without bias and
// groups the scores are increasing in l and the logits themselves are
// compared.  A logit (or c) of -inf masks its expert: it is never chosen, and
// slots that no expert is left for get expert -1 and weight 0.  A NaN logit
// is not chosen either and makes its token's weights NaN.
//
// A team of 64 or 16 lanes works on one token; lane l holds the EPL
// consecutive experts l EPL ...  Each of the `top` rounds takes the team's
// maximum through DPP row operations - of 32-bit keys where the logits are
// compared, of the high words of 64-bit keys and, where several experts share
// it, their low words - and drops the lowest expert that holds it.  No LDS and
// no divergent code in the rounds: 8 rounds over 256 experts are about 350
// instructions with 64 lanes (4 keys each) and 800 for four tokens at once
// with 16 (16 keys each).  Few tokens are bound by one wave's latency and take
// 64 lanes; many by issue and take 16.
//
// Measured on the GPU: 16 tokens of 256 experts (8 groups, biased sigmoid) 8.6
// us and 4.0 us for their row order, both one wave's latency; 8192 tokens of
// 128 experts (softmax, bf16) 6.1 us, 7.4 and, for the gradient, 6.5.
#include "spg_experts.h"
#include "spg_gemm_common.h"

#include <type_traits>

namespace spg {

namespace {

constexpr int kThreads = 256;

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
}
// the four exchanges that make a value uniform over a row of 16 lanes: with
// every combine symmetric, all lanes end with the same bits
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
// lane 15 of a row into the next row; lane 31 into rows 2 and 3
constexpr int kBcast15 = 0x142, kBcast31 = 0x143;

// The maximum over the team, in every lane (all lanes active: row operations
// read their neighbours).  64 lanes: each row's maximum travels through rows
// 1, 2, 3 to lane 63.
template <int TEAM>
__device__ __forceinline__ uint32_t team_max(uint32_t v)
{
    v = max(v, dpp<kXor1>(v));
    v = max(v, dpp<kXor2>(v));
    v = max(v, dpp<kHalfMirror>(v));
    v = max(v, dpp<kMirror>(v));
    if (TEAM == 64) {
        v = max(v, dpp<kBcast15>(v));
        v = max(v, dpp<kBcast31>(v));
        v = (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
    }
    return v;
}

template <int CTRL>
__device__ __forceinline__ double dpp64(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double((long long)((uint64_t)dpp<CTRL>((uint32_t)(b >> 32)) << 32 | dpp<CTRL>((uint32_t)b)));
}
template <int TEAM>
__device__ __forceinline__ double team_sum(double v)
{
    v += dpp64<kXor1>(v);
    v += dpp64<kXor2>(v);
    v += dpp64<kHalfMirror>(v);
    v += dpp64<kMirror>(v);
    if (TEAM == 64) {
        v += __shfl_xor(v, 16, 64);
        v += __shfl_xor(v, 32, 64);
    }
    return v;
}
template <int TEAM>
__device__ __forceinline__ float team_sum(float v)
{
    v += __uint_as_float(dpp<kXor1>(__float_as_uint(v)));
    v += __uint_as_float(dpp<kXor2>(__float_as_uint(v)));
    v += __uint_as_float(dpp<kHalfMirror>(__float_as_uint(v)));
    v += __uint_as_float(dpp<kMirror>(__float_as_uint(v)));
    if (TEAM == 64) {
        v += __shfl_xor(v, 16, 64);
        v += __shfl_xor(v, 32, 64);
    }
    return v;
}

// This team's lanes of a ballot, lane 0 of the team in bit 0.
template <int TEAM>
__device__ __forceinline__ uint64_t team_ballot(bool x)
{
    const uint64_t b = __ballot(x);
    if (TEAM == 64) return b;
    const int lane = threadIdx.x & 63;
    return (b >> (lane & ~(TEAM - 1))) & ((1ull << (TEAM & 63)) - 1);
}

// Keys: unsigned integers in the order of the values; 0 for what is never
// chosen (-inf and NaN).
__device__ __forceinline__ uint32_t key32(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f);      // -0 counts as +0
    const uint32_t k = (u >> 31) ? ~u : u | 0x80000000u;
    return v > -INFINITY ? k : 0u;                     // false for NaN
}
__device__ __forceinline__ uint64_t key64(double v)
{
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    const uint64_t k = (u >> 63) ? ~u : u | (1ull << 63);
    return v > -(double)INFINITY ? k : 0ull;
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const RouteArgs &a, int64_t t, int e)
{
    if (BF16) return __uint_as_float((uint32_t)((const uint16_t *)a.logits)[t * a.ld + e] << 16);
    return ((const float *)a.logits)[t * a.ld + e];
}

// The EPL logits from expert e0 on (-inf past the last expert): 16 bytes a
// load where rows are 16-byte aligned (a.vec) and the lane's all exist.
template <int EPL, bool BF16>
__device__ __forceinline__ void load_logits(const RouteArgs &a, int64_t t, bool live, int e0, float (&l)[EPL])
{
    constexpr int kPer = BF16 ? 8 : 4;
    if (EPL % kPer == 0 && a.vec && live && e0 + EPL <= a.E) {
#pragma unroll
        for (int v = 0; v < EPL / kPer; ++v) {
            const uint4 q = BF16 ? *reinterpret_cast<const uint4 *>((const uint16_t *)a.logits + t * a.ld + e0 + v * kPer)
                                 : *reinterpret_cast<const uint4 *>((const float *)a.logits + t * a.ld + e0 + v * kPer);
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (BF16) {
                    l[(v * kPer + 2 * i) % EPL] = bf16_lo(w[i]);
                    l[(v * kPer + 2 * i + 1) % EPL] = bf16_hi(w[i]);
                } else {
                    l[(v * kPer + i) % EPL] = __uint_as_float(w[i]);
                }
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = live && e0 + i < a.E ? load_logit<BF16>(a, t, e0 + i) : -INFINITY;
}

// Orders this wave's LDS accesses before and after (teams never span waves).
__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The two largest of (a1 >= a2) and (b1 >= b2).
__device__ __forceinline__ void merge2(double &a1, double &a2, double b1, double b2)
{
    const double lo = a1 < b1 ? a1 : b1, hi2 = a2 < b2 ? b2 : a2;
    a1 = a1 < b1 ? b1 : a1;
    a2 = lo < hi2 ? hi2 : lo;
}

// Which of this lane's experts' groups stay: bit i for expert tl EPL + i.
// c: its choices (-inf where never chosen).  scores: LDS of the token, one
// double per group; all: LDS of the token, one per expert.
template <int TEAM, int EPL>
__device__ __forceinline__ uint32_t kept_experts(const RouteArgs &a, const double (&c)[EPL], volatile double *scores,
                                                 volatile double *all)
{
    const int tl = threadIdx.x & (TEAM - 1), size = a.E / a.groups;
    const double none = -(double)INFINITY;
    auto rank = [&](int g, double v) {                    // groups before g
        int better = 0;
        for (int h = 0; h < a.groups; ++h) {
            const double o = scores[h];
            better += (o > v || (o == v && h < g)) ? 1 : 0;
        }
        return better;
    };
    const int lanes = size / EPL;
    if (size % EPL == 0 && (lanes & (lanes - 1)) == 0 && lanes <= TEAM) {
        // a group is a power of two of whole lanes: two largest in the lane,
        // then over the group's lanes
        double m1 = none, m2 = none;
#pragma unroll
        for (int i = 0; i < EPL; ++i) merge2(m1, m2, c[i], none);
        auto step = [&](auto ctrl) { merge2(m1, m2, dpp64<decltype(ctrl)::value>(m1), dpp64<decltype(ctrl)::value>(m2)); };
        if (lanes > 1) step(std::integral_constant<int, kXor1>{});
        if (lanes > 2) step(std::integral_constant<int, kXor2>{});
        if (lanes > 4) step(std::integral_constant<int, kHalfMirror>{});
        if (lanes > 8) step(std::integral_constant<int, kMirror>{});
        if (lanes > 16) merge2(m1, m2, __shfl_xor(m1, 16, 64), __shfl_xor(m2, 16, 64));
        if (lanes > 32) merge2(m1, m2, __shfl_xor(m1, 32, 64), __shfl_xor(m2, 32, 64));
        const int g = tl / lanes;
        const double v = m2 > none ? m1 + m2 : m1;
        if (tl % lanes == 0 && g < a.groups) scores[g] = v;
        wave_sync();
        return g < a.groups && v > none && rank(g, v) < a.top_groups ? ~0u : 0u;
    }
    // groups that cut across lanes: the choices through LDS
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (tl * EPL + i < a.E) all[tl * EPL + i] = c[i];
    wave_sync();
    for (int g = tl; g < a.groups; g += TEAM) {
        double m1 = none, m2 = none;
        for (int i = 0; i < size; ++i) merge2(m1, m2, all[g * size + i], none);
        scores[g] = m2 > none ? m1 + m2 : m1;
    }
    wave_sync();
    uint32_t keep = 0;
    int last = -1;
    bool in = false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = tl * EPL + i;
        if (e >= a.E) continue;
        const int g = (int)fdiv_q((uint32_t)e, a.div_group);
        if (g != last) {
            const double v = scores[g];
            in = v > none && rank(g, v) < a.top_groups;
            last = g;
        }
        keep |= in ? 1u << i : 0u;
    }
    return keep;
}

// Routes token t (live: it exists) with this team; lanes j < top return weight
// and expert of place j.  scores, all: the team's LDS (GROUPS only).
template <int TEAM, int EPL, bool BF16, bool PLAIN>
__device__ __forceinline__ void route_token(const RouteArgs &a, int64_t t, bool live, volatile double *scores,
                                            volatile double *all, float &w_out, int32_t &e_out)
{
#pragma clang fp contract(off)
    const int tl = threadIdx.x & (TEAM - 1);
    float l[EPL];
    float mx = -INFINITY;
    bool nan = false;
    load_logits<EPL, BF16>(a, t, live, tl * EPL, l);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        nan = nan || l[i] != l[i];
        mx = l[i] > mx ? l[i] : mx;
    }
    nan = team_ballot<TEAM>(nan) != 0;
    auto largest = [](float v) {                          // over the team, through the keys
        const uint32_t k = team_max<TEAM>(key32(v));
        return k == 0u ? -INFINITY : __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
    };
    mx = largest(mx);
    const bool soft = a.score == SPG_SCORE_SOFTMAX;
    // score of a logit before the softmax's division; an infinite maximum
    // counts as the only size that matters (1 for it, 0 for the others)
    auto raw = [&](float v) -> double {
        if (!(v > -INFINITY)) return 0.0;
        const double x = soft ? (v == mx ? 0.0 : (double)v - (double)mx) : -(double)v;
        const double y = exp(x);
        return soft ? y : 1.0 / (1.0 + y);
    };
    double z = 1.0;
    uint32_t hi[EPL], lo[PLAIN ? 1 : EPL];
    if (PLAIN) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) hi[i] = key32(l[i]);
        if (soft && !a.renorm) {
            double part = 0.0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) part += raw(l[i]);
            z = team_sum<TEAM>(part);
        }
    } else {
        double c[EPL], part = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            c[i] = raw(l[i]);
            part += c[i];
        }
        if (soft) z = team_sum<TEAM>(part);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = tl * EPL + i;
            if (soft) c[i] = c[i] / z;
            if (a.bias && e < a.E) c[i] = c[i] + (double)a.bias[e];
            if (!(l[i] > -INFINITY && c[i] > -(double)INFINITY)) c[i] = -(double)INFINITY;
        }
        const uint32_t keep = a.groups > 1 ? kept_experts<TEAM, EPL>(a, c, scores, all) : ~0u;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const uint64_t k = (keep >> i) & 1u ? key64(c[i]) : 0ull;
            hi[i] = (uint32_t)(k >> 32);
            lo[PLAIN ? 0 : i] = (uint32_t)k;
        }
    }
    // the rounds; a key of 0 (its high word is 0 for nothing else) is never chosen
    int32_t my_e = -1;
    for (int j = 0; j < a.top; ++j) {
        uint32_t m = hi[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) m = max(m, hi[i]);
        m = team_max<TEAM>(m);
        uint32_t mlo = 0;
        bool ties = false;
        if (!PLAIN) {
            int same = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) same += hi[i] == m ? 1 : 0;
            const uint64_t who = team_ballot<TEAM>(same > 0);
            // several experts with this high word in any team of the wave
            ties = __any(m != 0u && ((who & (who - 1)) != 0 || same > 1)) != 0;
            if (ties) {
#pragma unroll
                for (int i = 0; i < EPL; ++i) mlo = max(mlo, hi[i] == m ? lo[i] : 0u);
                mlo = team_max<TEAM>(mlo);
            }
        }
        // the lowest expert that holds the maximum, as the largest ~e
        uint32_t ne = 0;
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i)
            ne = hi[i] == m && (PLAIN || !ties || lo[PLAIN ? 0 : i] == mlo) ? ~(uint32_t)(tl * EPL + i) : ne;
        ne = team_max<TEAM>(m != 0u ? ne : 0u);
        const int32_t e = ne ? (int32_t)~ne : -1;
#pragma unroll
        for (int i = 0; i < EPL; ++i) hi[i] = tl * EPL + i == e ? 0u : hi[i];
        my_e = tl == j ? e : my_e;
    }
    const bool there = live && my_e >= 0;
    const float chosen = there ? load_logit<BF16>(a, t, my_e) : -INFINITY;
    double p = there ? raw(chosen) : 0.0;
    if (a.renorm && __any(there && p < 0x1p-860)) {
        // scores (below e^-596) from which 64 bits lose digits or everything -
        // a bias or a group can choose experts far below the largest logit:
        // shares relative to the largest chosen one.  Sigmoids that are all 0
        // in 64 bits stay 0.
        const float mc = largest(chosen);
        const bool far = soft ? (double)mc - (double)mx < -600.0 : mc < -600.0f && mc > -709.7827f;
        if (there && far) p = exp((double)chosen - (double)mc);
    }
    if (soft && !a.renorm) p = z > 0.0 ? p / z : 0.0;
    const double total = a.renorm ? team_sum<TEAM>(p) : 1.0;
    double w = total > 0.0 ? (double)a.scale * (p / total) : 0.0;
    if (nan) w = __longlong_as_double(0x7FF8000000000000ll);
    w_out = (float)w;
    e_out = my_e;
}

// ---- row order -------------------------------------------------------------

// Lanes of the wave holding the same expert as this lane (valid lanes only).
__device__ __forceinline__ uint64_t match_expert(int32_t e, bool valid, int bits)
{
    uint64_t m = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
        const uint64_t s = __ballot((e >> b) & 1);
        m &= ((e >> b) & 1) ? s : ~s;
    }
    return m;
}

constexpr int kOrderThreads = 1024, kOrderWaves = kOrderThreads / 64;
constexpr int kRouteThreads = 512;

// The row order of the n = T top entries of a.experts (flat, token-major), of
// which workgroup `part` of `parts` places its own: rows of an expert are
// ordered by entry.  The entries of an expert before and after the part come
// from the counts of chunks of a.chunk tokens (a.hist, written by the launch
// before), or, for few entries, every workgroup counts all of them in LDS
// itself: n / 1024 additions a thread, which collide where experts repeat.
// Measured behind the route launch (us): 8192 entries 7.2 counted here, 8.2
// from chunk counts; 65536 entries 21.7 and 8.2.
__global__ __launch_bounds__(kOrderThreads) void order_kernel(const RouteArgs a)
{
    extern __shared__ int32_t cnt[];                      // [kOrderWaves][E]
    __shared__ int32_t before[kRouteMaxExperts], after[kRouteMaxExperts];
    __shared__ int32_t wsum[kOrderWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = a.E;
    const int bits = 32 - __builtin_clz((unsigned)E);
    const int32_t *experts = a.experts;
    const int part = blockIdx.x, parts = gridDim.x;
    const int64_t n = a.T * a.top;
    int64_t n0, n1;
    int c0 = 0, c1 = 0;                                   // this part's chunks
    if (a.hist) {
        const int per = (a.chunks + parts - 1) / parts;
        c0 = min(a.chunks, part * per);
        c1 = min(a.chunks, c0 + per);
        n0 = min(n, (int64_t)c0 * a.chunk * a.top);
        n1 = min(n, (int64_t)c1 * a.chunk * a.top);
    } else {
        const int64_t step = (n + parts - 1) / parts;
        n0 = min(n, part * step);
        n1 = min(n, n0 + step);
    }
    const int64_t per = ((n1 - n0 + kOrderWaves - 1) / kOrderWaves + 63) / 64 * 64;
    const int64_t w0 = min(n1, n0 + wave * per), w1 = min(n1, w0 + per);
    for (int i = tid; i < kOrderWaves * E; i += kOrderThreads) cnt[i] = 0;
    for (int e = tid; e < E; e += kOrderThreads) before[e] = after[e] = 0;
    __syncthreads();
    int32_t *mine = cnt + wave * E;
    for (int64_t i = w0 + lane; i < w1; i += 64) {
        const int32_t e = experts[i];
        if ((uint32_t)e < (uint32_t)E) atomicAdd(&mine[e], 1);
    }
    if (a.hist) {
        // threads q, q + E', q + 2 E' ... (E' = E rounded up to a power of
        // two) share expert q's chunks
        const int e2 = 1 << (E > 1 ? 32 - __builtin_clz((unsigned)(E - 1)) : 0);
        const int e = tid & (e2 - 1), first = tid / e2, step = kOrderThreads / e2;
        if (e < E) {
            int32_t b = 0, f = 0;
#pragma unroll 8
            for (int c = first; c < a.chunks; c += step) {
                const int32_t v = a.hist[(int64_t)c * E + e];
                b += c < c0 ? v : 0;
                f += c >= c1 ? v : 0;
            }
            if (b) atomicAdd(&before[e], b);
            if (f) atomicAdd(&after[e], f);
        }
    } else {
        for (int64_t i = tid; i < n0; i += kOrderThreads) {
            const int32_t e = experts[i];
            if ((uint32_t)e < (uint32_t)E) atomicAdd(&before[e], 1);
        }
        for (int64_t i = n1 + tid; i < n; i += kOrderThreads) {
            const int32_t e = experts[i];
            if ((uint32_t)e < (uint32_t)E) atomicAdd(&after[e], 1);
        }
    }
    __syncthreads();
    // rows of experts below e: a scan over the experts (one per thread)
    int32_t own = 0, all = 0;
    if (tid < E) {
#pragma unroll
        for (int w = 0; w < kOrderWaves; ++w) own += cnt[w * E + tid];
        all = before[tid] + own + after[tid];
    }
    int32_t sum = all;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int32_t o = __shfl_up(sum, off, 64);
        if (lane >= off) sum += o;
    }
    if (lane == 63) wsum[wave] = sum;
    __syncthreads();
    int32_t at = sum - all, total = 0;
#pragma unroll
    for (int w = 0; w < kOrderWaves; ++w) {
        at += w < wave ? wsum[w] : 0;
        total += wsum[w];
    }
    if (tid < E) {
        if (part == 0) a.offsets[tid] = at;
        int32_t pos = at + before[tid];
#pragma unroll
        for (int w = 0; w < kOrderWaves; ++w) {           // where each wave's first entry goes
            const int32_t c = cnt[w * E + tid];
            cnt[w * E + tid] = pos;
            pos += c;
        }
    }
    if (part == 0) {
        if (tid == 0) a.offsets[E] = total;
        for (int64_t i = total + tid; i < n; i += kOrderThreads) a.rows[i] = -1;
    }
    __syncthreads();
    volatile int32_t *next = mine;                        // read and written by lanes of this wave
    for (int64_t i0 = w0; i0 < w1; i0 += 64) {
        const int64_t i = i0 + lane;
        const int32_t e = i < w1 ? experts[i] : -1;
        const bool valid = (uint32_t)e < (uint32_t)E;
        const uint64_t same = match_expert(e, valid, bits);
        int32_t pos = -1;
        if (valid) {
            pos = next[e] + __popcll(same & ((1ull << lane) - 1));
            a.rows[pos] = (int32_t)fdiv_q((uint32_t)i, a.div_top);
        }
        wave_sync();
        if (valid && (same >> lane) == 1ull) next[e] = pos + 1;      // the last lane of its expert
        wave_sync();
        if (i < w1) a.slots[i] = pos;
    }
}

// One team per token; a workgroup takes a chunk of a.chunk tokens (with
// a.hist it counts its experts), else as many as it has teams.
template <int TEAM, int EPL, bool BF16, bool PLAIN>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const RouteArgs a)
{
    constexpr int TOK = kRouteThreads / TEAM;
    extern __shared__ double lds_dyn[];                   // groups: scores [TOK][groups], choices [TOK][E]
    __shared__ int32_t lds_h[kRouteMaxExperts];
    const int tid = threadIdx.x, team = tid / TEAM, tl = tid & (TEAM - 1);
    const int64_t t0 = (int64_t)blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
    if (a.hist) {
        for (int e = tid; e < a.E; e += kRouteThreads) lds_h[e] = 0;
        __syncthreads();
    }
    for (int64_t tb = t0; tb < t1; tb += TOK) {
        const int64_t t = tb + team;
        float w;
        int32_t e;
        route_token<TEAM, EPL, BF16, PLAIN>(a, t, t < t1, lds_dyn + team * a.groups,
                                            lds_dyn + TOK * a.groups + (int64_t)team * a.E, w, e);
        if (t < t1 && tl < a.top) {
            a.weights[t * a.top + tl] = w;
            a.experts[t * a.top + tl] = e;
            if (a.hist && e >= 0) atomicAdd(&lds_h[e], 1);
        }
    }
    if (a.hist) {
        __syncthreads();
        for (int e = tid; e < a.E; e += kRouteThreads) a.hist[(int64_t)blockIdx.x * a.E + e] = lds_h[e];
    }
}

// The experts of each chunk of tokens counted (for experts chosen elsewhere).
__global__ __launch_bounds__(kRouteThreads) void count_kernel(const RouteArgs a)
{
    __shared__ int32_t lds_h[kRouteMaxExperts];
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) lds_h[e] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
    for (int64_t i = t0 * a.top + threadIdx.x; i < t1 * a.top; i += kRouteThreads) {
        const int32_t e = a.experts[i];
        if ((uint32_t)e < (uint32_t)a.E) atomicAdd(&lds_h[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kRouteThreads) a.hist[(int64_t)blockIdx.x * a.E + e] = lds_h[e];
}

// ---- gradient of the logits --------------------------------------------------
// With q_j the chosen scores' shares:
//   renormalised:  d/dl of scale q_j; softmax over the chosen (the softmax's
//                  own sum cancels): dl_j = scale q_j (g_j - sum g q)
//                  sigmoid: dl_j = scale q_j (1 - p_j) (g_j - sum g q)
//   else softmax:  dl_e = p_e ([e chosen] scale g - sum scale g p)
//   else sigmoid:  dl_j = scale g_j p_j (1 - p_j)
// One wave per token: lane j < top works out choice j, then the wave writes
// the dense row (NaN where a logit of the token is).  An expert that stands
// twice in a row gets both parts.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(const RouteArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    if (t >= a.T) return;
    const bool soft = a.score == SPG_SCORE_SOFTMAX;
    // on their way while the experts and then their logits are
    const float first = load_logit<BF16>(a, t, min(lane, a.E - 1)), second = load_logit<BF16>(a, t, min(lane + 64, a.E - 1));
    int32_t e = lane < a.top ? a.experts[t * a.top + lane] : -1;
    if ((uint32_t)e >= (uint32_t)a.E) e = -1;
    const float g = e >= 0 ? a.grad[t * a.top + lane] * a.scale : 0.0f;
    const float l = e >= 0 ? load_logit<BF16>(a, t, e) : -INFINITY;
    float mine = 0.0f, common = 0.0f, mx = -INFINITY, rz = 0.0f;
    const bool dense = soft && !a.renorm;
    // a NaN logit, chosen or not, makes its token's weights NaN: and so its gradient
    bool nan = first != first || second != second;
    if (dense) mx = fmaxf(first, second);
    for (int i0 = 128; i0 < a.E; i0 += 64) {
        const float v = load_logit<BF16>(a, t, min(i0 + lane, a.E - 1));
        nan = nan || v != v;
        if (dense) mx = fmaxf(mx, v);
    }
    const float zero = __any(nan) ? __uint_as_float(0x7FC00000u) : 0.0f;
    if (!dense) mx = l;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off, 64));
    auto ex = [&](float v) { return v == mx ? 1.0f : expf(v - mx); };
    if (soft) {
        float z = 0.0f;
        if (dense) {
            for (int i = lane; i < a.E; i += 64) z += ex(load_logit<BF16>(a, t, i));
        } else if (e >= 0) {
            z = ex(l);
        }
        z = team_sum<64>(z);
        rz = z > 0.0f ? 1.0f / z : 0.0f;
        const float q = e >= 0 ? ex(l) * rz : 0.0f;
        const float dot = team_sum<64>(g * q);
        if (dense) {
            mine = g * q;
            common = dot;
        } else {
            mine = q * (g - dot);
        }
    } else if (a.renorm) {
        // p = exp(min(l, 0)) / (1 + exp(-|l|)), taken relative to the largest
        // chosen score where all are small: in 32 bits p is 0 below logits of
        // -88 and 1 / sum p overflows, though the shares are ordinary numbers.
        // (64-bit shares instead: 8192 tokens of 128 experts 6.8 us, 5.9 so.)
        // Where exp(-l) overflows 64 bits the weights are 0, and so is this.
        const bool some = mx > -709.7827f;
        const float t = expf(-fabsf(l));
        const float u = some && e >= 0 ? expf(fminf(l, 0.0f) - fminf(mx, 0.0f)) / (1.0f + t) : 0.0f;
        const float z = team_sum<64>(u), q = z > 0.0f ? u / z : 0.0f;
        const float dot = team_sum<64>(g * q);
        mine = q * ((l < 0.0f ? 1.0f : t) / (1.0f + t)) * (g - dot);
    } else {
        // 1 - p as the sigmoid of -l: exact where p rounds to 1
        const float p = e >= 0 ? 1.0f / (1.0f + expf(-l)) : 0.0f, n = e >= 0 ? 1.0f / (1.0f + expf(l)) : 0.0f;
        mine = g * p * n;
    }
    // four columns per lane, every choice compared with each
    const bool vec = a.E % 4 == 0 && ((uintptr_t)a.grad_logits & (BF16 ? 7u : 15u)) == 0;
    for (int i0 = 0; i0 < a.E; i0 += 256) {
        const int i = i0 + 4 * lane;
        float v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            v[c] = dense && i + c < a.E ? -ex(load_logit<BF16>(a, t, i + c)) * rz * common + zero : zero;
        for (int j = 0; j < a.top; ++j) {
            const int32_t ej = __builtin_amdgcn_readlane(e, j) - i;
            const float mj = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(mine), j));
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] += ej == c ? mj : 0.0f;
        }
        if (i >= a.E) continue;
        const int64_t at = t * a.E + i;
        if (BF16) {
            uint16_t *o = (uint16_t *)a.grad_logits + at;
            if (vec) {
                *reinterpret_cast<uint2 *>(o) = make_uint2(gemm::pack_bf16x2(v[0], v[1]), gemm::pack_bf16x2(v[2], v[3]));
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (i + c < a.E) o[c] = (uint16_t)f32_to_bf16(v[c]);
            }
        } else {
            float *o = (float *)a.grad_logits + at;
            if (vec) {
                *reinterpret_cast<v4f *>(o) = v4f{v[0], v[1], v[2], v[3]};
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (i + c < a.E) o[c] = v[c];
            }
        }
    }
}

// ---- combine -----------------------------------------------------------------
// out[t] = residual[t] + sum_j w[t, j] y[slot[t, j]], fp32 sums in the order
// of j, one rounding.  A stream over the chosen rows: one workgroup per token
// and 2048 columns, 16 bytes per lane and row, up to eight rows in flight.
// VEC: every pointer and row stride is 16-byte aligned and H % 8 == 0; else
// one element per lane.  4096 x 8 rows of 2048: 28.5 us (5.9 TB/s), the
// gradients 50 us (5.7 TB/s).

// 16 bytes of an expert's row, read once: non-temporal, so that the rows do
// not push each other through the caches (4096 tokens x 6 rows of 7168: 95 us
// with ordinary loads and stores of rows and outputs, 77 us; with the residual
// read so too 86 us.  The backward pass measured the other way: 4096 x 8 rows
// of 2048 50 us, 60 us with non-temporal stores).
__device__ __forceinline__ uint4 once(const uint16_t *p)
{
    const v4i t = __builtin_nontemporal_load(reinterpret_cast<const v4i *>(p));
    return make_uint4((uint32_t)t[0], (uint32_t)t[1], (uint32_t)t[2], (uint32_t)t[3]);
}

template <bool VEC>
__global__ __launch_bounds__(kThreads) void combine_kernel(const CombineArgs a)
{
    constexpr int W = VEC ? 8 : 1;
    const int64_t t = blockIdx.x;
    const int64_t col = ((int64_t)blockIdx.y * kThreads + threadIdx.x) * W;
    if (col >= a.H) return;
    float s[W];
    if (VEC) {
        uint4 r = make_uint4(0, 0, 0, 0);
        if (a.residual) r = *reinterpret_cast<const uint4 *>(a.residual + t * a.ldr + col);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < W; ++i) s[i] = (i & 1) ? bf16_hi(w[(i >> 1) & 3]) : bf16_lo(w[(i >> 1) & 3]);
    } else {
        s[0] = a.residual ? bf16_lo(a.residual[t * a.ldr + col]) : 0.0f;
    }
    const int32_t *slots = a.slots + t * a.top;
    const float *wt = a.weights + t * a.top;
    for (int j0 = 0; j0 < a.top; j0 += 8) {
        uint4 v[8];
        uint16_t h[8];
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool in = j0 + j < a.top;
            const int32_t slot = in ? slots[j0 + j] : -1;
            const bool ok = slot >= 0 && (int64_t)slot < a.R;
            f[j] = ok ? wt[j0 + j] : 0.0f;
            v[j] = make_uint4(0, 0, 0, 0);
            h[j] = 0;
            if (ok) {
                const uint16_t *p = a.y + (int64_t)slot * a.ldy + col;
                if (VEC)
                    v[j] = once(p);
                else
                    h[j] = *p;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (VEC) {
                const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                for (int i = 0; i < W; ++i)
                    s[i] = __builtin_fmaf(f[j], (i & 1) ? bf16_hi(w[(i >> 1) & 3]) : bf16_lo(w[(i >> 1) & 3]), s[i]);
            } else {
                s[0] = __builtin_fmaf(f[j], bf16_lo(h[j]), s[0]);
            }
        }
    }
    uint16_t *o = a.out + t * a.ldo + col;
    if (VEC) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = gemm::pack_bf16x2(s[(2 * i) % W], s[(2 * i + 1) % W]);
        __builtin_nontemporal_store(v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]}, reinterpret_cast<v4i *>(o));
    } else {
        *o = (uint16_t)f32_to_bf16(s[0]);
    }
}

// grad_y[slot[t, j]] = w[t, j] g[t], grad_w[t, j] = <g[t], y[slot[t, j]]>:
// one workgroup per token, eight choices at a time, so g is read once per
// eight rows; the dots are summed in fp32 per lane, then over the workgroup
// in a fixed order.
template <bool VEC>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(const CombineArgs a)
{
    constexpr int W = VEC ? 8 : 1;
    __shared__ float lds_d[kThreads / 64][8];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int32_t *slots = a.slots + t * a.top;
    const float *wt = a.weights + t * a.top;
    for (int j0 = 0; j0 < a.top; j0 += 8) {
        float d[8];
        int64_t row[8];
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int32_t slot = j0 + j < a.top ? slots[j0 + j] : -1;
            const bool ok = slot >= 0 && (int64_t)slot < a.R;
            row[j] = ok ? (int64_t)slot : -1;
            f[j] = ok ? wt[j0 + j] : 0.0f;
            d[j] = 0.0f;
        }
        for (int64_t col = (int64_t)tid * W; col < a.H; col += kThreads * W) {
            float g[W];
            if (VEC) {
                const uint4 r = *reinterpret_cast<const uint4 *>(a.grad + t * a.ldr + col);
                const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                for (int i = 0; i < W; ++i) g[i] = (i & 1) ? bf16_hi(w[(i >> 1) & 3]) : bf16_lo(w[(i >> 1) & 3]);
            } else {
                g[0] = bf16_lo(a.grad[t * a.ldr + col]);
            }
            uint4 v[8];
            uint16_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = make_uint4(0, 0, 0, 0);
                h[j] = 0;
                if (row[j] >= 0) {
                    const uint16_t *p = a.y + row[j] * a.ldy + col;
                    if (VEC)
                        v[j] = *reinterpret_cast<const uint4 *>(p);
                    else
                        h[j] = *p;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (row[j] < 0) continue;
                uint16_t *o = a.out + row[j] * a.ldo + col;
                if (VEC) {
                    const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
                    uint32_t q[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        d[j] = __builtin_fmaf(g[(2 * i) % W], bf16_lo(w[i]), d[j]);
                        d[j] = __builtin_fmaf(g[(2 * i + 1) % W], bf16_hi(w[i]), d[j]);
                        q[i] = gemm::pack_bf16x2(f[j] * g[(2 * i) % W], f[j] * g[(2 * i + 1) % W]);
                    }
                    *reinterpret_cast<uint4 *>(o) = make_uint4(q[0], q[1], q[2], q[3]);
                } else {
                    d[j] = __builtin_fmaf(g[0], bf16_lo(h[j]), d[j]);
                    *o = (uint16_t)f32_to_bf16(f[j] * g[0]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = team_sum<64>(d[j]);
            if (lane == 0) lds_d[wave][j] = s;
        }
        __syncthreads();
        if (tid < 8 && j0 + tid < a.top) {
            float s = 0.0f;
            for (int w = 0; w < kThreads / 64; ++w) s += lds_d[w][tid];
            a.grad_weights[t * a.top + j0 + tid] = s;
        }
        __syncthreads();
    }
}

hipError_t launch_order(const RouteArgs &a, hipStream_t s)
{
    // parts of at least 1024 entries (one step of every wave), at most 64,
    // and with chunk counts at most one per chunk
    int64_t parts = (a.T * a.top + 1023) / 1024;
    parts = parts < 1 ? 1 : parts > 64 ? 64 : parts;
    if (a.hist && parts > a.chunks) parts = a.chunks;
    order_kernel<<<(unsigned)parts, kOrderThreads, (size_t)kOrderWaves * a.E * sizeof(int32_t), s>>>(a);
    return hipGetLastError();
}

template <int TEAM, int EPL, bool BF16, bool PLAIN>
hipError_t launch_route(const RouteArgs &in, hipStream_t s)
{
    constexpr int TOK = kRouteThreads / TEAM;
    RouteArgs a = in;
    if (a.hist == nullptr) {
        a.chunk = TOK;
        a.chunks = (int32_t)((a.T + TOK - 1) / TOK);
    }
    if (a.T > 0) {
        const size_t choices = a.groups > 1 ? (size_t)TOK * (a.groups + a.E) * sizeof(double) : 0;
        route_kernel<TEAM, EPL, BF16, PLAIN><<<(unsigned)a.chunks, kRouteThreads, choices, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return a.offsets != nullptr ? launch_order(a, s) : hipSuccess;
}

// 64 lanes a token up to kRouteWide tokens (four waves a SIMD), and where 16
// lanes could not hold the experts or the places.
constexpr int64_t kRouteWide = 4096;

template <bool BF16, bool PLAIN>
hipError_t launch_route_size(const RouteArgs &a, hipStream_t s)
{
    if (a.T > kRouteWide && a.top <= 16) {
        if (a.E <= 64) return launch_route<16, 4, BF16, PLAIN>(a, s);
        if (a.E <= 128) return launch_route<16, 8, BF16, PLAIN>(a, s);
        if (a.E <= 256) return launch_route<16, 16, BF16, PLAIN>(a, s);
    }
    if (a.E <= 64) return launch_route<64, 1, BF16, PLAIN>(a, s);
    if (a.E <= 128) return launch_route<64, 2, BF16, PLAIN>(a, s);
    if (a.E <= 256) return launch_route<64, 4, BF16, PLAIN>(a, s);
    if (a.E <= 512) return launch_route<64, 8, BF16, PLAIN>(a, s);
    return launch_route<64, 16, BF16, PLAIN>(a, s);
}

bool aligned16(const void *p, int64_t ld) { return ((uintptr_t)p & 15) == 0 && (ld & 7) == 0; }

}  // namespace

// Chunks of the row order's counts: whole rounds of a route workgroup's teams
// (32 tokens of 16 lanes, 8 of 64), at most 256 chunks, since every part of
// the row order sums them all.
int32_t route_chunk(int64_t T, int32_t top)
{
    if (T * top <= kRouteSelfCount) return 0;
    const int64_t unit = T > kRouteWide ? 32 : 8, c = (T + 255) / 256;
    return (int32_t)((c + unit - 1) / unit * unit);
}

hipError_t launch_expert_route(const RouteArgs &a, hipStream_t s)
{
    const bool plain = a.bias == nullptr && a.groups == 1;
    if (a.bf16) return plain ? launch_route_size<true, true>(a, s) : launch_route_size<true, false>(a, s);
    return plain ? launch_route_size<false, true>(a, s) : launch_route_size<false, false>(a, s);
}

hipError_t launch_expert_sort(const RouteArgs &a, hipStream_t s)
{
    if (a.hist) {
        count_kernel<<<(unsigned)a.chunks, kRouteThreads, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return launch_order(a, s);
}

hipError_t launch_expert_route_backward(const RouteArgs &a, hipStream_t s)
{
    const unsigned grid = (unsigned)((a.T + 3) / 4);
    if (a.bf16)
        route_backward_kernel<true><<<grid, kThreads, 0, s>>>(a);
    else
        route_backward_kernel<false><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_expert_combine(const CombineArgs &a, hipStream_t s)
{
    const bool vec = a.H % 8 == 0 && aligned16(a.y, a.ldy) && aligned16(a.out, a.ldo) &&
                     (!a.residual || aligned16(a.residual, a.ldr));
    const int64_t per = kThreads * (vec ? 8 : 1);
    const dim3 grid((unsigned)a.T, (unsigned)((a.H + per - 1) / per));
    if (vec)
        combine_kernel<true><<<grid, kThreads, 0, s>>>(a);
    else
        combine_kernel<false><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_expert_combine_backward(const CombineArgs &a, hipStream_t s)
{
    const bool vec = a.H % 8 == 0 && aligned16(a.y, a.ldy) && aligned16(a.out, a.ldo) && aligned16(a.grad, a.ldr);
    if (vec)
        combine_backward_kernel<true><<<(unsigned)a.T, kThreads, 0, s>>>(a);
    else
        combine_backward_kernel<false><<<(unsigned)a.T, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace spg
