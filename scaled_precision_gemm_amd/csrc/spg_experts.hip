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
// A team of 16 lanes (64 where E > 256 or top > 16) works on one token; lane
// l holds the EPL consecutive experts l EPL .., so of equal values the lowest
// lane has the lowest index.  Each of the `top` rounds takes the team's
// maximum - of the keys' high words through DPP row operations, then of the
// low words where more than one lane holds the maximum - and the winner drops
// its expert.  Four tokens share a wave's rounds.
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

template <int TEAM>
__device__ __forceinline__ uint32_t team_max(uint32_t v)
{
    v = max(v, dpp<kXor1>(v));
    v = max(v, dpp<kXor2>(v));
    v = max(v, dpp<kHalfMirror>(v));
    v = max(v, dpp<kMirror>(v));
    if (TEAM == 64) {
        v = max(v, (uint32_t)__shfl_xor((int)v, 16, 64));
        v = max(v, (uint32_t)__shfl_xor((int)v, 32, 64));
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

// LDS of one token while it is routed: its choices (groups only), its group
// scores, then the chosen experts and their scores.
template <int TEAM>
struct TokenLds {
    double score[kRouteMaxGroups];
    double p[TEAM == 16 ? 16 : kRouteMaxTop];
    int32_t e[TEAM == 16 ? 16 : kRouteMaxTop];
    uint64_t kept;
};

// Routes the token of this team (live: it exists); `c` is room for E doubles
// when GROUPS.  On return lanes j < top hold weight and expert of choice j.
// Every lane of the workgroup calls it (it holds barriers).
template <int TEAM, int EPL, bool BF16, bool PLAIN>
__device__ __forceinline__ void route_token(const RouteArgs &a, int64_t t, bool live, TokenLds<TEAM> &L, double *c,
                                            float &w_out, int32_t &e_out)
{
#pragma clang fp contract(off)
    const int tl = threadIdx.x & (TEAM - 1);
    using Key = typename std::conditional<PLAIN, uint32_t, uint64_t>::type;
    float l[EPL];
    Key key[EPL];
    float mx = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = tl * EPL + i;
        l[i] = live && e < a.E ? load_logit<BF16>(a, t, e) : -INFINITY;
        nan = nan || l[i] != l[i];
        mx = l[i] > mx ? l[i] : mx;
    }
    nan = team_ballot<TEAM>(nan) != 0;
    // the largest logit (fp32 order through the keys) and the softmax sum
    {
        const uint32_t k = team_max<TEAM>(key32(mx));
        mx = k == 0u ? -INFINITY : __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
    }
    const bool soft = a.score == SPG_SCORE_SOFTMAX;
    // score of a logit before the softmax's division; an infinite maximum
    // counts as the only size that matters (1 for it, 0 for the others)
    auto raw = [&](float v) -> double {
        if (!(v > -INFINITY)) return 0.0;
        if (soft) return v == mx ? 1.0 : exp((double)v - (double)mx);
        return 1.0 / (1.0 + exp(-(double)v));
    };
    double z = 1.0;
    if (PLAIN) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = key32(l[i]);
        if (soft && !a.renorm) {
            double part = 0.0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) part += raw(l[i]);
            z = team_sum<TEAM>(part);
        }
    } else {
        double p[EPL], part = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            p[i] = raw(l[i]);
            part += p[i];
        }
        if (soft) z = team_sum<TEAM>(part);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = tl * EPL + i;
            double v = soft ? p[i] / z : p[i];
            if (a.bias && e < a.E) v = v + (double)a.bias[e];
            if (!(l[i] > -INFINITY)) v = -(double)INFINITY;
            key[i] = (Key)key64(v);
            if (a.groups > 1 && e < a.E) c[e] = v;
        }
        if (a.groups > 1) {
            __syncthreads();
            const int size = a.E / a.groups;
            for (int gI = tl; gI < a.groups; gI += TEAM) {
                double m1 = -(double)INFINITY, m2 = m1;
                for (int i = 0; i < size; ++i) {
                    const double v = c[gI * size + i];
                    if (v > m1) {
                        m2 = m1;
                        m1 = v;
                    } else if (v > m2) {
                        m2 = v;
                    }
                }
                L.score[gI] = m2 > -(double)INFINITY ? m1 + m2 : m1;
            }
            if (tl == 0) L.kept = 0;
            __syncthreads();
            for (int gI = tl; gI < a.groups; gI += TEAM) {
                const double v = L.score[gI];
                int better = 0;
                for (int h = 0; h < a.groups; ++h) {
                    const double o = L.score[h];
                    better += (o > v || (o == v && h < gI)) ? 1 : 0;
                }
                if (better < a.top_groups && v > -(double)INFINITY)
                    atomicOr((unsigned long long *)&L.kept, 1ull << gI);
            }
            __syncthreads();
            const uint64_t kept = L.kept;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const uint32_t gI = fdiv_q((uint32_t)(tl * EPL + i), a.div_group);
                if (gI >= 64u || !((kept >> gI) & 1ull)) key[i] = 0;
            }
        }
    }
    // the rounds
    int32_t my_e = -1;
    for (int j = 0; j < a.top; ++j) {
        Key best = key[0];
        int bi = 0;
#pragma unroll
        for (int i = 1; i < EPL; ++i)
            if (key[i] > best) {
                best = key[i];
                bi = i;
            }
        bool cand;
        if (PLAIN) {
            const uint32_t m = team_max<TEAM>((uint32_t)best);   // in every lane: row operations read all 16
            cand = best != 0 && best == m;
        } else {
            const uint32_t hi = (uint32_t)((uint64_t)best >> 32);
            const uint32_t mh = team_max<TEAM>(hi);
            cand = best != 0 && hi == mh;
            const uint32_t lo = cand ? (uint32_t)best : 0u;
            const uint32_t ml = team_max<TEAM>(lo);
            cand = cand && lo == ml;
        }
        const uint64_t who = team_ballot<TEAM>(cand);
        const int winner = who ? __builtin_ctzll(who) : -1;
        if (tl == winner) {
            L.e[j] = tl * EPL + bi;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i == bi) {
                    key[i] = 0;
                    L.p[j] = raw(l[i]);
                }
        } else if (winner < 0 && tl == 0) {
            L.e[j] = -1;
            L.p[j] = 0.0;
        }
    }
    __syncthreads();
    double pj = 0.0;
    if (tl < a.top) {
        pj = L.p[tl];
        my_e = L.e[tl];
    }
    if (soft && !a.renorm) pj = z > 0.0 ? pj / z : 0.0;
    const double total = a.renorm ? team_sum<TEAM>(pj) : 1.0;
    double w = total > 0.0 ? (double)a.scale * (pj / total) : 0.0;
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

constexpr int kSortThreads = 1024, kOneThreads = 512;

// Ranks entries [n0, n1) of `experts` (flat, token-major) into the row order:
// base[e] (LDS) is the position of the first of them for expert e.  Each wave
// takes a contiguous run of entries, counted first (cnt[wave][e]) so that the
// order is that of the entries.  Entries with no expert get slot -1.
template <int NT>
__device__ __forceinline__ void sort_entries(const RouteArgs &a, const int32_t *experts, int64_t n0, int64_t n1,
                                             int32_t *base, int32_t *cnt)
{
    constexpr int kSortWaves = NT / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int E = a.E;
    const int bits = 32 - __builtin_clz((unsigned)E);
    const int64_t n = n1 - n0, per = ((n + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
    const int64_t w0 = n0 + min(n, wave * per), w1 = n0 + min(n, (wave + 1) * per);
    for (int i = tid; i < kSortWaves * E; i += NT) cnt[i] = 0;
    __syncthreads();
    int32_t *mine = cnt + wave * E;
    for (int64_t i = w0 + lane; i < w1; i += 64) {
        const int32_t e = experts[i];
        if ((uint32_t)e < (uint32_t)E) atomicAdd(&mine[e], 1);
    }
    __syncthreads();
    for (int e = tid; e < E; e += NT) {
        int32_t at = base[e];
        for (int w = 0; w < kSortWaves; ++w) {
            const int32_t c = cnt[w * E + e];
            cnt[w * E + e] = at;
            at += c;
        }
    }
    __syncthreads();
    // the next position of each expert, read and written by lanes of one wave
    volatile int32_t *next = mine;
    for (int64_t i0 = w0; i0 < w1; i0 += 64) {
        const int64_t i = i0 + lane;
        const int32_t e = i < w1 ? experts[i] : -1;
        const bool valid = (uint32_t)e < (uint32_t)E;
        const uint64_t same = match_expert(e, valid, bits);
        int32_t pos = -1;
        if (valid) {
            const uint64_t below = same & ((1ull << lane) - 1);
            pos = next[e] + __popcll(below);
            a.rows[pos] = (int32_t)fdiv_q((uint32_t)i, a.div_top);
        }
        __builtin_amdgcn_wave_barrier();
        if (valid && (same >> lane) == 1ull) next[e] = pos + 1;      // the last lane of its expert
        __builtin_amdgcn_wave_barrier();
        if (i < w1) a.slots[i] = pos;
    }
}

// start[e] = rows of experts below e, for the totals in start; returns
// (in every thread) the sum.
template <int NT>
__device__ __forceinline__ int32_t exclusive_scan(int32_t *start, int E, int32_t *wsum)
{
    constexpr int kWaves = NT / 64, kPer = kRouteMaxExperts / NT;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int32_t v[kPer], mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        v[i] = tid * kPer + i < E ? start[tid * kPer + i] : 0;
        mine += v[i];
    }
    int32_t s = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int32_t o = __shfl_up(s, off, 64);
        if (lane >= off) s += o;
    }
    if (lane == 63) wsum[wave] = s;
    __syncthreads();
    int32_t at = s - mine, all = 0;
    for (int w = 0; w < kWaves; ++w) {
        at += w < wave ? wsum[w] : 0;
        all += wsum[w];
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (tid * kPer + i < E) start[tid * kPer + i] = at;
        at += v[i];
    }
    __syncthreads();
    return all;
}

// Tokens in order, one team each; a workgroup takes `chunk` tokens and counts
// its experts for the row order.
template <int TEAM, int EPL, bool BF16, bool PLAIN>
__global__ __launch_bounds__(kThreads) void route_kernel(const RouteArgs a)
{
    constexpr int TOK = kThreads / TEAM;
    __shared__ TokenLds<TEAM> lds_t[TOK];
    extern __shared__ double lds_c[];
    __shared__ int32_t lds_h[kRouteMaxExperts];
    const int tid = threadIdx.x, tl = tid & (TEAM - 1), team = tid / TEAM;
    const int64_t t0 = (int64_t)blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
    const bool count = a.offsets != nullptr;
    if (count) {
        for (int e = tid; e < a.E; e += kThreads) lds_h[e] = 0;
        __syncthreads();
    }
    for (int64_t tb = t0; tb < t1; tb += TOK) {
        const int64_t t = tb + team;
        const bool live = t < t1;
        float w;
        int32_t e;
        route_token<TEAM, EPL, BF16, PLAIN>(a, t, live, lds_t[team], lds_c + (int64_t)team * a.E, w, e);
        if (live && tl < a.top) {
            a.weights[t * a.top + tl] = w;
            a.experts[t * a.top + tl] = e;
            if (count && e >= 0) atomicAdd(&lds_h[e], 1);
        }
        __syncthreads();
    }
    if (count)
        for (int e = tid; e < a.E; e += kThreads) a.hist[(int64_t)blockIdx.x * a.E + e] = lds_h[e];
}

// The same for at most kRouteOneLaunch tokens in one workgroup, the row order
// included: a decode step's routing is one launch.
template <int TEAM, int EPL, bool BF16, bool PLAIN>
__global__ __launch_bounds__(kOneThreads) void route_one_kernel(const RouteArgs a)
{
    constexpr int TOK = kOneThreads / TEAM;
    __shared__ TokenLds<TEAM> lds_t[TOK];
    __shared__ int32_t lds_e[kRouteOneLaunch * kRouteMaxTop];
    __shared__ int32_t lds_start[kRouteMaxExperts];
    __shared__ int32_t lds_wsum[kOneThreads / 64];
    extern __shared__ double lds_dyn[];
    const int tid = threadIdx.x, tl = tid & (TEAM - 1), team = tid / TEAM;
    for (int e = tid; e < a.E; e += kOneThreads) lds_start[e] = 0;
    __syncthreads();
    for (int64_t tb = 0; tb < a.T; tb += TOK) {
        const int64_t t = tb + team;
        const bool live = t < a.T;
        float w;
        int32_t e;
        route_token<TEAM, EPL, BF16, PLAIN>(a, t, live, lds_t[team], lds_dyn + (int64_t)team * a.E, w, e);
        if (live && tl < a.top) {
            a.weights[t * a.top + tl] = w;
            a.experts[t * a.top + tl] = e;
            lds_e[t * a.top + tl] = e;
            if (e >= 0) atomicAdd(&lds_start[e], 1);
        }
        __syncthreads();
    }
    if (a.offsets == nullptr) return;
    const int32_t all = exclusive_scan<kOneThreads>(lds_start, a.E, lds_wsum);
    for (int e = tid; e < a.E; e += kOneThreads) a.offsets[e] = lds_start[e];
    if (tid == 0) a.offsets[a.E] = all;
    const int64_t n = a.T * a.top;
    for (int64_t i = all + tid; i < n; i += kOneThreads) a.rows[i] = -1;
    sort_entries<kOneThreads>(a, lds_e, 0, n, lds_start, (int32_t *)lds_dyn);
}

// Experts of one chunk of tokens counted (the row order of given experts).
__global__ __launch_bounds__(kThreads) void count_kernel(const RouteArgs a)
{
    __shared__ int32_t lds_h[kRouteMaxExperts];
    for (int e = threadIdx.x; e < a.E; e += kThreads) lds_h[e] = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
    for (int64_t i = t0 * a.top + threadIdx.x; i < t1 * a.top; i += kThreads) {
        const int32_t e = a.experts[i];
        if ((uint32_t)e < (uint32_t)a.E) atomicAdd(&lds_h[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kThreads) a.hist[(int64_t)blockIdx.x * a.E + e] = lds_h[e];
}

// The row order of at most kRouteOneLaunch tokens' experts, in one workgroup.
__global__ __launch_bounds__(kOneThreads) void sort_one_kernel(const RouteArgs a)
{
    __shared__ int32_t lds_start[kRouteMaxExperts];
    __shared__ int32_t lds_wsum[kOneThreads / 64];
    extern __shared__ double lds_dyn[];
    const int tid = threadIdx.x;
    const int64_t n = a.T * a.top;
    for (int e = tid; e < a.E; e += kOneThreads) lds_start[e] = 0;
    __syncthreads();
    for (int64_t i = tid; i < n; i += kOneThreads) {
        const int32_t e = a.experts[i];
        if ((uint32_t)e < (uint32_t)a.E) atomicAdd(&lds_start[e], 1);
    }
    __syncthreads();
    const int32_t all = exclusive_scan<kOneThreads>(lds_start, a.E, lds_wsum);
    for (int e = tid; e < a.E; e += kOneThreads) a.offsets[e] = lds_start[e];
    if (tid == 0) a.offsets[a.E] = all;
    for (int64_t i = all + tid; i < n; i += kOneThreads) a.rows[i] = -1;
    sort_entries<kOneThreads>(a, a.experts, 0, n, lds_start, (int32_t *)lds_dyn);
}

// Row order from the chunks' counts: every workgroup sums the counts of the
// chunks before its own (and of all, for the experts' starts) and ranks its
// own chunk's entries.
__global__ __launch_bounds__(kSortThreads) void order_kernel(const RouteArgs a)
{
    extern __shared__ double lds_dyn[];
    __shared__ int32_t lds_start[kRouteMaxExperts];
    __shared__ int32_t lds_wsum[kSortThreads / 64];
    const int tid = threadIdx.x;
    int32_t before = 0, total = 0;
    if (tid < a.E)
#pragma unroll 8
        for (int c = 0; c < a.chunks; ++c) {
            const int32_t v = a.hist[(int64_t)c * a.E + tid];
            before += c < (int)blockIdx.x ? v : 0;
            total += v;
        }
    if (tid < a.E) lds_start[tid] = total;
    __syncthreads();
    const int32_t all = exclusive_scan<kSortThreads>(lds_start, a.E, lds_wsum);
    const int64_t n = a.T * a.top;
    if (blockIdx.x == 0) {
        if (tid < a.E) a.offsets[tid] = lds_start[tid];
        if (tid == 0) a.offsets[a.E] = all;
        for (int64_t i = all + tid; i < n; i += kSortThreads) a.rows[i] = -1;
    }
    __syncthreads();
    if (tid < a.E) lds_start[tid] += before;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * a.chunk, t1 = min(a.T, t0 + a.chunk);
    sort_entries<kSortThreads>(a, a.experts, t0 * a.top, t1 * a.top, lds_start, (int32_t *)lds_dyn);
}

// ---- gradient of the logits --------------------------------------------------
// With q_j the chosen scores' shares:
//   renormalised:  d/dl of scale q_j; softmax over the chosen (the softmax's
//                  own sum cancels): dl_j = scale q_j (g_j - sum g q)
//                  sigmoid: dp_j = scale (g_j - sum g q) / sum p, dl = dp p (1 - p)
//   else softmax:  dl_e = p_e ([e chosen] scale g - sum scale g p)
//   else sigmoid:  dl_j = scale g_j p_j (1 - p_j)
// One wave per token: lane j < top works out choice j, then the wave writes
// the dense row.  An expert that stands twice in a row gets both parts.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(const RouteArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    if (t >= a.T) return;
    const bool soft = a.score == SPG_SCORE_SOFTMAX;
    int32_t e = lane < a.top ? a.experts[t * a.top + lane] : -1;
    if ((uint32_t)e >= (uint32_t)a.E) e = -1;
    const float g = e >= 0 ? a.grad[t * a.top + lane] * a.scale : 0.0f;
    const float l = e >= 0 ? load_logit<BF16>(a, t, e) : -INFINITY;
    float mine = 0.0f, common = 0.0f, mx = -INFINITY, rz = 0.0f;
    const bool dense = soft && !a.renorm;
    if (dense) {
        for (int i = lane; i < a.E; i += 64) mx = fmaxf(mx, load_logit<BF16>(a, t, i));
    } else {
        mx = l;
    }
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
    } else {
        // 1 - p as the sigmoid of -l: exact where p rounds to 1
        const float p = e >= 0 ? 1.0f / (1.0f + expf(-l)) : 0.0f, n = e >= 0 ? 1.0f / (1.0f + expf(l)) : 0.0f;
        if (a.renorm) {
            const float z = team_sum<64>(p);
            const float dot = team_sum<64>(g * p);
            mine = z > 0.0f ? (g - dot / z) / z * (p * n) : 0.0f;
        } else {
            mine = g * p * n;
        }
    }
    for (int i0 = 0; i0 < a.E; i0 += 64) {
        const int i = i0 + lane;
        float v = dense && i < a.E ? -ex(load_logit<BF16>(a, t, i)) * rz * common : 0.0f;
        for (int j = 0; j < a.top; ++j) {
            const int32_t ej = __shfl(e, j, 64);
            const float mj = __shfl(mine, j, 64);
            if (ej == i) v += mj;
        }
        if (i < a.E) {
            if (BF16)
                ((uint16_t *)a.grad_logits)[t * a.E + i] = (uint16_t)f32_to_bf16(v);
            else
                ((float *)a.grad_logits)[t * a.E + i] = v;
        }
    }
}

// ---- combine -----------------------------------------------------------------
// out[t] = residual[t] + sum_j w[t, j] y[slot[t, j]], fp32 sums in the order
// of j, one rounding.  A stream over the chosen rows: one workgroup per token
// and 2048 columns, 16 bytes per lane and row, up to eight rows in flight.
// VEC: every pointer and row stride is 16-byte aligned and H % 8 == 0; else
// one element per lane.
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
                    v[j] = *reinterpret_cast<const uint4 *>(p);
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
        *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[2], w[3]);
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

template <int TEAM, int EPL, bool BF16, bool PLAIN>
hipError_t launch_route(const RouteArgs &a, hipStream_t s)
{
    if (a.T <= kRouteOneLaunch) {
        const size_t choices = a.groups > 1 ? (size_t)(kOneThreads / TEAM) * a.E * sizeof(double) : 0;
        const size_t counts = a.offsets ? (size_t)(kOneThreads / 64) * a.E * sizeof(int32_t) : 0;
        route_one_kernel<TEAM, EPL, BF16, PLAIN>
            <<<1, kOneThreads, choices > counts ? choices : counts, s>>>(a);
        return hipGetLastError();
    }
    const size_t choices = a.groups > 1 ? (size_t)(kThreads / TEAM) * a.E * sizeof(double) : 0;
    route_kernel<TEAM, EPL, BF16, PLAIN><<<(unsigned)a.chunks, kThreads, choices, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.offsets == nullptr) return e;
    order_kernel<<<(unsigned)a.chunks, kSortThreads, (size_t)(kSortThreads / 64) * a.E * sizeof(int32_t), s>>>(a);
    return hipGetLastError();
}

template <bool BF16, bool PLAIN>
hipError_t launch_route_size(const RouteArgs &a, hipStream_t s)
{
    if (a.top <= 16) {
        if (a.E <= 64) return launch_route<16, 4, BF16, PLAIN>(a, s);
        if (a.E <= 128) return launch_route<16, 8, BF16, PLAIN>(a, s);
        if (a.E <= 256) return launch_route<16, 16, BF16, PLAIN>(a, s);
    }
    if (a.E <= 256) return launch_route<64, 4, BF16, PLAIN>(a, s);
    if (a.E <= 512) return launch_route<64, 8, BF16, PLAIN>(a, s);
    return launch_route<64, 16, BF16, PLAIN>(a, s);
}

bool aligned16(const void *p, int64_t ld) { return ((uintptr_t)p & 15) == 0 && (ld & 7) == 0; }

}  // namespace

// At most 256 chunks, so the sums over the chunks' counts stay short, and at
// least 64 tokens each.
int64_t route_chunk(int64_t T)
{
    const int64_t c = (T + 255) / 256;
    return c < 64 ? 64 : c;
}

hipError_t launch_expert_route(const RouteArgs &a, hipStream_t s)
{
    const bool plain = a.bias == nullptr && a.groups == 1;
    if (a.bf16) return plain ? launch_route_size<true, true>(a, s) : launch_route_size<true, false>(a, s);
    return plain ? launch_route_size<false, true>(a, s) : launch_route_size<false, false>(a, s);
}

hipError_t launch_expert_sort(const RouteArgs &a, hipStream_t s)
{
    if (a.T <= kRouteOneLaunch) {
        sort_one_kernel<<<1, kOneThreads, (size_t)(kOneThreads / 64) * a.E * sizeof(int32_t), s>>>(a);
        return hipGetLastError();
    }
    count_kernel<<<(unsigned)a.chunks, kThreads, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    order_kernel<<<(unsigned)a.chunks, kSortThreads, (size_t)(kSortThreads / 64) * a.E * sizeof(int32_t), s>>>(a);
    return hipGetLastError();
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
