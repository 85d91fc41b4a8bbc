// The norm over all gradients of a step, and the gradients scaled to at most a
// given norm.
//
//   n = sqrt(sum over all tensors of g^2)        64-bit sums
//   g' = g (n > max ? max / n : 1)               fp32, one rounding to g's type
//
// max / n is a 64-bit quotient, held as an fp32 number and a power of two: below
// fp32's normal range it would lose bits that g', of a large g, still has.
//
// A stream: every gradient is read for the sum and, where it is scaled, read
// and written once more: 336 million bf16 elements in nine tensors take 149 us
// for the sums and 228 for the scaling, 2.0 GB at 5.3 TB/s, what a copy reaches.
// Few small tensors take the launches' time: 16 us a call for one of 1000
// elements, 0.6 us for every further one (the host's).
//
// Chunks of kGradChunk elements, none across two tensors, are dealt to at most
// kGradWorkgroups workgroups in turn; a workgroup leaves one partial sum, and
// they are added in order, so the same tensors give the same bits.  Squares are
// formed and added in 64 bits: 10^8 of them added in fp32 would lose the last
// ones, and fp32's largest values squared overflow it.
#include "spg_gemm_common.h"
#include "spg_gradients.h"

namespace spg {

namespace {

constexpr int kThreads = 256;

// 16 bytes at any address that an element may have.
struct __attribute__((packed, aligned(2))) Raw16 {
    uint32_t w[4];
};
template <bool BF16>
__device__ __forceinline__ uint4 load16(const void *p)
{
    if (BF16) {
        const Raw16 v = *reinterpret_cast<const Raw16 *>(p);
        return make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    }
    struct __attribute__((packed, aligned(4))) R {
        uint32_t w[4];
    };
    const R v = *reinterpret_cast<const R *>(p);
    return make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}

// Vectors v0 + 256 i of `vecs` (at least one), zeros past them.  No branch
// stands between the loads and nothing is moved between them, so that all are
// in flight at once.
template <bool BF16>
__device__ __forceinline__ void load_vectors(uint4 (&r)[8], const uint8_t *b, int v0, int vecs)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int v = v0 + i * kThreads;
        r[i] = load16<BF16>(b + (int64_t)(v < vecs ? v : 0) * 16);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (v0 + i * kThreads >= vecs) r[i] = make_uint4(0, 0, 0, 0);
}

// The tensor of chunk c: the last one whose first chunk is not behind it.
__device__ __forceinline__ int find_tensor(const GradTensors &t, uint32_t c)
{
    int lo = 0, hi = t.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.first[mid] <= c)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ double square(float f, double s) { return __builtin_fma((double)f, (double)f, s); }

// Sum of the squares of n elements at p over this thread's share.
template <bool BF16>
__device__ __forceinline__ double chunk_sum(const void *p, int n)
{
    constexpr int W = BF16 ? 8 : 4, SIZE = BF16 ? 2 : 4;
    const uint8_t *b = (const uint8_t *)p;
    double s = 0.0;
    const int vecs = n / W;
    for (int v0 = (int)threadIdx.x; v0 < vecs; v0 += kThreads * 8) {
        uint4 r[8];
        load_vectors<BF16>(r, b, v0, vecs);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (BF16) {
                    s = square(bf16_lo(w[k]), s);
                    s = square(bf16_hi(w[k]), s);
                } else {
                    s = square(__uint_as_float(w[k]), s);
                }
            }
        }
    }
    const int at = vecs * W + (int)threadIdx.x;
    if (at < n)
        s = square(BF16 ? bf16_lo(*(const uint16_t *)(b + (int64_t)at * SIZE)) : *(const float *)(b + (int64_t)at * SIZE), s);
    return s;
}

__device__ __forceinline__ double block_sum(double s, double *lds)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) s += lds[w];
    return s;
}

__global__ __launch_bounds__(kThreads) void grad_sums_kernel(const GradTensors t, double *partials)
{
    __shared__ double lds[kThreads / 64];
    double s = 0.0;
    for (uint32_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        const int i = find_tensor(t, c);
        const int64_t at = (int64_t)(c - t.first[i]) * kGradChunk;
        const int n = (int)min(t.n[i] - at, kGradChunk);
        if (t.bf16[i])
            s += chunk_sum<true>((const uint16_t *)t.src[i] + at, n);
        else
            s += chunk_sum<false>((const float *)t.src[i] + at, n);
    }
    s = block_sum(s, lds);
    if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

// What scales gradients of norm n.  A 64-bit norm that is not finite (a gradient
// is NaN or infinite) scales nothing: the caller sees it.
__device__ __forceinline__ GradFactor factor_of(double n, double max_norm)
{
    const double q = n > max_norm && n < __builtin_inf() ? max_norm / n : 1.0;
    const int e = q > 0.0 && q < 0x1p-126 ? __builtin_amdgcn_frexp_exp(q) : 0;
    return GradFactor{(float)__builtin_amdgcn_ldexp(q, -e), e};
}
__device__ __forceinline__ float scaled(float g, const GradFactor &f) { return __builtin_amdgcn_ldexpf(g * f.f, f.e); }

__global__ __launch_bounds__(1024) void grad_norm_kernel(const double *partials, int64_t parts, double max_norm, float *norm,
                                                          GradFactor *factor)
{
    __shared__ double lds[16];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < parts; i += 1024) s += partials[i];
    s = block_sum(s, lds);
    if (threadIdx.x == 0) {
        const double n = __builtin_sqrt(s);
        norm[0] = (float)n;
        if (factor) factor[0] = factor_of(n, max_norm);
    }
}

template <bool BF16>
__device__ __forceinline__ void chunk_scale(const void *p, void *q, int n, const GradFactor &f)
{
    constexpr int W = BF16 ? 8 : 4, SIZE = BF16 ? 2 : 4;
    const uint8_t *b = (const uint8_t *)p;
    uint8_t *o = (uint8_t *)q;
    const int vecs = n / W;
    for (int v0 = (int)threadIdx.x; v0 < vecs; v0 += kThreads * 8) {
        uint4 r[8];
        load_vectors<BF16>(r, b, v0, vecs);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int v = v0 + i * kThreads;
            uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = BF16 ? gemm::pack_bf16x2(scaled(bf16_lo(w[k]), f), scaled(bf16_hi(w[k]), f))
                            : __float_as_uint(scaled(__uint_as_float(w[k]), f));
            if (v < vecs) {
                if (BF16) {
                    *reinterpret_cast<Raw16 *>(o + (int64_t)v * 16) = Raw16{{w[0], w[1], w[2], w[3]}};
                } else {
                    struct __attribute__((packed, aligned(4))) R {
                        uint32_t w[4];
                    };
                    *reinterpret_cast<R *>(o + (int64_t)v * 16) = R{{w[0], w[1], w[2], w[3]}};
                }
            }
        }
    }
    const int at = vecs * W + (int)threadIdx.x;
    if (at < n) {
        if (BF16)
            *(uint16_t *)(o + (int64_t)at * SIZE) = (uint16_t)f32_to_bf16(scaled(bf16_lo(*(const uint16_t *)(b + (int64_t)at * SIZE)), f));
        else
            *(float *)(o + (int64_t)at * SIZE) = scaled(*(const float *)(b + (int64_t)at * SIZE), f);
    }
}

__global__ __launch_bounds__(kThreads) void grad_scale_kernel(const GradTensors t, const GradFactor *factor, const double *partials,
                                                              int64_t parts, double max_norm, float *norm)
{
    __shared__ double lds[kThreads / 64];
    GradFactor f;
    if (partials) {
        double s = 0.0;
        for (int64_t i = threadIdx.x; i < parts; i += kThreads) s += partials[i];
        const double n = __builtin_sqrt(block_sum(s, lds));
        f = factor_of(n, max_norm);
        if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = (float)n;
    } else {
        f = *factor;
    }
    for (uint32_t c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
        const int i = find_tensor(t, c);
        if (f.f == 1.0f && t.src[i] == t.dst[i]) continue;        // nothing changes
        const int64_t at = (int64_t)(c - t.first[i]) * kGradChunk;
        const int n = (int)min(t.n[i] - at, kGradChunk);
        if (t.bf16[i])
            chunk_scale<true>((const uint16_t *)t.src[i] + at, (uint16_t *)t.dst[i] + at, n, f);
        else
            chunk_scale<false>((const float *)t.src[i] + at, (float *)t.dst[i] + at, n, f);
    }
}

}  // namespace

hipError_t launch_grad_sums(const GradTensors &t, double *partials, hipStream_t s)
{
    const unsigned grid = (unsigned)grad_parts(t.first[t.count]);
    grad_sums_kernel<<<grid, kThreads, 0, s>>>(t, partials);
    return hipGetLastError();
}

hipError_t launch_grad_norm(const double *partials, int64_t parts, double max_norm, float *norm, GradFactor *factor,
                            hipStream_t s)
{
    grad_norm_kernel<<<1, 1024, 0, s>>>(partials, parts, max_norm, norm, factor);
    return hipGetLastError();
}

hipError_t launch_grad_scale(const GradTensors &t, const GradFactor *factor, const double *partials, int64_t parts, double max_norm,
                             float *norm, hipStream_t s)
{
    const unsigned grid = (unsigned)grad_parts(t.first[t.count]);
    grad_scale_kernel<<<grid, kThreads, 0, s>>>(t, factor, partials, parts, max_norm, norm);
    return hipGetLastError();
}

}  // namespace spg
