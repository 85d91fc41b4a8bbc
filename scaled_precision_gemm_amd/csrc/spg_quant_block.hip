// FP8 E4M3 quantizer with one fp32 scale per 128 elements: per 128 elements
// of a row (activations and gradients entering a product), per 128 elements
// of a column (gradients whose product runs along the rows) or per 128 x 128
// block (weights, read in both directions by forward and backward products).
//
//   s = fl32(max |x| / 448) over the group, q = E4M3(fl32(x / s))
//
// with the arithmetic of the row-wise quantizer (spg_quant_common.h), so a
// group of 128 gets the codes that quantize_rowwise would give a row of 128.
//
// The work is a stream: 2 bytes in and 1 + 4 / 128 (rows, columns) bytes out
// per element.  A group fits in registers, so the tensor is read once: every
// thread has its whole share of loads in flight before the first maximum.
// Measured: 34816 x 5120 in blocks 100 us, 5.3 TB/s read and written (a plain
// copy 4.9); 16 x 5120 in rows 4.4 us, the time of one wave's loads, maximum
// and stores, inside a call of 9 us that its two output tensors and one launch
// take on the host.
#include "spg_gemm_block.h"
#include "spg_quant_common.h"

namespace spg {

namespace {

using namespace quant;

constexpr int kGroup = 128;
constexpr int kRowTile = 16;      // rows of a workgroup of the row kernel
constexpr int kColTile = 512;     // columns of a workgroup of the row kernel (four groups)

__device__ __forceinline__ uint32_t max16(uint32_t m)
{
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
    return m;
}

// Row groups.  One workgroup per 16 rows x 512 columns: wave w takes rows
// 4 w .. 4 w + 3, each as one 1 KiB segment (lane l: columns 8 l .. 8 l + 7),
// and the 16 lanes of a group reduce its maximum among themselves.  The
// scales leave group-major ([groups, rows]), as the product reads them: 16
// consecutive rows of a group as one 64-byte segment, gathered in LDS.
__global__ __launch_bounds__(kThreads) void quant_block_row_kernel(
    const uint16_t *__restrict__ x, int64_t rows, int64_t K, int64_t ldx, int64_t bstride, uint8_t *__restrict__ q,
    int64_t ldq, int64_t qbstride, float *__restrict__ scale)
{
    __shared__ float lds_s[kColTile / kGroup][kRowTile];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t r0 = (int64_t)blockIdx.x * kRowTile, c0 = (int64_t)blockIdx.y * kColTile, b = blockIdx.z;
    const int64_t col = c0 + lane * 8;
    const uint16_t *xb = x + b * bstride;
    uint8_t *qb = q + b * qbstride;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = r0 + wave * 4 + i;
        v[i] = make_uint4(0, 0, 0, 0);
        if (row < rows && col < K) v[i] = ld16(xb + row * ldx + col);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t row = r0 + wave * 4 + i;
        const RowScale t = row_scale(__uint_as_float(max16(amax8(v[i])) << 16));
        if ((lane & 15) == 0) lds_s[lane >> 4][wave * 4 + i] = t.s;
        if (row < rows && col < K)
            with_encode_mode(t, [&](auto mode_c) {
                *reinterpret_cast<uint2 *>(qb + row * ldq + col) = encode8_e4m3<decltype(mode_c)::value>(v[i], t);
            });
    }
    __syncthreads();
    const int64_t groups = (K + kGroup - 1) / kGroup;
    const int g = (int)threadIdx.x >> 4, r = (int)threadIdx.x & 15;
    if (g < kColTile / kGroup && c0 / kGroup + g < groups && r0 + r < rows)
        scale[(b * groups + c0 / kGroup + g) * rows + r0 + r] = lds_s[g][r];
}

// One E4M3 code of x with its own scale (COLUMN tiling: neighbouring columns
// have different scales); the value encode8_e4m3 gives.
__device__ __forceinline__ float quot_any(float x, const RowScale &t) { return quot<true>(x, t); }
__device__ __forceinline__ uint32_t encode_slow(uint32_t h, float s)
{
    return s > 0.0f ? encode_e4m3(__uint_as_float(h << 16) / s) : (h >> 8) & 0x80u;
}

// 128 x 128 tiles: thread t holds columns 8 (t % 16) .. + 7 of rows
// t / 16 + 16 i (i = 0 .. 7), 32 registers, so one wave load covers four
// 256-byte row segments.  BLOCK: one maximum of the tile, scale plane
// [row blocks, column blocks].  COLUMN: one maximum per column, over the
// thread's 8 rows, the 4 threads of a wave that share its columns and the 4
// waves; scale plane [row blocks, K].
template <bool COLUMN>
__global__ __launch_bounds__(kThreads) void quant_block_tile_kernel(
    const uint16_t *__restrict__ x, int64_t rows, int64_t K, int64_t ldx, int64_t bstride, uint8_t *__restrict__ q,
    int64_t ldq, int64_t qbstride, float *__restrict__ scale)
{
    __shared__ uint32_t lds_m[4][kGroup];
    __shared__ uint32_t lds4[4];
    const int wave = threadIdx.x >> 6, c16 = threadIdx.x & 15, r16 = threadIdx.x >> 4;
    const int64_t r0 = (int64_t)blockIdx.y * kGroup, c0 = (int64_t)blockIdx.x * kGroup, b = blockIdx.z;
    const int64_t col = c0 + c16 * 8;
    const uint16_t *xb = x + b * bstride;
    uint8_t *qb = q + b * qbstride;
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = r0 + r16 + 16 * i;
        v[i] = make_uint4(0, 0, 0, 0);
        if (row < rows && col < K) v[i] = ld16(xb + row * ldx + col);
    }
    if (!COLUMN) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, amax8(v[i]));
        const RowScale t = row_scale(__uint_as_float(block_max_u32(m, lds4) << 16));
        if (threadIdx.x == 0) scale[(b * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = t.s;
        with_encode_mode(t, [&](auto mode_c) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t row = r0 + r16 + 16 * i;
                if (row < rows && col < K)
                    *reinterpret_cast<uint2 *>(qb + row * ldq + col) = encode8_e4m3<decltype(mode_c)::value>(v[i], t);
            }
        });
        return;
    }
    // halves of word j: columns 2 j and 2 j + 1
    uint32_t m[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m[2 * j] = max(m[2 * j], w[j] & 0x7FFFu);
            m[2 * j + 1] = max(m[2 * j + 1], (w[j] >> 16) & 0x7FFFu);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], 16, 64));
        m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], 32, 64));
    }
    if ((threadIdx.x & 63) < 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) lds_m[wave][c16 * 8 + j] = m[j];
    }
    __syncthreads();
    RowScale t[8];
    bool fast = true;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = c16 * 8 + j;
        t[j] = row_scale(__uint_as_float(max(max(lds_m[0][c], lds_m[1][c]), max(lds_m[2][c], lds_m[3][c])) << 16));
        fast = fast && t[j].fast;
    }
    if (r16 == 0 && col < K) {
        float *s = scale + (b * gridDim.y + blockIdx.y) * K + col;      // K % 16 == 0: 8 columns exist
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = t[j].s;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = r0 + r16 + 16 * i;
        if (row >= rows || col >= K) continue;
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t out[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (fast) {
                int d = __builtin_amdgcn_cvt_pk_fp8_f32(quot_any(bf16_lo(w[2 * h]), t[4 * h]),
                                                        quot_any(bf16_hi(w[2 * h]), t[4 * h + 1]), 0, false);
                out[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(quot_any(bf16_lo(w[2 * h + 1]), t[4 * h + 2]),
                                                                   quot_any(bf16_hi(w[2 * h + 1]), t[4 * h + 3]), d, true);
            } else {
                out[h] = encode_slow(w[2 * h] & 0xFFFFu, t[4 * h].s) | encode_slow(w[2 * h] >> 16, t[4 * h + 1].s) << 8 |
                         encode_slow(w[2 * h + 1] & 0xFFFFu, t[4 * h + 2].s) << 16 |
                         encode_slow(w[2 * h + 1] >> 16, t[4 * h + 3].s) << 24;
            }
        }
        *reinterpret_cast<uint2 *>(qb + row * ldq + col) = make_uint2(out[0], out[1]);
    }
}

}  // namespace

hipError_t launch_quantize_block128(const uint16_t *x, int64_t batch, int64_t rows, int64_t K, int64_t ldx,
                                    int64_t bstride, uint8_t *q, int64_t ldq, int64_t qbstride, float *scale,
                                    int tiling, hipStream_t s)
{
    if (tiling == SPG_BLOCK_ROW) {
        const dim3 grid((unsigned)((rows + kRowTile - 1) / kRowTile), (unsigned)((K + kColTile - 1) / kColTile),
                        (unsigned)batch);
        quant_block_row_kernel<<<grid, kThreads, 0, s>>>(x, rows, K, ldx, bstride, q, ldq, qbstride, scale);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)((K + kGroup - 1) / kGroup), (unsigned)((rows + kGroup - 1) / kGroup), (unsigned)batch);
    if (tiling == SPG_BLOCK_COLUMN)
        quant_block_tile_kernel<true><<<grid, kThreads, 0, s>>>(x, rows, K, ldx, bstride, q, ldq, qbstride, scale);
    else
        quant_block_tile_kernel<false><<<grid, kThreads, 0, s>>>(x, rows, K, ldx, bstride, q, ldq, qbstride, scale);
    return hipGetLastError();
}

}  // namespace spg
