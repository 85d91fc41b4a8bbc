// Byte transpose of FP8 codes for K-major operands (spg_layout): a stored
// [R, C] code matrix (row stride ld, batch stride bstride) becomes [C, R]
// with row stride ldd, which the NT GEMM kernels then read K-contiguous.
//
// One workgroup per 128 x 128 block of one batch entry.  A thread loads 16
// bytes of four consecutive source rows (128-byte row segments), transposes
// its four 4 x 4 byte squares in registers with byte permutes, and writes 16
// words - four rows of one column each - to LDS; then it takes 16 bytes of a
// column (four words) and stores them as one 16-byte piece of a destination
// row.  HBM-bound: each byte is read and written once.  (Bytes one at a time
// through LDS, 32 LDS accesses a thread for 16 bytes: the two copies of a 4096 x
// 4096 x 4096 product took 20 us, in registers 15.6.)  Both operands of a
// product go in one launch (4096 x 2048 over 4000 tokens: 8.0 + 5.8 us in two
// launches, 9.5 in one, 5.1 TB/s read and written).
#include "spg_common.h"

namespace spg {

namespace {

constexpr int kTB = (int)kTransposeEdge;   // block edge (bytes)

// Word (column, group of four rows) in LDS: 32 words a column, the group
// XOR-ed with 8 ((column / 16) % 4) and neighbouring columns exchanged in the
// upper half, so that the 64 words a wave writes at once - eight groups of
// eight columns 16 apart - fall on 64 banks.
__device__ __forceinline__ uint32_t word(uint32_t col, uint32_t grp)
{
    return (col ^ (col >> 6)) * 32 + (grp ^ (((col >> 4) & 3u) << 3));
}

struct Jobs {
    TransposeJob job[2];
    uint32_t nbc[2], per[2];       // block columns, blocks of a batch entry
    uint32_t first;                // blocks of job 0
};

// One-dimensional grid of the jobs' blocks, job 0's first, block columns
// fastest.
__global__ __launch_bounds__(256) void transpose_u8_kernel(const Jobs a)
{
    __shared__ __attribute__((aligned(16))) uint32_t tile[kTB * 32];
    const int t = threadIdx.x;
    const int which = blockIdx.x >= a.first ? 1 : 0;
    const TransposeJob &job = a.job[which];
    const int64_t R = job.R, C = job.C, ld = job.ld, ldd = job.ldd;
    const uint32_t bid = blockIdx.x - (which ? a.first : 0u), per = a.per[which], nbc = a.nbc[which];
    const int64_t b = bid / per;
    const uint32_t rem = bid - (uint32_t)b * per;
    const int64_t r0 = (int64_t)(rem / nbc) * kTB, c0 = (int64_t)(rem % nbc) * kTB;
    const uint8_t *s = job.src + b * job.bstride;
    uint8_t *d = job.dst + b * C * ldd;

    // load: source rows r0 + 4 (t / 8) .. + 3, bytes c0 + 16 (t % 8) .. + 15
    {
        const uint32_t grp = (uint32_t)t >> 3, cc = ((uint32_t)t & 7) * 16;
        const int64_t col = c0 + cc;
        uint32_t w[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = r0 + 4 * grp + i;
            uint4 q = make_uint4(0, 0, 0, 0);
            if (row < R && col + 16 <= C) {
                q = *reinterpret_cast<const uint4 *>(s + row * ld + col);   // 16-byte aligned
            } else if (row < R && col < C) {
                uint32_t e[4] = {0, 0, 0, 0};
                for (int j = 0; j < 16 && col + j < C; ++j) e[j >> 2] |= (uint32_t)s[row * ld + col + j] << (8 * (j & 3));
                q = make_uint4(e[0], e[1], e[2], e[3]);
            }
            w[i][0] = q.x;
            w[i][1] = q.y;
            w[i][2] = q.z;
            w[i][3] = q.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // byte selectors: 0 - 3 the second operand's bytes, 4 - 7 the first's
            const uint32_t a0 = __builtin_amdgcn_perm(w[1][j], w[0][j], 0x05010400u);
            const uint32_t a1 = __builtin_amdgcn_perm(w[1][j], w[0][j], 0x07030602u);
            const uint32_t b0 = __builtin_amdgcn_perm(w[3][j], w[2][j], 0x05010400u);
            const uint32_t b1 = __builtin_amdgcn_perm(w[3][j], w[2][j], 0x07030602u);
            tile[word(cc + 4 * j, grp)] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);
            tile[word(cc + 4 * j + 1, grp)] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
            tile[word(cc + 4 * j + 2, grp)] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
            tile[word(cc + 4 * j + 3, grp)] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
        }
    }
    __syncthreads();

    // store: destination rows c0 + t / 8 + 32 i (source columns), bytes r0 + 16 (t % 8) .. + 15
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t oc = ((uint32_t)t >> 3) + 32 * i, rc = ((uint32_t)t & 7) * 16;
        const int64_t orow = c0 + oc, ocol = r0 + rc;
        if (orow >= C || ocol >= R) continue;
        // the XOR moves whole groups of eight words: four words stay together
        const uint4 q = *reinterpret_cast<const uint4 *>(&tile[word(oc, rc / 4)]);
        uint8_t *out = d + orow * ldd + ocol;
        if (ocol + 16 <= R) {
            *reinterpret_cast<uint4 *>(out) = q;                            // ldd % 16 == 0
        } else {
            const uint32_t e[4] = {q.x, q.y, q.z, q.w};
            for (int j = 0; j < 16 && ocol + j < R; ++j) out[j] = (uint8_t)(e[j >> 2] >> (8 * (j & 3)));
        }
    }
}

}  // namespace

hipError_t launch_transpose_u8(const TransposeJob *jobs, int n, hipStream_t s)
{
    Jobs a = {};
    int64_t blocks = 0;
    int used = 0;
    auto launch = [&]() -> hipError_t {
        if (used == 0) return hipSuccess;
        transpose_u8_kernel<<<dim3((unsigned)blocks), 256, 0, s>>>(a);
        a = {};
        blocks = used = 0;
        return hipGetLastError();
    };
    for (int i = 0; i < n && i < 2; ++i) {
        const TransposeJob &j = jobs[i];
        const int64_t nbc = (j.C + kTB - 1) / kTB, nbr = (j.R + kTB - 1) / kTB, mine = nbc * nbr * j.batch;
        if (mine == 0) continue;
        if (mine >= kTransposeMaxBlocks) return hipErrorInvalidValue;   // checked by the caller
        if (blocks + mine >= kTransposeMaxBlocks) {
            const hipError_t e = launch();
            if (e != hipSuccess) return e;
        }
        a.job[used] = j;
        a.nbc[used] = (uint32_t)nbc;
        a.per[used] = (uint32_t)(nbc * nbr);
        blocks += mine;
        if (used == 0) a.first = (uint32_t)blocks;
        ++used;
    }
    return launch();
}

}  // namespace spg
