// Packed product for many columns: what its two kernels share (rfx_gemm.hip,
// FP2 and FP3 on the f16 matrix core; rfx_gemm_mx.hip, FP4 on the
// block-scaled one).
#pragma once

#include "rfx_epi.h"
#include "rfx_internal.h"
#include "rfx_wfrag.h"

namespace rfx {

struct GemmArgs {
    const uint8_t *W;
    int N, S, q;         // rows, K tiles of 256, columns
    int row_blocks, col_blocks, splits;
    const uint8_t *xh;   // the columns as operands, see the kernels
    const void *sx;      // ... and their scales
    int qp;              // columns padded to whole column blocks
    float *y;            // [q][N]
    float *part;         // [split][q][N4] where splits > 1
    int N4;
    bool vec;            // y and resid rows are 16-byte aligned
    EpiArgs epi;
};

// Rows and columns of a workgroup, bytes of the columns' operands and of
// their scales per 16 columns and K tile, workgroups to aim at.
struct GemmShape {
    int rows, tiles, frag, scale, want;
};
GemmShape gemm_mx_shape(int64_t N, int64_t S, int tiles);

int gemm_mx_launch(const GemmArgs &a, const GemmShape &g, const int8_t *xq, const float *xs, int nb, hipStream_t st);

namespace dev {

typedef float f32x4 __attribute__((ext_vector_type(4)));

struct GemmBlock {
    int rb, cb, sp, s_begin, s_end;
};

// Workgroups go round the eight XCDs in order; give each XCD a contiguous
// run of blocks, rows fastest within a split, so that its L2 keeps the run's
// columns. False: none left.
__device__ __forceinline__ bool gemm_block(const GemmArgs &a, GemmBlock &b)
{
    const int n = a.row_blocks * a.col_blocks * a.splits;
    const int per = (n + 7) / 8;
    const int id = blockIdx.x % 8 * per + blockIdx.x / 8;
    if (id >= n)
        return false;
    b.rb = id % a.row_blocks;
    b.cb = id / a.row_blocks % a.col_blocks;
    b.sp = id / (a.row_blocks * a.col_blocks);
    b.s_begin = a.S * b.sp / a.splits;
    b.s_end = a.S * (b.sp + 1) / a.splits;
    return true;
}

// Four rows of one column, bias added, to y.
__device__ __forceinline__ void finish_rows(const GemmArgs &a, f32x4 z, int col, int row, int left, bool quad)
{
    const size_t at = (size_t)col * a.N + row;
    f32x4 r = {0.f, 0.f, 0.f, 0.f};
    if (a.epi.resid) {
        if (quad) {
            r = *reinterpret_cast<const f32x4 *>(a.epi.resid + at);
        } else {
#pragma unroll
            for (int v = 0; v < 4; v++)
                if (v < left)
                    r[v] = a.epi.resid[at + v];
        }
    }
#pragma unroll
    for (int v = 0; v < 4; v++)
        z[v] = activate(z[v], a.epi.act) + r[v];
    if (quad) {
        *reinterpret_cast<f32x4 *>(a.y + at) = z;
    } else {
#pragma unroll
        for (int v = 0; v < 4; v++)
            if (v < left)
                a.y[at + v] = z[v];
    }
}

// A workgroup's results, o[column][row] in LDS at a pitch of ROWS + 4 (which
// puts the four column groups of a store on different banks), to y or to the
// split's partials: bias, residual and result are read and written four rows
// a lane, whole lines at a time. Wave w takes columns w, w + WAVES, ...
template <int ROWS, int COLS, int WAVES>
__device__ __forceinline__ void store_block(const GemmArgs &a, const GemmBlock &b, const float *o)
{
    constexpr int OP = ROWS + 4;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c_end = min(COLS, a.q - b.cb * COLS);
#pragma unroll
    for (int r = 4 * lane; r < ROWS; r += 256) {
        const int row = b.rb * ROWS + r, left = a.N - row;
        if (left <= 0)
            return;
        if (a.splits > 1) {
            for (int c = wave; c < c_end; c += WAVES) // rows up to N4 exist
                *reinterpret_cast<f32x4 *>(a.part + ((size_t)b.sp * a.q + b.cb * COLS + c) * a.N4 + row) =
                    *reinterpret_cast<const f32x4 *>(o + c * OP + r);
            continue;
        }
        const bool quad = left >= 4 && a.vec; // four rows at a time, 16-byte aligned
        f32x4 bias = {0.f, 0.f, 0.f, 0.f};
        if (a.epi.bias)
#pragma unroll
            for (int v = 0; v < 4; v++)
                bias[v] = a.epi.bias[min(row + v, a.N - 1)];
#pragma unroll 4
        for (int c = wave; c < c_end; c += WAVES) {
            const f32x4 z = *reinterpret_cast<const f32x4 *>(o + c * OP + r) + bias;
            finish_rows(a, z, b.cb * COLS + c, row, left, quad);
        }
    }
}

} // namespace dev
} // namespace rfx
