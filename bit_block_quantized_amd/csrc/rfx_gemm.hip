// Packed product with bias, activation and residual in its epilogue:
// y = resid + act(W x + bias) for q columns. One to four columns take the
// GEMV kernels (rfx_gemv.hip), FP4 with more the block-scaled matrix core
// (rfx_gemm_mx.hip); this file has the entry points and the form for more
// columns of FP2 and FP3, whose f16 block scales no matrix core applies.
//
// Per 32-weight block the product is the exact integer block dot D on
// v_mfma_f32_16x16x32_f16 (both sides' codes as f16, sums below 2^24), then
// acc += D * (weight scale * activation scale) in fp32, as in the prefill
// FFN. A 16 x 16 block product takes the matrix pipe 16 cycles and its scale
// products (v_mfma_f32_4x4x1) 8, beside 16 cycles of fused multiply-adds and
// the weights' decode on the vector pipe. Neither pipe is full: by counters
// the vector pipe is busy 56 % of the time, the matrix pipe 38 %, LDS 19 %, so
// the two waves of a SIMD mostly take turns. A wave takes two 16-row weight
// tiles, decoded in registers, against up to eight 16-column tiles: the decode
// (about 15 operations per weight tile and block) is spread over the columns,
// and each column fragment read from LDS serves two products. A workgroup of
// eight waves covers 256 rows and up to 128 columns; per 256-element K tile its
// column fragments arrive in LDS by direct loads from a copy of the codes in
// fragment order, made by a first launch ([column tile][block][lane] x 16
// bytes of f16, zero past q and K, so the loop has no bounds to check). 2048
// columns of 4096 x 7168: 210 us for FP2, 209 for FP3 (575 TFLOP/s).
// Few row and column blocks: K is split over workgroups, and a last launch
// adds the partials in split order and applies the epilogue.
#include "rfx_gemm.h"

using namespace rfx;
using namespace rfx::dev;

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int M = 2;                      // 16-row weight tiles per wave
constexpr int kRows = 16 * M * kWaves;    // rows per workgroup

// Scales of a block in LDS: whole direct loads of 64 lanes.
template <int NT>
constexpr int kScaleRow = NT < 4 ? 64 : 16 * NT;

// One wave per (column tile, block): the codes of 16 columns as the A operand
// (lane l: column l % 16, elements 8 (l / 16) .. + 7 of the block).
__global__ __launch_bounds__(256) void gemm_columns_kernel(const int8_t *xq, const float *xs, int q, int nb, int nbp,
                                                           int qp, uint8_t *xh, float *sx)
{
    const int lane = threadIdx.x & 63;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int b = (int)(id % nbp), tt = (int)(id / nbp);
    if (16 * tt >= qp)
        return;
    const int col = 16 * tt + (lane & 15), g = lane >> 4;
    const bool ok = col < q && b < nb;
    u32x2 c = {0u, 0u};
    if (ok)
        c = *reinterpret_cast<const u32x2 *>(xq + ((size_t)col * nb + b) * 32 + 8 * g);
    uint32_t f[4];
    i8x4_to_f16(c.x, f[0], f[1]);
    i8x4_to_f16(c.y, f[2], f[3]);
    *reinterpret_cast<u32x4 *>(xh + ((size_t)id * 64 + lane) * 16) = (u32x4){f[0], f[1], f[2], f[3]};
    if (g == 0)
        sx[(size_t)b * qp + col] = ok ? xs[(size_t)col * nb + b] : 0.0f;
}

// One half K tile (four blocks): the wave's weights w against the NT column
// tiles in LDS. The products of column tile tt are issued before those of tt
// - 1 are scaled, and tt + 1's operands are read meanwhile. after_first runs
// once the first block has its weights.
template <int F, int NT, class Hook>
__device__ __forceinline__ void gemm_half(const WHalf<F> (&w)[M], const char *frag, const char *lsx, int hf,
                                          float (&acc)[M][NT][4], Hook &&after_first)
{
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    const u32x4 *fr = reinterpret_cast<const u32x4 *>(frag) + lane;
    const float *sxl = reinterpret_cast<const float *>(lsx) + 4 * g + (lane & 3);
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int b = 4 * hf + j;
        u32x4 av = fr[b * 64];
        float sa = sxl[b * kScaleRow<NT>];
        f16x8 wv[M];
        float sw[M];
#pragma unroll
        for (int m = 0; m < M; m++) {
            wv[m] = wfrag<F>(w[m], j, g);
            sw[m] = wscale<F>(w[m], j);
        }
        if (j == 0) {
            __builtin_amdgcn_sched_barrier(0);
            after_first();
            __builtin_amdgcn_sched_barrier(0);
        }
        f32x4 dp[M];
        float sp = 0.f;
#pragma unroll
        for (int tt = 0; tt <= NT; tt++) {
            f32x4 dc[M];
            float sc_n = sa;
            if (tt < NT) {
#pragma unroll
                for (int m = 0; m < M; m++)
                    dc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, av), wv[m], zero, 0, 0, 0);
            }
            if (tt + 1 < NT) {
                av = fr[((tt + 1) * 8 + b) * 64];
                sa = sxl[b * kScaleRow<NT> + 16 * (tt + 1)];
            }
            if (tt > 0) {
#pragma unroll
                for (int m = 0; m < M; m++) {
                    // output lane l, register v: A(lane 4 (l / 4) + v) * B(lane l),
                    // the product's layout of column scale * row scale
                    const f32x4 sc = __builtin_amdgcn_mfma_f32_4x4x1f32(sp, sw[m], zero, 0, 0, 0);
#pragma unroll
                    for (int v = 0; v < 4; v++)
                        acc[m][tt - 1][v] = fmaf(dp[m][v], sc[v], acc[m][tt - 1][v]);
                }
            }
            if (tt < NT) {
#pragma unroll
                for (int m = 0; m < M; m++)
                    dp[m] = dc[m];
                sp = sc_n;
            }
        }
    }
}

template <int F, int NT>
__global__ __launch_bounds__(kThreads, NT == 4 ? 4 : 2) void gemm_kernel(GemmArgs a)
{
    constexpr int TB = TileFmt<F>::bytes, COLS = 16 * NT;
    constexpr int kFrag = NT * 8 * 1024, kSx = 8 * kScaleRow<NT> * 4;
    __shared__ __align__(16) char smem[2 * (kFrag + kSx)];
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    GemmBlock blk;
    if (!gemm_block(a, blk))
        return;
    const int rb = blk.rb, cb = blk.cb, s_begin = blk.s_begin, s_end = blk.s_end;

    const int row0 = rb * kRows + 16 * M * wave;
    const uint8_t *tb[M];
    int rin[M];
#pragma unroll
    for (int m = 0; m < M; m++) {
        const int rr = row0 + 16 * m < a.N ? row0 + 16 * m : 0; // rows past N: any rows, never stored
        tb[m] = a.W + (size_t)(rr >> 6) * a.S * TB;
        rin[m] = (rr & 63) + (lane & 15);
    }
    const int nbp = 8 * a.S;
    // wave w stages block w of a K tile: the fragments of the column tiles
    // and the columns' scales
    const auto stage = [&](int s, int buf) {
        const int b = 8 * s + wave;
        char *fb = smem + buf * (kFrag + kSx), *sb = fb + kFrag;
#pragma unroll
        for (int tt = 0; tt < NT; tt++)
            lds_dma16(a.xh + (((size_t)(cb * NT + tt) * nbp + b) * 64 + lane) * 16, fb + (tt * 8 + wave) * 1024);
        const float *sr = static_cast<const float *>(a.sx) + (size_t)b * a.qp + cb * COLS;
#pragma unroll
        for (int i = 0; i < kScaleRow<NT> / 64; i++) // fewer than 64 columns: some lanes read theirs again
            lds_dma4(sr + (64 * i + lane) % COLS, sb + (wave * kScaleRow<NT> + 64 * i) * 4);
    };

    float acc[M][NT][4] = {};
    WHalf<F> wa[M], wb[M];
#pragma unroll
    for (int m = 0; m < M; m++)
        wa[m] = load_whalf<F>(tb[m] + (size_t)s_begin * TB, rin[m], g, 0);
    stage(s_begin, 0);
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
    int buf = 0;
    for (int s = s_begin; s < s_end; s++, buf ^= 1) {
        const char *frag = smem + buf * (kFrag + kSx), *lsx = frag + kFrag;
        const int sn = s + 1 < s_end ? s + 1 : s;
#pragma unroll
        for (int m = 0; m < M; m++)
            wb[m] = load_whalf<F>(tb[m] + (size_t)s * TB, rin[m], g, 1);
        gemm_half<F, NT>(wa, frag, lsx, 0, acc, [] {});
        __builtin_amdgcn_s_waitcnt(0x0F70); // wb: the only loads in flight
        gemm_half<F, NT>(wb, frag, lsx, 1, acc, [&] {
            stage(sn, buf ^ 1);
#pragma unroll
            for (int m = 0; m < M; m++)
                wa[m] = load_whalf<F>(tb[m] + (size_t)sn * TB, rin[m], g, 0);
        });
        // the next tile has landed in every wave's LDS before any reads it
        __builtin_amdgcn_s_waitcnt(0x0F70);
        __syncthreads();
    }
    // the results through the loop's buffers
    constexpr int OP = kRows + 4;
    static_assert(COLS * OP * 4 <= 2 * (kFrag + kSx), "results fit the loop's buffers");
    float *o = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int m = 0; m < M; m++)
#pragma unroll
        for (int tt = 0; tt < NT; tt++)
#pragma unroll
            for (int v = 0; v < 4; v++)
                o[(16 * tt + 4 * g + v) * OP + 16 * M * wave + 16 * m + (lane & 15)] = acc[m][tt][v];
    __syncthreads();
    store_block<kRows, COLS, kWaves>(a, blk, o);
}

// Adds the splits' partials in order and applies the epilogue: four rows of
// one column per thread.
__global__ __launch_bounds__(256) void gemm_join_kernel(GemmArgs a)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= (int64_t)a.q * a.N4)
        return;
    const int col = (int)(i / a.N4), row = (int)(i % a.N4);
    const float *p = a.part + (size_t)col * a.N4 + row;
    const size_t stride = (size_t)a.q * a.N4;
    f32x4 sum = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll 4
    for (int s = 1; s < a.splits; s++)
        sum += *reinterpret_cast<const f32x4 *>(p + s * stride);
    if (a.epi.bias)
#pragma unroll
        for (int v = 0; v < 4; v++)
            sum[v] += a.epi.bias[min(row + v, a.N - 1)];
    const int left = a.N - row;
    finish_rows(a, sum, col, row, left, left >= 4 && a.vec);
}

// The first kGemvSlotBytes of a workspace belong to the GEMV form's exchange
// slots, which every call leaves zero; the rest needs no initialisation.

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

struct Plan {
    GemmShape g;
    int row_blocks, col_blocks, splits, qp, N4;
    size_t xh, sx, part, bytes;
};

// Columns per workgroup: the fewest 16-column tiles (1, 2, 4 or 8) that take
// all columns, so that few columns keep registers and LDS for more
// workgroups; fewer where even one K tile each would leave a quarter of the
// compute units idle (us, fewer and fewest: FP3 1024 x 1024 with 64 and 200
// columns 12.0 and 15.7, 13.3 and 18.7; FP4 2048 x 2048 with 64 12.0 and
// 15.6; FP3 7168 x 2048 with 32, 224 workgroups, 18.7 and 15.8). K is split until every compute unit has one workgroup (two
// below eight tiles), down to one K tile each, FP4 to two where it has more
// than four: in us, one and two tiles each, FP3 1024 x 1024 with 6 and 200
// columns 11.4 and 13.3, 18.7 and 23.9, 4096 x 4096 with 64 22.8 and 24.4;
// FP4 1024 x 1024 with 64 12.9 and 14.2, but 4096 x 4096 with 64 20.1 and 18.4.
GemmShape f16_shape(int64_t N, int64_t S, int tiles)
{
    int nt = tiles <= 1 ? 1 : tiles <= 2 ? 2 : tiles <= 4 ? 4 : 8;
    while (nt > 1 && ceil_div(N, kRows) * ceil_div(tiles, nt) * S < 192)
        nt /= 2;
    return {kRows, nt, 8 * 1024, 8 * 64, nt == 8 ? 256 : 512};
}

Plan plan(int fmt, int64_t N, int64_t K, int q)
{
    Plan p{};
    const int tiles = (q + 15) / 16;
    const int64_t S = ceil_div(K, kTileCols);
    p.g = fmt == RFX_FP4 ? gemm_mx_shape(N, S, tiles) : f16_shape(N, S, tiles);
    p.row_blocks = (int)ceil_div(N, p.g.rows);
    p.col_blocks = (tiles + p.g.tiles - 1) / p.g.tiles;
    p.qp = p.col_blocks * p.g.tiles * 16;
    const int64_t blocks = (int64_t)p.row_blocks * p.col_blocks;
    int64_t splits = p.g.want / blocks;
    const int64_t most = fmt == RFX_FP4 && S > 4 ? S / 2 : S;
    splits = splits > most ? most : splits;
    p.splits = (int)(splits < 1 ? 1 : splits);
    p.N4 = (int)((N + 3) / 4 * 4);
    p.xh = align256((size_t)(p.qp / 16) * S * p.g.frag);
    p.sx = align256((size_t)(p.qp / 16) * S * p.g.scale);
    p.part = p.splits > 1 ? align256((size_t)p.splits * q * p.N4 * 4) : 0;
    p.bytes = kGemvSlotBytes + p.xh + p.sx + p.part;
    return p;
}

bool many_ok(int fmt) { return fmt == RFX_FP2 || fmt == RFX_FP3 || fmt == RFX_FP4; }

// What the kernels' 32-bit row numbers (rounded up to whole workgroups) and K
// tile numbers (times up to 512 splits) hold.
bool small_enough(const rfx_qmat *W) { return W->rows <= 1 << 30 && W->cols <= 1 << 29; }

template <int F>
int launch(const GemmArgs &a, int nt, const int8_t *xq, const float *xs, int nb, hipStream_t st)
{
    const int64_t frags = (int64_t)(a.qp / 16) * 8 * a.S;
    hipLaunchKernelGGL(gemm_columns_kernel, dim3((unsigned)((frags + 3) / 4)), dim3(256), 0, st, xq, xs, a.q, nb, 8 * a.S,
                       a.qp, const_cast<uint8_t *>(a.xh), static_cast<float *>(const_cast<void *>(a.sx)));
    const int err = hip_status("gemm columns launch");
    if (err)
        return err;
    const int n = a.row_blocks * a.col_blocks * a.splits;
    const dim3 grid((n + 7) / 8 * 8), block(kThreads);
    switch (nt) {
    case 1: hipLaunchKernelGGL((gemm_kernel<F, 1>), grid, block, 0, st, a); break;
    case 2: hipLaunchKernelGGL((gemm_kernel<F, 2>), grid, block, 0, st, a); break;
    case 4: hipLaunchKernelGGL((gemm_kernel<F, 4>), grid, block, 0, st, a); break;
    default: hipLaunchKernelGGL((gemm_kernel<F, 8>), grid, block, 0, st, a); break;
    }
    return hip_status("gemm launch");
}

} // namespace

extern "C" {

size_t rfx_gemm_workspace_bytes(const rfx_qmat *W, int q)
{
    if (!W || !fmt_ok(W->fmt) || W->rows < 1 || W->cols < 32 || W->cols % 32 || q < 1 || q > RFX_GEMM_MAX_Q)
        return 0;
    if (q <= 4)
        return rfx_gemv_workspace_bytes(W, q);
    return many_ok(W->fmt) && small_enough(W) ? plan(W->fmt, W->rows, W->cols, q).bytes : 0;
}

int rfx_gemm(const rfx_qmat *W, const int8_t *xq, const float *xs, const int32_t *xsum, int q, const float *bias, int act,
             const float *resid, float *y, void *ws, size_t ws_bytes, void *stream)
{
    int st = check_qmat(W, "W", false);
    if (st)
        return st;
    if (q < 1 || q > RFX_GEMM_MAX_Q)
        return fail(RFX_E_INVAL, "rfx_gemm: q=%d (1..%d)", q, RFX_GEMM_MAX_Q);
    if (act < RFX_ACT_NONE || act > RFX_ACT_GELU_TANH)
        return fail(RFX_E_INVAL, "rfx_gemm: act=%d", act);
    if ((st = check_ptr(xq, 16, "xq")) || (st = check_ptr(xs, 4, "xs")) || (st = check_ptr(xsum, 4, "xsum")) ||
        (st = check_ptr(y, 4, "y")) || (bias && (st = check_ptr(bias, 4, "bias"))) ||
        (resid && (st = check_ptr(resid, 4, "resid"))))
        return st;
    if (q > 4 && !many_ok(W->fmt))
        return fail(RFX_E_UNSUPPORTED, "rfx_gemm: format %d with more than 4 columns (FP2, FP3 and FP4 only)", W->fmt);
    if (q > 4 && !small_enough(W))
        return fail(RFX_E_UNSUPPORTED, "rfx_gemm: %d x %d with more than 4 columns (at most 2^30 rows, 2^29 columns of W)",
                    W->rows, W->cols);
    const size_t need = rfx_gemm_workspace_bytes(W, q);
    if (need) {
        if (!ws || ws_bytes < need)
            return fail(RFX_E_WORKSPACE, "rfx_gemm: workspace %zu < %zu bytes", ws ? ws_bytes : (size_t)0, need);
        if ((st = check_ptr(ws, 256, "ws")))
            return st;
    }
    const EpiArgs e{bias, resid, act};
    const hipStream_t hs = (hipStream_t)stream;
    if (q <= 4)
        return gemv_epi(W, xq, xs, xsum, q, e, y, ws, hs);

    const Plan p = plan(W->fmt, W->rows, W->cols, q);
    GemmArgs a{};
    a.W = static_cast<const uint8_t *>(W->data);
    a.N = W->rows;
    a.S = (int)ceil_div(W->cols, kTileCols);
    a.q = q;
    a.row_blocks = p.row_blocks;
    a.col_blocks = p.col_blocks;
    a.splits = p.splits;
    a.qp = p.qp;
    a.N4 = p.N4;
    char *w = static_cast<char *>(ws) + kGemvSlotBytes;
    a.xh = reinterpret_cast<const uint8_t *>(w);
    a.sx = w + p.xh;
    a.part = reinterpret_cast<float *>(w + p.xh + p.sx);
    a.y = y;
    a.epi = e;
    a.vec = W->rows % 4 == 0 && !((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(resid)) & 15);
    const int nb = W->cols / 32;
    if (W->fmt == RFX_FP4)
        st = gemm_mx_launch(a, p.g, xq, xs, nb, hs);
    else
        st = W->fmt == RFX_FP2 ? launch<RFX_FP2>(a, p.g.tiles, xq, xs, nb, hs) : launch<RFX_FP3>(a, p.g.tiles, xq, xs, nb, hs);
    if (st || p.splits == 1)
        return st;
    const int64_t quads = (int64_t)q * p.N4 / 4;
    hipLaunchKernelGGL(gemm_join_kernel, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, hs, a);
    return hip_status("gemm join launch");
}

} // extern "C"
