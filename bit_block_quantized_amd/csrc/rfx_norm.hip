// The residual's addition, the RMS norm of the sum and the 8-bit activations
// of the normalised row, in one pass:
//
//   h = x + delta,   y = h w / sqrt(mean(h^2) + eps),
//   per 32 elements: s = max |y| (1 / 127), code = round(y / s), sum of codes.
//
// Bound by memory where there are many rows: 4099 rows of 7168 with delta, weight
// and all outputs take 104 us, 507 MB at 4.9 TB/s (a large copy has 4.8, a read
// of 235 MB and a write of 272 one after the other would take 108). One row of
// 4096, and four of 7168, take 3.7, mostly the launch. Each row is read once and
// held in the registers of one workgroup, four elements of every THREADS * 4
// per thread, until its sum of squares is known. The sum, the root and the products are fp64 (the vector
// pipe's fp64 rate is its fp32 rate, and there are some 60 operations to
// spare per element): y is then the fp32 number next to the exact value but
// for one in 2^28, and the codes do not depend on the order of the sum.
// Eight neighbouring lanes hold a block of 32, so its maximum and its sum of
// codes are lane exchanges of the vector pipe.
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "rfx.h"
#include "rfx_internal.h"

using namespace rfx;

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxCols = 1 << 20;
constexpr int kMaxNormRows = 1 << 21; // of 1024 threads: below 2^32

// Over the eight lanes of a block: neighbours, pairs, and i against 7 - i.
template <class Op>
__device__ __forceinline__ int block8(int v, Op op)
{
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xf, 0xf, true));  // lanes 1 0 3 2
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xf, 0xf, true));  // lanes 2 3 0 1
    return op(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, true)); // 7 - i of 8
}

struct RowOut {
    float *sum, *y;
    uint32_t *xq;
    float *xs;
    int32_t *xsum;
};

// Four elements of one block in each of its eight lanes to codes, scale and
// sum. The scale is by definition a product, within a step of the quotient that
// rfx_quantize_act takes (about one scale in twenty is that step off); the codes'
// division is IEEE's. Magnitudes are compared as whole numbers, which order as
// they do and have NaN above all, so that a NaN is its block's scale. i4: the
// four's index in its row.
__device__ __forceinline__ void quantize4(const f32x4 y, int i4, const RowOut &o)
{
#pragma clang fp contract(off)
    int a = 0;
#pragma unroll
    for (int k = 0; k < 4; k++)
        a = max(a, __float_as_int(fabsf(y[k])));
    a = block8(a, [](int p, int q) { return max(p, q); });
    const float s = __int_as_float(a) * (1.0f / 127.0f);
    uint32_t packed = 0u;
    int sum = 0;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        int c = 0;
        if (s != 0.0f)
            c = (int)fminf(fmaxf(rintf(y[k] / s), -127.0f), 127.0f);
        sum += c;
        packed |= ((uint32_t)c & 0xffu) << (8 * k);
    }
    sum = block8(sum, [](int p, int q) { return p + q; });
    o.xq[i4] = packed;
    if ((threadIdx.x & 7) == 0) {
        o.xs[i4 >> 3] = s;
        o.xsum[i4 >> 3] = sum;
    }
}

// The fp32 number next to h w r.
__device__ __forceinline__ f32x4 scaled(const f32x4 h, const f32x4 w, double r)
{
    f32x4 y;
#pragma unroll
    for (int k = 0; k < 4; k++)
        y[k] = (float)((double)h[k] * (double)w[k] * r);
    return y;
}

// One workgroup per row. NV: fours per thread, or 0 for rows that the
// registers do not hold: those are read twice.
template <int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void norm_kernel(rfx_norm a)
{
    constexpr int N = NV ? NV : 1, WAVES = THREADS / 64;
    __shared__ double part[WAVES];
    const int tid = threadIdx.x, n4 = a.cols / 4;
    const size_t row = blockIdx.x;
    const f32x4 *x = reinterpret_cast<const f32x4 *>(a.x + (int64_t)row * a.x_stride);
    const f32x4 *d = reinterpret_cast<const f32x4 *>(a.delta ? a.delta + (int64_t)row * a.delta_stride : nullptr);
    const f32x4 *w = reinterpret_cast<const f32x4 *>(a.weight);
    const f32x4 one = {1.f, 1.f, 1.f, 1.f}, zero = {0.f, 0.f, 0.f, 0.f};
    const auto fetch = [&](int i) { return d ? x[i] + d[i] : x[i]; };

    f32x4 h[N], wv[N];
    double ss = 0.0;
    const auto add = [&](const f32x4 &v) {
#pragma unroll
        for (int k = 0; k < 4; k++)
            ss = fma((double)v[k], (double)v[k], ss);
    };
    if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int i = tid + j * THREADS;
            h[j] = i < n4 ? fetch(i) : zero;
        }
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int i = tid + j * THREADS;
            wv[j] = w && i < n4 ? w[i] : one;
        }
#pragma unroll
        for (int j = 0; j < NV; j++)
            add(h[j]);
    } else {
        for (int i = tid; i < n4; i += THREADS)
            add(fetch(i));
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        ss += __shfl_xor(ss, o, 64);
    if ((tid & 63) == 0)
        part[tid >> 6] = ss;
    __syncthreads();
    ss = 0.0;
#pragma unroll
    for (int i = 0; i < WAVES; i++)
        ss += part[i];
    const double ms = ss / a.cols + (double)a.eps;
    const double r = ms == 0.0 ? 0.0 : 1.0 / sqrt(ms); // a row of zeros stays one, a NaN spreads

    const size_t at = row * (size_t)a.cols;
    const RowOut o = {a.sum ? a.sum + at : nullptr, a.y ? a.y + at : nullptr, reinterpret_cast<uint32_t *>(a.xq ? a.xq + at : nullptr),
                      a.xq ? a.xs + at / 32 : nullptr, a.xq ? a.xsum + at / 32 : nullptr};
    const auto finish = [&](int i, const f32x4 &hv, const f32x4 &wi) {
        if (o.sum)
            reinterpret_cast<f32x4 *>(o.sum)[i] = hv;
        const f32x4 y = scaled(hv, wi, r);
        if (o.y)
            reinterpret_cast<f32x4 *>(o.y)[i] = y;
        if (o.xq)
            quantize4(y, i, o);
    };
    if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int i = tid + j * THREADS;
            if (i < n4) // whole blocks: n4 and THREADS are multiples of 8
                finish(i, h[j], wv[j]);
        }
    } else {
        for (int i = tid; i < n4; i += THREADS)
            finish(i, fetch(i), w ? w[i] : one);
    }
}

template <int THREADS>
void launch(const rfx_norm &a, hipStream_t st)
{
    const int per = (a.cols / 4 + THREADS - 1) / THREADS;
    const dim3 grid(a.q), block(THREADS);
#define RFX_NORM(NV) hipLaunchKernelGGL((norm_kernel<THREADS, NV>), grid, block, 0, st, a)
    if (per <= 1)
        RFX_NORM(1);
    else if (per <= 2)
        RFX_NORM(2);
    else if (per <= 4)
        RFX_NORM(4);
    else if (per <= 8)
        RFX_NORM(8);
    else
        RFX_NORM(0);
#undef RFX_NORM
}

} // namespace

extern "C" int rfx_add_rms_norm(const rfx_norm *A, void *stream)
{
    if (!A)
        return fail(RFX_E_INVAL, "rfx_add_rms_norm: arguments are NULL");
    if (A->q < 0 || A->q > kMaxNormRows || A->cols < 32 || A->cols % 32 || A->cols > kMaxCols)
        return fail(RFX_E_INVAL, "rfx_add_rms_norm: q=%d cols=%d (at most %d rows of a multiple of 32, at most %d)", A->q,
                    A->cols, kMaxNormRows, kMaxCols);
    if (!(A->eps >= 0.0f) || A->eps > 1e30f)
        return fail(RFX_E_INVAL, "rfx_add_rms_norm: eps=%g", (double)A->eps);
    const struct {
        int64_t stride;
        const void *p;
        const char *name;
    } rows[2] = {{A->x_stride, A->x, "x"}, {A->delta_stride, A->delta, "delta"}};
    for (const auto &r : rows)
        if (r.p && (r.stride < A->cols || r.stride % 4 || r.stride > (int64_t)1 << 40))
            return fail(RFX_E_INVAL, "rfx_add_rms_norm: %s_stride=%lld (a multiple of 4, at least cols)", r.name, (long long)r.stride);
    if (!A->sum && !A->y && !A->xq)
        return fail(RFX_E_INVAL, "rfx_add_rms_norm: no output");
    if (A->sum && A->sum == A->y)
        return fail(RFX_E_INVAL, "rfx_add_rms_norm: sum and y are one buffer");
    int st = check_ptr(A->x, 16, "x");
    if (st || (A->delta && (st = check_ptr(A->delta, 16, "delta"))) || (A->weight && (st = check_ptr(A->weight, 16, "weight"))) ||
        (A->sum && (st = check_ptr(A->sum, 16, "sum"))) || (A->y && (st = check_ptr(A->y, 16, "y"))))
        return st;
    if (A->xq && ((st = check_ptr(A->xq, 16, "xq")) || (st = check_ptr(A->xs, 4, "xs")) || (st = check_ptr(A->xsum, 4, "xsum"))))
        return st;
    if (A->q == 0)
        return RFX_OK;
    // Few rows: a row over 16 waves, so that each thread has few elements;
    // many rows: four waves, whose rows are in flight beside others'.
    if (A->q < 512 || A->cols > 256 * 4 * 8)
        launch<1024>(*A, (hipStream_t)stream);
    else
        launch<256>(*A, (hipStream_t)stream);
    return hip_status("add_rms_norm launch");
}
