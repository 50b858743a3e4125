// Packed FP4 product for more than four columns, y = resid + act(W x + bias),
// on v_mfma_scale_f32_16x16x128_f8f6f4.
//
// The matrix core takes the packed E2M1 weights as they are stored and
// applies their e8m0 exponents, so nothing is decoded. The other operand's
// scales are powers of two as well, but a column's block scale is any fp32
// number; so a column enters as five FP6 (E2M3) digits:
//   code * scale = 2^E (d0 + 2^-4 d1 + 2^-9 d2 + 2^-14 d3 + 2^-19 d4) + r,
// each digit the E2M3 value nearest to what is left (halves of its steps
// times 2^4, then 2^5, stay within its range), E the exponent that puts the
// block's largest value into (3.75, 7.5]. |r| <= 2^(E - 22), 2^-23.9 of that
// largest value: as much as fp32 rounds it by. Four digits would be 1.25
// times as fast in the loop, with 2^-19 of it.
// The ten products of a K tile (five digits, two half tiles) are summed from
// zero, the smallest digits first, and added to the accumulator in fp32: an
// output rounds once per 256 weights, where the f16 form rounds once per 32.
//
// Bound by the power of the matrix core: random operands run this instruction
// at 5.5 to 6.2 PFLOP/s here (zeros at 8 to 9), which is 100 us for the five
// digits of 2048 columns of 4096 x 7168; then by the columns' way from L2
// through LDS. Measured there: 164 to 168 us in all (730 TFLOP/s of the
// product), 16 of them for the columns' launch and about 12 for bias,
// residual and result; with the loop's loads left out 143, its LDS reads too
// 134. The f16 form, which decodes weights and scales every block's product,
// took 192 to 212.
//
// A wave takes RT 16-row tiles of W, read once from memory into registers a
// K tile ahead, against CT 16-column tiles of digits in LDS, 24 bytes a lane
// for RT products. Eight waves (two per SIMD) with 64 columns: one wave per
// SIMD with twice the rows reads half as much LDS but took 190.

#include "rfx_gemm.h"
#include "rfx_mx4.h"

using namespace rfx;
using namespace rfx::dev;

namespace {

typedef uint32_t u32x6 __attribute__((ext_vector_type(6)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x32 __attribute__((ext_vector_type(32)));

constexpr int kDigits = 5;
// Bytes of a column tile's digits in a K tile: per half tile h and digit d
// the first 16 bytes of all lanes, then, after all of those, the last 8.
constexpr int kFrags = 2 * kDigits, kTail = kFrags * 1024, kFragBytes = kFrags * 1536;
constexpr int kScaleBytes = 128; // per lane two scale bytes, h = 0 and 1
constexpr int kOff[kDigits] = {0, 4, 9, 14, 19};

// One wave per (column tile, K tile, half h): lane l has block 2 (l / 16) + h
// of column l % 16. Zero past q and K.
__global__ __launch_bounds__(256) void mx_columns_kernel(const int8_t *xq, const float *xs, int q, int nb, int S, int n,
                                                         uint8_t *xh, uint8_t *sx)
{
    const int lane = threadIdx.x & 63;
    const int id = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (id >= n)
        return;
    const int h = id & 1, ts = id >> 1, tt = ts / S, s = ts - tt * S;
    const int col = 16 * tt + (lane & 15), b = 8 * s + 2 * (lane >> 4) + h;
    const bool ok = col < q && b < nb;
    u32x4 c0 = {0u, 0u, 0u, 0u}, c1 = {0u, 0u, 0u, 0u};
    float x = 0.f;
    if (ok) {
        const size_t at = (size_t)col * nb + b;
        c0 = *reinterpret_cast<const u32x4 *>(xq + at * 32);
        c1 = *reinterpret_cast<const u32x4 *>(xq + at * 32 + 16);
        x = xs[at];
    }
    // Even nibbles of a code word hold weights 8g + 0..3, odd ones 8g + 4..7;
    // the conversion interleaves its two operands alike.
    f32x16 v[2];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t w = i < 4 ? c0[i] : c1[i - 4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float f = (float)(int8_t)(w >> (8 * j));
            v[i & 1][4 * (i >> 1) + j] = f;
            top = fmaxf(top, fabsf(f));
        }
    }
    const uint32_t tb = __float_as_uint(top * fabsf(x)); // NaN and infinities: the scale that means NaN
    const int e = (int)(tb >> 23), E = e == 255 ? 255 : max(e - 2 + ((tb & 0x7FFFFFu) > 0x700000u ? 1 : 0), kOff[kDigits - 1]);
    const float unit = ldexpf(x, 127 - E);
    v[0] *= unit;
    v[1] *= unit;
    uint8_t *out = xh + (size_t)ts * kFragBytes;
#pragma unroll
    for (int d = 0; d < kDigits; d++) {
        const u32x6 f = __builtin_amdgcn_cvt_scalef32_2xpk16_fp6_f32(v[0], v[1], 1.0f);
        const int fr = h * kDigits + d;
        *reinterpret_cast<u32x4 *>(out + fr * 1024 + lane * 16) = (u32x4){f[0], f[1], f[2], f[3]};
        *reinterpret_cast<u32x2 *>(out + kTail + fr * 512 + lane * 8) = (u32x2){f[4], f[5]};
        if (d + 1 < kDigits) {
            const f32x32 back = __builtin_amdgcn_cvt_scalef32_pk32_f32_fp6(f, 1.0f);
            const float up = d == 0 ? 16.0f : 32.0f;
#pragma unroll
            for (int i = 0; i < 16; i++) {
                v[0][i] = (v[0][i] - back[2 * i]) * up;
                v[1][i] = (v[1][i] - back[2 * i + 1]) * up;
            }
        }
    }
    sx[(size_t)ts * kScaleBytes + lane * 2 + h] = (uint8_t)E;
}

template <int RT>
struct WTile {
    u32x4 a[RT][2]; // chunk 2 (l / 16) + h of row l % 16 of each row tile
    uint32_t s[RT]; // its two scale bytes
};

// tile[j]: tile of 64 rows with row tiles 4 j .. 4 j + 3 of the wave (uniform,
// so that a load is base, lane offset and constant). at: the lane's chunk,
// sat: its scale bytes.
template <int RT>
__device__ __forceinline__ WTile<RT> load_w(const uint8_t *const (&tile)[(RT + 3) / 4], size_t off, uint32_t at, uint32_t sat)
{
    WTile<RT> w;
#pragma unroll
    for (int m = 0; m < RT; m++) {
        const uint8_t *t = tile[m / 4] + off;
        w.s[m] = *reinterpret_cast<const uint16_t *>(t + sat + m % 4 * 128);
#pragma unroll
        for (int h = 0; h < 2; h++)
            w.a[m][h] = *reinterpret_cast<const u32x4 *>(t + at + h * 1024 + m % 4 * 256);
    }
    return w;
}

template <int H>
__device__ __forceinline__ f32x4 product(const i32x8 &a, const u32x4 &w, const f32x4 &c, uint32_t sa, uint32_t sb)
{
    const i32x8 b = {(int)w.x, (int)w.y, (int)w.z, (int)w.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 2, 4, H, (int)sa, H, (int)sb);
}

template <int RT, int CT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 1) void gemm_mx_kernel(GemmArgs a)
{
    constexpr int TB = TileFmt<RFX_FP4>::bytes, ROWS = 16 * RT * WAVES, COLS = 16 * CT, OP = ROWS + 4;
    constexpr int kScales = CT < 2 ? 256 : CT * kScaleBytes; // whole direct loads of 64 lanes
    constexpr int kStage = CT * kFragBytes + kScales;
    constexpr int kSmem = 2 * kStage > COLS * OP * 4 ? 2 * kStage : COLS * OP * 4;
    __shared__ __align__(16) char smem[kSmem];
    const int lane = threadIdx.x & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    GemmBlock blk;
    if (!gemm_block(a, blk))
        return;

    const int row0 = blk.rb * ROWS + 16 * RT * wave;
    const uint8_t *tile[(RT + 3) / 4];
#pragma unroll
    for (int j = 0; j < (RT + 3) / 4; j++) {
        const int rr = row0 + 64 * j < a.N ? row0 + 64 * j : 0; // rows past N: any rows, never stored
        tile[j] = a.W + (size_t)(rr >> 6) * a.S * TB;
    }
    const uint32_t rin = (row0 & 63) + (lane & 15), at = 2048 * g + rin * 16, sat = 8192 + rin * 8 + 2 * g;
    // each column tile's 15 KB by WAVES / CT waves (some chunks twice)
    static_assert(WAVES % CT == 0, "whole column tiles per wave");
    constexpr int PW = WAVES / CT;
    const int st = wave % CT, sk = wave / CT;
    const uint8_t *xsrc = a.xh + (size_t)(blk.cb * CT + st) * a.S * kFragBytes;
    const int sc_at = (wave * 256 + lane * 4) % (CT * kScaleBytes); // one column tile: some lanes read theirs again
    const uint8_t *ssrc = static_cast<const uint8_t *>(a.sx) + (size_t)(blk.cb * CT + sc_at / kScaleBytes) * a.S * kScaleBytes +
                          sc_at % kScaleBytes;
    constexpr int PIECES = (15 + PW - 1) / PW; // loads per wave and K tile
    constexpr int PER = (PIECES + CT) / (CT + 1);  // issued at a time, in the first half of a K tile's products
    const auto stage = [&](int s, int buf, int i0, int i1) {
        char *fb = smem + buf * kStage;
        const uint8_t *src = xsrc + (size_t)s * kFragBytes;
#pragma unroll
        for (int i = i0; i < i1; i++) {
            const int k = min(i * PW + sk, 14);
            lds_dma16(src + k * 1024 + (uint32_t)lane * 16, fb + st * kFragBytes + k * 1024);
        }
        if (i0 == 0 && wave < kScales / 256)
            lds_dma4(ssrc + (size_t)s * kScaleBytes, fb + CT * kFragBytes + wave * 256);
    };

    f32x4 acc[RT][CT] = {};
    WTile<RT> w = load_w<RT>(tile, (size_t)blk.s_begin * TB, at, sat);
    stage(blk.s_begin, 0, 0, PIECES);
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
    int buf = 0;
    for (int s = blk.s_begin; s < blk.s_end; s++, buf ^= 1) {
        const int sn = s + 1 < blk.s_end ? s + 1 : s;
        const WTile<RT> wn = load_w<RT>(tile, (size_t)sn * TB, at, sat);
        stage(sn, buf ^ 1, 0, PER);
        const char *fb = smem + buf * kStage;
        const uint16_t *sb = reinterpret_cast<const uint16_t *>(fb + CT * kFragBytes) + lane;
        uint32_t sc[CT];
#pragma unroll
        for (int tt = 0; tt < CT; tt++)
            sc[tt] = sb[tt * 64];
        // Batch i: the five digits of half i % 2 of column tile i / 2. The
        // next one's are read after the first products of this one: with
        // direct loads to LDS in flight every wait for an LDS read is a wait
        // for all of them, which by then were issued 4 RT products ago.
        const auto read = [&](int i, i32x8 (&x)[kDigits]) {
            const char *f = fb + i / 2 * kFragBytes + i % 2 * (kDigits * 1024) + lane * 16;
            const char *e = fb + i / 2 * kFragBytes + kTail + i % 2 * (kDigits * 512) + lane * 8;
#pragma unroll
            for (int d = kDigits - 1; d >= 0; d--) {
                const u32x4 lo = *reinterpret_cast<const u32x4 *>(f + d * 1024);
                const u32x2 hi = *reinterpret_cast<const u32x2 *>(e + d * 512);
                x[d] = (i32x8){(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, 0, 0};
            }
        };
        i32x8 x[2][kDigits];
        f32x4 t[RT];
        read(0, x[0]);
#pragma unroll
        for (int i = 0; i < 2 * CT; i++) {
            const int tt = i / 2, h = i % 2;
#pragma unroll
            for (int d = kDigits - 1; d >= 0; d--) { // the smallest first
                const uint32_t sa = sc[tt] - kOff[d] * 0x0101u;
#pragma unroll
                for (int m = 0; m < RT; m++) {
                    const f32x4 c = h == 0 && d == kDigits - 1 ? (f32x4){0.f, 0.f, 0.f, 0.f} : t[m];
                    t[m] = h == 0 ? product<0>(x[0][d], w.a[m][0], c, sa, w.s[m]) : product<1>(x[1][d], w.a[m][1], c, sa, w.s[m]);
                    if (h == 1 && d == 0)
                        acc[m][tt] += t[m];
                }
                if (d == kDigits - 1 && i + 1 < 2 * CT) {
                    __builtin_amdgcn_sched_barrier(0);
                    read(i + 1, x[~i & 1]);
                    if ((i + 1) * PER < PIECES)
                        stage(sn, buf ^ 1, (i + 1) * PER, min(PIECES, (i + 2) * PER));
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        // the next tile has landed in every wave's LDS before any reads it
        __builtin_amdgcn_s_waitcnt(0x0F70);
        __syncthreads();
        w = wn;
    }
    // results through the loop's buffers: lane l, register v: column 4 (l /
    // 16) + v, row l % 16
    float *o = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int m = 0; m < RT; m++)
#pragma unroll
        for (int tt = 0; tt < CT; tt++)
#pragma unroll
            for (int v = 0; v < 4; v++)
                o[(16 * tt + 4 * g + v) * OP + 16 * (RT * wave + m) + (lane & 15)] = acc[m][tt][v];
    __syncthreads();
    store_block<ROWS, COLS, WAVES>(a, blk, o);
}

template <int RT, int CT, int WAVES>
void launch(const GemmArgs &a, hipStream_t st)
{
    const int n = a.row_blocks * a.col_blocks * a.splits;
    hipLaunchKernelGGL((gemm_mx_kernel<RT, CT, WAVES>), dim3((n + 7) / 8 * 8), dim3(64 * WAVES), 0, st, a);
}

} // namespace

namespace rfx {

// 512 rows per workgroup where they still occupy three quarters of the
// compute units (fewer columns where not even one K tile each fills them,
// as in the f16 form): 2048 columns of 4096 x 7168 (256 workgroups) took 164 us
// against 187 with 256 rows, 1024 of 7168 x 2048 (224) 54 against 63, but 512
// of it (112) 42 against 34 and 1024 of 4096 x 7168 (128) 99 against 97.
GemmShape gemm_mx_shape(int64_t N, int64_t S, int tiles)
{
    int ct = tiles <= 1 ? 1 : tiles <= 2 ? 2 : 4;
    while (ct > 1 && ceil_div(N, 256) * ceil_div(tiles, ct) * S < 192)
        ct /= 2;
    const bool tall = ct == 4 && ceil_div(N, 512) * ((tiles + 3) / 4) >= 192;
    return {tall ? 512 : ct == 1 ? 128 : 256, ct, kFragBytes, kScaleBytes, ct == 4 ? 256 : 512};
}

int gemm_mx_launch(const GemmArgs &a, const GemmShape &g, const int8_t *xq, const float *xs, int nb, hipStream_t st)
{
    const int64_t n = (int64_t)(a.qp / 16) * a.S * 2;
    hipLaunchKernelGGL(mx_columns_kernel, dim3((unsigned)((n + 3) / 4)), dim3(256), 0, st, xq, xs, a.q, nb, a.S, (int)n,
                       const_cast<uint8_t *>(a.xh), static_cast<uint8_t *>(const_cast<void *>(a.sx)));
    const int err = hip_status("gemm columns launch");
    if (err)
        return err;
    if (g.tiles == 1)
        launch<2, 1, 4>(a, st);
    else if (g.tiles == 2)
        launch<4, 2, 4>(a, st);
    else if (g.rows == 256)
        launch<2, 4, 8>(a, st);
    else
        launch<4, 4, 8>(a, st);
    return hip_status("gemm launch");
}

} // namespace rfx
