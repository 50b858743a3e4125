// Low-rank adapters of many requests beside a shared projection:
//
//   y[t] = resid[t] + c[a] B[a] (A[a] x[t]),   a = ids[t],
//
// A[a] of rank x cols, B[a] of rows x rank, for up to four matrices (query,
// key and value projections) over the same x. Two launches: v = A x into the
// workspace, then y.
//
// Few tokens are bound by the adapters' bytes (each token may have its own),
// prompts by x, resid and y. Both launches take 16 tokens as the columns of
// v_mfma_16x16x32 products whose rows are one adapter's, for each adapter
// among the 16 tokens in turn; the columns of other adapters' tokens are zero,
// so one accumulator collects all. Tokens may have any order of adapters;
// runs of one adapter (a prompt) cost one pass. An adapter that is not finite
// makes the others' columns NaN (zero times infinity): where sums of several
// adapters hold a NaN, they are made again one adapter at a time, of which only
// its tokens take the result. Sums apart from the start cost 300 tokens of as
// many requests 66 us instead of 49.
//
// Adapters are 16-bit, x and v fp32: these enter as 16-bit terms, bf16 as
// three that sum to the fp32 value, fp16 as two (the second 2^11 larger, with
// sums of its own, so that it stays clear of fp16's subnormals), 2^-22 of the
// value. fp16 has few exponents: a token's x and v are brought into them by a
// power of two of its own, so that elements down to 2^-21 of the largest have
// that precision and smaller ones 2^-43 of the largest. Sums are fp32.
//
// Measured: one token, rank 16, query, key and value (4096 x 4096 + 2 x 1024)
// 8.5 us, the time of two launches that wait for memory twice (one launch in
// which every workgroup makes v itself took 10.0); 64 tokens of 48 adapters of
// rank 64, 4096 x 4096, 17.3 (the 37 MB of those that occur take 6); 4001 tokens
// of seven prompts, rank 32, 79.5: 32 for the first launch (66 MB of x, ten at its
// start and end) and 48 for the second (197 MB, 4.1 TB/s; a large copy has 4.8).
#include <algorithm>

#include "rfx_kv.h"

using namespace rfx;
using namespace rfx::dev;

namespace {

constexpr int kMaxRank = 128;
constexpr int kMats = RFX_LORA_MAX_MATS;
constexpr int kMaxLoraTokens = 1 << 19; // 16 a workgroup along the grid's y
constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kMaxSplits = 16;

struct LoraArgs {
    rfx_lora l;
    int R16;          // rank in whole tiles of 16
    int tiles;        // of all matrices
    int groups;       // of up to eight tiles
    int splits, slots;
    int down;         // workgroups of the first launch
    int T16;          // tokens in whole tiles
    float *v;         // [splits][T16][n_mats * R16]
    int row_blocks[kMats]; // of the second launch
    int turns;             // of its workgroups over the rows, with the same v
    int vec;          // bit m: rows of matrix m are 16-byte aligned
};

// Terms of an fp32 operand and the sums that collect their products.
template <class T>
struct Terms;

template <>
struct Terms<BF16> {
    static constexpr int N = 3, SUMS = 1;
    static __device__ __forceinline__ void split(const float (&x)[8], u4 (&t)[3]) { split_terms<BF16, 3>(x, t); }
    // One term's product, the smallest first (s = 0).
    static __device__ __forceinline__ void mma(int s, u4 a, const u4 (&t)[3], f32x4 (&c)[1]) { c[0] = BF16::mma16(a, t[2 - s], c[0]); }
    static __device__ __forceinline__ f32x4 total(const f32x4 (&c)[1]) { return c[0]; }
};

template <>
struct Terms<F16> {
    static constexpr int N = 2, SUMS = 2;
    static __device__ __forceinline__ void split(const float (&x)[8], u4 (&t)[2])
    {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t u = F16::pack(x[2 * i], x[2 * i + 1]);
            const f2 back = F16::unpack(u);
            t[0][i] = u;
            t[1][i] = F16::pack((x[2 * i] - back.x) * 0x1p11f, (x[2 * i + 1] - back.y) * 0x1p11f);
        }
    }
    static __device__ __forceinline__ void mma(int s, u4 a, const u4 (&t)[2], f32x4 (&c)[2]) { c[s] = F16::mma16(a, t[s], c[s]); }
    static __device__ __forceinline__ f32x4 total(const f32x4 (&c)[2]) { return c[0] + c[1] * 0x1p-11f; }
};

// The power of two that brings `top` into 128 .. 256 (tiny and huge ones as near
// as a normal power does, infinity anywhere), and what undoes it.
__device__ __forceinline__ float fitting(float top)
{
    const int ex = (int)(__float_as_uint(top) >> 23);
    return __uint_as_float((uint32_t)max(1, min(253, 254 + 7 - ex)) << 23);
}
__device__ __forceinline__ float inverse(float power) { return __uint_as_float((254u << 23) - __float_as_uint(power)); }

// A token's factor of x, that of what its columns had so far, made smaller where
// the next ones (at most `top` in this lane) would leave fp16, its sums with it.
// That takes elements 2^7 times as large: rescaling is rare. The four lanes of a
// token have the same factor.
template <int TILES, int SUMS>
__device__ __forceinline__ void refit(float top, float &factor, f32x4 (&acc)[TILES][SUMS])
{
    if (__any(top * factor > 0x1p15f)) {
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float next = top * factor > 0x1p15f ? fitting(top) : factor, f = next * inverse(factor);
#pragma unroll
        for (int i = 0; i < TILES; i++)
#pragma unroll
            for (int s = 0; s < SUMS; s++)
                acc[i][s] *= f;
        factor = next;
    }
}

// The adapter of token t, -1 for none.
__device__ __forceinline__ int adapter_of(const rfx_lora &l, int t)
{
    if (t >= l.n_tokens)
        return -1;
    const int a = l.ids[t];
    return (unsigned)a < (unsigned)l.n_adapters ? a : -1;
}

// Waves per SIMD that the registers leave room for.
constexpr int down_waves(int tiles, int nb, int sums) { return tiles * nb * (2 + sums) > 36 || (sums > 1 && tiles > 6) ? 1 : 2; }

// v = A x: a workgroup takes NB times 16 tokens, one of `splits` parts of the
// columns (a quarter of it per wave, added through LDS) and every slots-th
// adapter of its tokens, against TILES of the 16-row tiles of all matrices,
// which stand one after the other. 64 columns at a time, so that a row's 128
// bytes are read together, with the next ones' loads in flight.
template <class T, int TILES, int NB>
__global__ __launch_bounds__(kThreads, down_waves(TILES, NB, Terms<T>::SUMS)) void lora_down_kernel(LoraArgs a)
{
    using X = Terms<T>;
    constexpr int SUMS = TILES * NB > 4 ? 4 : TILES * NB; // tiles in LDS at a time
    constexpr int XP = 128 + 16, WP = 64 + 16;            // pitches of 32 columns of x and of A
    constexpr int PIECE = NB > 1 ? 16 * NB * XP + 16 * TILES * WP : 0, LDS = PIECE > SUMS * 1024 ? PIECE : SUMS * 1024;
    __shared__ __align__(16) char smem[kWaves * LDS];
    __shared__ int bad[kWaves];
    auto &sums = *reinterpret_cast<f32x4 (*)[kWaves][SUMS][64]>(smem);
    const rfx_lora &l = a.l;
    const int lane = threadIdx.x & 63, r16 = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Workgroups go round the eight XCDs in order: a contiguous run of them to
    // each, so that its L2 keeps the few adapters of its tokens.
    [[maybe_unused]] char *piece = smem + wave * LDS;
    int b = blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
    if (b >= a.down)
        return;
    const int split = b % a.splits;
    b /= a.splits;
    const int tile0 = b % a.groups * TILES;
    b /= a.groups;
    const int blocks = a.T16 / (16 * NB), slot = b / blocks, t0 = (b - slot * blocks) * 16 * NB;
    const int steps = (l.cols + 63) / 64, part = a.splits * kWaves, p = split * kWaves + wave;
    const int k0 = (int)((int64_t)steps * p / part), k1 = (int)((int64_t)steps * (p + 1) / part);

    f32x4 acc[NB][TILES][X::SUMS];
    [[maybe_unused]] float factor[NB]; // of the lane's tokens
    int id[NB];
    bool mine[NB]; // this workgroup has the lane's token
    uint32_t all = 0;
#pragma unroll
    for (int n = 0; n < NB; n++) {
        id[n] = adapter_of(l, t0 + 16 * n + r16);
        all |= ((uint32_t)__ballot(id[n] >= 0) & 0xffffu) << 16 * n;
    }

    // All of this workgroup's adapters at once (only = 0), or, where that holds a
    // NaN, one after the other. The same in every wave.
    for (int only = 0;;) {
        int from_tile = tile0; // addresses are made anew: kept, they take the sums' registers
        asm volatile("" : "+s"(from_tile));
#pragma unroll
        for (int n = 0; n < NB; n++) {
            mine[n] = false;
            factor[n] = 0x1p126f;
#pragma unroll
            for (int i = 0; i < TILES; i++)
#pragma unroll
                for (int s = 0; s < X::SUMS; s++)
                    acc[n][i][s] = (f32x4){0.f, 0.f, 0.f, 0.f};
        }
        int taken = 0;
        uint32_t todo = all;
        for (int turn = 0; todo; turn++) {
            const int first = __builtin_ctz(todo);
            int ad = __builtin_amdgcn_readlane(id[0], first & 15);
            if (NB > 1 && first >= 16)
                ad = __builtin_amdgcn_readlane(id[NB - 1], first & 15);
            bool own = turn % a.slots == slot;
            taken += own;
            own &= !only || taken == only;
            uint32_t keep[NB];
            const float *x[NB];
#pragma unroll
            for (int n = 0; n < NB; n++) {
                const bool match = id[n] == ad;
                todo &= ~(((uint32_t)__ballot(match) & 0xffffu) << 16 * n);
                mine[n] |= match & own;
                keep[n] = match ? ~0u : 0u;
                // (few tokens) lanes of other adapters' tokens read along with the first one's
                x[n] = l.x + (int64_t)(t0 + (match ? 16 * n + r16 : first)) * l.x_stride + 8 * g4;
            }
            if (!own || k0 >= k1)
                continue;
            if constexpr (NB == 1) {
                const uint16_t *w[TILES];
#pragma unroll
                for (int i = 0; i < TILES; i++) {
                    const int row = 16 * min(from_tile + i, a.tiles - 1), m = row / a.R16, r = min(row - m * a.R16 + r16, l.rank - 1);
                    w[i] = static_cast<const uint16_t *>(l.mats[m].a) + ((size_t)ad * l.rank + r) * l.cols + 8 * g4;
                }
                struct Step {
                    f32x4 x[2][NB][2];
                    u4 w[TILES][2];
                } s0, s1;
                const auto load = [&](Step &s, int k) { // columns past the last: the step's first half again
                    const size_t at = 64 * (size_t)min(k, k1 - 1), up = at + 32 < (size_t)l.cols ? 32 : 0;
#pragma unroll
                    for (int h = 0; h < 2; h++)
#pragma unroll
                        for (int n = 0; n < NB; n++)
#pragma unroll
                            for (int q = 0; q < 2; q++)
                                s.x[h][n][q] = *reinterpret_cast<const f32x4 *>(x[n] + at + h * up + 4 * q);
#pragma unroll
                    for (int i = 0; i < TILES; i++)
#pragma unroll
                        for (int h = 0; h < 2; h++)
                            s.w[i][h] = *reinterpret_cast<const u4 *>(w[i] + at + h * up);
                    __builtin_amdgcn_sched_barrier(0);
                };
                const auto compute = [&](const Step &s, int k) {
                    if constexpr (X::SUMS > 1)
#pragma unroll
                        for (int n = 0; n < NB; n++) {
                            float top = 0.f;
#pragma unroll
                            for (int e = 0; e < 16; e++)
                                top = fmaxf(top, fabsf(s.x[e >> 3][n][(e >> 2) & 1][e & 3]));
                            refit(keep[n] ? top : 0.f, factor[n], acc[n]);
                        }
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const uint32_t in = 64 * k + 32 * h < l.cols ? ~0u : 0u;
#pragma unroll
                        for (int n = 0; n < NB; n++) {
                            float xc[8];
                            u4 t[X::N];
#pragma unroll
                            for (int e = 0; e < 8; e++)
                                xc[e] = X::SUMS > 1 ? s.x[h][n][e >> 2][e & 3] * factor[n] : s.x[h][n][e >> 2][e & 3];
                            X::split(xc, t);
#pragma unroll
                            for (int q = 0; q < X::N; q++)
                                t[q] &= keep[n] & in;
#pragma unroll
                            for (int q = 0; q < X::N; q++) // neighbours do not depend on one another
#pragma unroll
                                for (int j = 0; j < TILES; j++)
                                    X::mma(q, s.w[j][h], t, acc[n][j]);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                };
                load(s0, k0);
                for (int k = k0; k < k1; k += 2) {
                    load(s1, k + 1);
                    compute(s0, k);
                    if (k + 1 == k1)
                        break;
                    load(s0, k + 2);
                    compute(s1, k + 1);
                }
            } else {
                // 32 columns at a time through the wave's own piece of LDS: a load
                // whose 16 lanes of a quarter read 16 rows takes the cycles of
                // sixteen, one that reads whole lines of two (x) or four (A) rows
                // those of as many.
                const int first_k = 2 * k0, last_k = min(2 * k1, l.cols / 32);
                const float *px[2 * NB];
#pragma unroll
                for (int j = 0; j < 2 * NB; j++)
                    px[j] = l.x + (int64_t)min(t0 + 8 * j + (lane >> 3), l.n_tokens - 1) * l.x_stride + 4 * (lane & 7);
                const uint16_t *pw[TILES];
#pragma unroll
                for (int i = 0; i < TILES; i++) {
                    const int row = 16 * min(from_tile + i, a.tiles - 1), m = row / a.R16, r = min(row - m * a.R16 + (lane >> 2), l.rank - 1);
                    pw[i] = static_cast<const uint16_t *>(l.mats[m].a) + ((size_t)ad * l.rank + r) * l.cols + 8 * (lane & 3);
                }
                constexpr int AHEAD = 2; // steps in flight
                f32x4 xn[AHEAD][2 * NB];
                u4 wn[AHEAD][TILES];
                const auto load = [&](int u, int k) {
                    const int at = 32 * min(k, last_k - 1);
#pragma unroll
                    for (int j = 0; j < 2 * NB; j++)
                        xn[u][j] = *reinterpret_cast<const f32x4 *>(px[j] + at);
#pragma unroll
                    for (int i = 0; i < TILES; i++)
                        wn[u][i] = *reinterpret_cast<const u4 *>(pw[i] + at);
                };
                const auto step = [&](int u, int k) {
#pragma unroll
                    for (int j = 0; j < 2 * NB; j++)
                        *reinterpret_cast<f32x4 *>(piece + (8 * j + (lane >> 3)) * XP + 16 * (lane & 7)) = xn[u][j];
#pragma unroll
                    for (int i = 0; i < TILES; i++)
                        *reinterpret_cast<u4 *>(piece + 16 * NB * XP + (16 * i + (lane >> 2)) * WP + 16 * (lane & 3)) = wn[u][i];
                    load(u, k + AHEAD);
                    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                    u4 w[TILES];
#pragma unroll
                    for (int i = 0; i < TILES; i++)
                        w[i] = *reinterpret_cast<const u4 *>(piece + 16 * NB * XP + (16 * i + r16) * WP + 16 * g4);
#pragma unroll
                    for (int n = 0; n < NB; n++) {
                        const char *p = piece + (16 * n + r16) * XP + 32 * g4;
                        const f32x4 x0 = *reinterpret_cast<const f32x4 *>(p), x1 = *reinterpret_cast<const f32x4 *>(p + 16);
                        float xc[8];
                        u4 t[X::N];
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            xc[e] = x0[e];
                            xc[e + 4] = x1[e];
                        }
                        if constexpr (X::SUMS > 1) {
                            float top = 0.f;
#pragma unroll
                            for (int e = 0; e < 8; e++)
                                top = fmaxf(top, fabsf(xc[e]));
                            refit(keep[n] ? top : 0.f, factor[n], acc[n]);
#pragma unroll
                            for (int e = 0; e < 8; e++)
                                xc[e] *= factor[n];
                        }
                        X::split(xc, t);
#pragma unroll
                        for (int q = 0; q < X::N; q++)
                            t[q] &= keep[n];
#pragma unroll
                        for (int q = 0; q < X::N; q++)
#pragma unroll
                            for (int i = 0; i < TILES; i++)
                                X::mma(q, w[i], t, acc[n][i]);
                    }
                    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                };
#pragma unroll
                for (int u = 0; u < AHEAD; u++)
                    load(u, first_k + u);
                for (int k = first_k; k < last_k; k += AHEAD)
#pragma unroll
                    for (int u = 0; u < AHEAD; u++)
                        if (k + u < last_k)
                            step(u, k + u);
            }
        }
        if (!taken)
            return;
        if (NB > 1 || only)
            __syncthreads(); // the pieces, or the last ones, become the sums
        if (!only && taken > 1) {
            float any = 0.f;
#pragma unroll
            for (int n = 0; n < NB; n++)
#pragma unroll
                for (int i = 0; i < TILES; i++)
#pragma unroll
                    for (int s = 0; s < X::SUMS; s++)
                        any += (acc[n][i][s][0] + acc[n][i][s][1]) + (acc[n][i][s][2] + acc[n][i][s][3]);
            const bool nan = __ballot(any != any) != 0;
            if (lane == 0)
                bad[wave] = nan;
            __syncthreads();
            if (bad[0] | bad[1] | bad[2] | bad[3]) {
                only = 1;
                continue;
            }
        }
        // lane: token r16 of its sixteen, rows 4 g4 .. + 3 of tile i
        const int RS = l.n_mats * a.R16;
#pragma unroll
        for (int j = 0; j < TILES * NB; j += SUMS) {
            if (j)
                __syncthreads();
#pragma unroll
            for (int i = j; i < j + SUMS; i++)
                if (i < TILES * NB)
                    sums[wave][i - j][lane] = X::SUMS > 1 ? X::total(acc[i / TILES][i % TILES]) * inverse(factor[i / TILES])
                                                          : X::total(acc[i / TILES][i % TILES]);
            __syncthreads();
            const int i = j + wave, n = i / TILES, tile = from_tile + i % TILES; // SUMS is at most the waves' number
            if (wave < SUMS && i < TILES * NB && tile < a.tiles) {
                f32x4 s = sums[0][wave][lane];
#pragma unroll
                for (int w = 1; w < kWaves; w++)
                    s += sums[w][wave][lane];
                if (NB > 1 && n ? mine[NB - 1] : mine[0])
                    *reinterpret_cast<f32x4 *>(a.v + ((size_t)split * a.T16 + t0 + 16 * n + r16) * RS + 16 * tile + 4 * g4) = s;
            }
        }
        if (!only || ++only > taken)
            return;
        __syncthreads(); // the sums are read
    }
}

// y = resid + c B v: a workgroup takes 16 tokens, whose v it adds up once in
// LDS, a wave RT tiles of 16 rows. KS: steps of 32 over the rank. Where rows
// are few per wave, ADS adapters' tiles are read at a time.
template <class T, int KS, int RT, int ADS>
__global__ __launch_bounds__(kThreads) void lora_up_kernel(LoraArgs a)
{
    using X = Terms<T>;
    constexpr int CH = 4 * KS;                       // chunks of eight ranks
    constexpr int PARTS = kThreads / (16 * CH);      // threads that share the splits of a chunk
    constexpr int VP = 32 * KS + 4;                  // pitch of a token's v
    __shared__ __align__(16) float sv[PARTS][16][VP];
    const rfx_lora &l = a.l;
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int t0 = blockIdx.y * 16, t = t0 + r16;
    int m = 0, rb = blockIdx.x;
    while (m + 1 < l.n_mats && rb >= a.row_blocks[m])
        rb -= a.row_blocks[m++];
    const rfx_lora_mat &M = l.mats[m];
    constexpr int STRIDE = kWaves * 16 * RT; // rows of the workgroup's waves
    int n0 = (rb * a.turns * kWaves + wave) * 16 * RT;
    const int n_end = min(M.rows, n0 + a.turns * STRIDE);
    const int id = adapter_of(l, t);
    const uint32_t all = (uint32_t)__ballot(id >= 0) & 0xffffu;
    const bool any = all != 0; // the same in every wave
    // more than one adapter
    const bool several = any && (all & ~(uint32_t)__ballot(id == __builtin_amdgcn_readlane(id, any ? __builtin_ctz(all) : 0)));
    if (!any && M.resid == M.y)
        return;

    // Step k's part of a row of an adapter's B; past the last, the last again.
    const auto load_b = [&](const uint16_t *p, int n, int k) {
        const int r = 32 * k + 8 * g4;
        const u4 x = *reinterpret_cast<const u4 *>(p + (size_t)min(n, M.rows - 1) * l.rank + (r < l.rank ? r : 0));
        return r < l.rank ? x : (u4){0, 0, 0, 0};
    };
    // The next ADS adapters: their rows of B from next_n on, and who has them.
    bool live[ADS];
    uint32_t keep[ADS], todo = all;
    int next_n = n0;
    u4 w[ADS][RT][KS];
    const auto fetch = [&] {
#pragma unroll
        for (int j = 0; j < ADS; j++) {
            live[j] = todo != 0;
            if (!live[j])
                continue;
            const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
            const bool match = id == ad;
            todo &= ~(uint32_t)__ballot(match);
            keep[j] = match ? ~0u : 0u;
            const uint16_t *p = static_cast<const uint16_t *>(M.b) + (size_t)ad * M.rows * l.rank;
#pragma unroll
            for (int i = 0; i < RT; i++)
#pragma unroll
                for (int k = 0; k < KS; k++)
                    w[j][i][k] = load_b(p, next_n + 16 * i + r16, k);
        }
    };
    // The residual's rows, ahead of everything that they are added to.
    const bool vec = a.vec >> m & 1;
    const float *resid = M.resid + (size_t)t * M.rows;
    f32x4 next_y[RT];
    const auto load_resid = [&](int from) {
#pragma unroll
        for (int i = 0; i < RT; i++) {
            const int n = from + 16 * i + 4 * g4;
            next_y[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
            if (vec && M.resid && t < l.n_tokens && n < M.rows)
                next_y[i] = *reinterpret_cast<const f32x4 *>(resid + n);
        }
    };
    load_resid(n0);
    float out = 1.0f;
    u4 vt[KS][X::N];
    if (any) {
        fetch();
        const float c = id >= 0 && M.scale ? M.scale[id] : 1.0f;
        // the splits of v in order: every PARTS-th by one thread
        {
            const int RS = l.n_mats * a.R16, ch = tid % CH, tok = tid / CH % 16, part = tid / (16 * CH);
            const bool on = 8 * ch < l.rank;
            const float *p = a.v + (size_t)(t0 + tok) * RS + m * a.R16 + (on ? 8 * ch : 0);
            const size_t stride = (size_t)a.T16 * RS;
            f32x4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
#pragma unroll 4
            for (int s = part; s < a.splits; s += PARTS) {
                s0 += *reinterpret_cast<const f32x4 *>(p + s * stride);
                s1 += *reinterpret_cast<const f32x4 *>(p + s * stride + 4);
            }
            *reinterpret_cast<f32x4 *>(&sv[part][tok][8 * ch]) = s0;
            *reinterpret_cast<f32x4 *>(&sv[part][tok][8 * ch + 4]) = s1;
        }
        __syncthreads();
        // the lane's part of its token's v, times the adapter's factor
        float v[KS][8];
#pragma unroll
        for (int k = 0; k < KS; k++) {
            const int r = 32 * k + 8 * g4;
            const bool on = id >= 0 && r < l.rank; // what no one wrote may be anything
            f32x4 s0 = *reinterpret_cast<const f32x4 *>(&sv[0][r16][r]), s1 = *reinterpret_cast<const f32x4 *>(&sv[0][r16][r + 4]);
#pragma unroll
            for (int q = 1; q < PARTS; q++) {
                s0 += *reinterpret_cast<const f32x4 *>(&sv[q][r16][r]);
                s1 += *reinterpret_cast<const f32x4 *>(&sv[q][r16][r + 4]);
            }
#pragma unroll
            for (int e = 0; e < 4; e++) {
                v[k][e] = on ? s0[e] * c : 0.f;
                v[k][e + 4] = on ? s1[e] * c : 0.f;
            }
        }
        if (X::SUMS > 1) { // a power of two off, and on again below
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < KS; k++)
#pragma unroll
                for (int e = 0; e < 8; e++)
                    top = fmaxf(top, fabsf(v[k][e]));
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float in = fitting(top);
            out = inverse(in);
#pragma unroll
            for (int k = 0; k < KS; k++)
#pragma unroll
                for (int e = 0; e < 8; e++)
                    v[k][e] *= in;
        }
#pragma unroll
        for (int k = 0; k < KS; k++)
            X::split(v[k], vt[k]);
    }
    for (; n0 < n_end; n0 += STRIDE) {
        // lane: token r16, rows 4 g4 .. + 3 of tile i
        f32x4 acc[RT][X::SUMS], y[RT];
#pragma unroll
        for (int i = 0; i < RT; i++) {
#pragma unroll
            for (int s = 0; s < X::SUMS; s++)
                acc[i][s] = (f32x4){0.f, 0.f, 0.f, 0.f};
            y[i] = next_y[i];
        }
        if (n0 + STRIDE < n_end)
            load_resid(n0 + STRIDE);
        for (bool more = any; more;) {
            u4 now[ADS][RT][KS];
            bool on[ADS];
            uint32_t who[ADS];
#pragma unroll
            for (int j = 0; j < ADS; j++) {
                on[j] = live[j];
                who[j] = keep[j];
#pragma unroll
                for (int i = 0; i < RT; i++)
#pragma unroll
                    for (int k = 0; k < KS; k++)
                        now[j][i][k] = w[j][i][k];
            }
            more = todo != 0;
            if (!more) {
                todo = all;
                next_n += STRIDE;
            }
            if (ADS == 1 && next_n < n_end) // the next ones' loads before these's products
                fetch();
#pragma unroll
            for (int j = 0; j < ADS; j++) {
                if (!on[j])
                    continue;
#pragma unroll
                for (int k = 0; k < KS; k++) {
                    u4 tm[X::N];
#pragma unroll
                    for (int s = 0; s < X::N; s++)
                        tm[s] = vt[k][s] & who[j];
#pragma unroll
                    for (int s = 0; s < X::N; s++)
#pragma unroll
                        for (int i = 0; i < RT; i++)
                            X::mma(s, now[j][i][k], tm, acc[i]);
                }
            }
            if (ADS > 1 && next_n < n_end)
                fetch();
        }
        f32x4 sum[RT];
        float nan = 0.f;
#pragma unroll
        for (int i = 0; i < RT; i++) {
            const f32x4 total = X::total(acc[i]);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                sum[i][e] = id >= 0 ? total[e] : 0.f;
                nan += sum[i][e];
            }
        }
        if (several && __ballot(nan != nan)) { // apart
#pragma unroll 1
            for (uint32_t left = all; left;) {
                const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
                const bool match = id == ad;
                left &= ~(uint32_t)__ballot(match);
                const uint16_t *p = static_cast<const uint16_t *>(M.b) + (size_t)ad * M.rows * l.rank;
#pragma unroll
                for (int i = 0; i < RT; i++) {
                    f32x4 one[X::SUMS];
#pragma unroll
                    for (int s = 0; s < X::SUMS; s++)
                        one[s] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < KS; k++) {
                        const u4 b = load_b(p, n0 + 16 * i + r16, k);
#pragma unroll
                        for (int s = 0; s < X::N; s++)
                            X::mma(s, b, vt[k], one);
                    }
                    const f32x4 total = X::total(one);
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        sum[i][e] = match ? total[e] : sum[i][e];
                }
            }
        }
        if (t >= l.n_tokens)
            continue;
#pragma unroll
        for (int i = 0; i < RT; i++) {
            const int n = n0 + 16 * i + 4 * g4, left = M.rows - n;
            if (left <= 0)
                continue;
            const size_t at = (size_t)t * M.rows + n;
            y[i] += sum[i] * out;
            if (vec) {
                *reinterpret_cast<f32x4 *>(M.y + at) = y[i];
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (e < left)
                        M.y[at + e] = M.resid ? y[i][e] + resid[n + e] : y[i][e];
            }
        }
    }
}

struct Plan {
    int R16, tiles, groups, splits, slots, T16;
    bool wide; // 32 tokens per workgroup of the first launch
    size_t bytes;
};

Plan plan(int T, int rank, int n_mats, int cols, int n_adapters)
{ // the same for both types: a workspace may serve either
    Plan p{};
    p.R16 = (rank + 15) / 16 * 16;
    p.tiles = n_mats * p.R16 / 16;
    p.groups = (p.tiles + 7) / 8;
    // 300 tokens of two prompts 18.0 us with 32 a workgroup and 22.0 with 16, 400
    // 20.6 and 27.0; 200 tokens of 64 requests 16.9 and 15.2.
    p.wide = T > 256;
    const int per = p.wide ? 32 : 16, blocks = T > per ? (T + per - 1) / per : 1;
    p.T16 = blocks * per;
    // Adapters of a block of tokens: side by side where tokens are few and
    // may each have their own, one after the other where they are many.
    p.slots = T <= 128 ? 16 : T <= 256 ? 4 : 1;
    p.slots = p.slots < T ? p.slots : T;
    p.slots = p.slots < n_adapters ? p.slots : n_adapters;
    // Columns split until there is a workgroup for every place, down to a step
    // of 64 columns per wave. Few tokens: for every adapter's place, since the
    // second launch reads v once per split: 64 tokens, 48 adapters of rank 64, 18
    // us with four splits and 24 with sixteen; one token 8.5 with sixteen and 10.0
    // with four.
    const int waves = down_waves(p.tiles < 8 ? p.tiles : 8, p.wide ? 2 : 1, 1), most = (cols + 255) / 256;
    const int want = T <= 128 ? std::max(4, 256 / (blocks * p.slots * p.groups)) : 256 * waves / (blocks * p.groups);
    p.splits = std::max(1, std::min({want, most, kMaxSplits}));
    p.bytes = (size_t)p.splits * p.T16 * n_mats * p.R16 * sizeof(float);
    return p;
}

bool shape_ok(int T, int rank, int n_mats, int cols, int n_adapters)
{
    return T >= 0 && T <= kMaxLoraTokens && rank >= 8 && rank <= kMaxRank && rank % 8 == 0 && n_mats >= 1 && n_mats <= kMats &&
           cols >= 32 && cols % 32 == 0 && cols <= 1 << 20 && n_adapters >= 1 && n_adapters <= 1 << 20;
}

template <class T, int NB>
void launch_down_tiles(LoraArgs &a, hipStream_t st)
{
    a.down = a.T16 / (16 * NB) * a.slots * a.groups * a.splits;
    const dim3 grid((a.down + 7) / 8 * 8), block(kThreads);
#define RFX_LORA(TILES) hipLaunchKernelGGL((lora_down_kernel<T, TILES, NB>), grid, block, 0, st, a)
    if (a.tiles <= 1)
        RFX_LORA(1);
    else if (a.tiles <= 2)
        RFX_LORA(2);
    else if (a.tiles <= 3)
        RFX_LORA(3);
    else if (a.tiles <= 4)
        RFX_LORA(4);
    else if (a.tiles <= 6)
        RFX_LORA(6);
    else
        RFX_LORA(8);
#undef RFX_LORA
}

template <class T>
int launch_down(LoraArgs &a, bool wide, hipStream_t st)
{
    if (wide)
        launch_down_tiles<T, 2>(a, st);
    else
        launch_down_tiles<T, 1>(a, st);
    return hip_status("lora down launch");
}

template <class T, int KS>
void launch_up_rank(LoraArgs &a, bool many, hipStream_t st)
{
    int blocks = 0;
    a.turns = 1;
    for (;; a.turns = 2) {
        blocks = 0;
        for (int m = 0; m < a.l.n_mats; m++)
            blocks += a.row_blocks[m] = (int)ceil_div(a.l.mats[m].rows, (many ? 32 : 16) * kWaves * a.turns);
        // Two turns where the chip is full without (4001 tokens 80.9 us, with
        // one 82.4, four 85.3; 300 tokens 18.4 and 17.1).
        if (!many || a.turns == 2 || (int64_t)blocks * (a.T16 / 16) < 2048)
            break;
    }
    const dim3 grid(blocks, a.T16 / 16), block(kThreads);
    if (many)
        hipLaunchKernelGGL((lora_up_kernel<T, KS, 2, 1>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((lora_up_kernel<T, KS, 1, 16 / KS>), grid, block, 0, st, a);
}

template <class T>
int launch_up(LoraArgs &a, hipStream_t st)
{
    const bool many = a.l.n_tokens > 256;
    if (a.l.rank <= 32)
        launch_up_rank<T, 1>(a, many, st);
    else if (a.l.rank <= 64)
        launch_up_rank<T, 2>(a, many, st);
    else
        launch_up_rank<T, 4>(a, many, st);
    return hip_status("lora up launch");
}

} // namespace

extern "C" {

size_t rfx_lora_workspace_bytes(int n_tokens, int rank, int n_mats, int cols, int n_adapters)
{
    return shape_ok(n_tokens, rank, n_mats, cols, n_adapters) ? plan(n_tokens, rank, n_mats, cols, n_adapters).bytes : 0;
}

int rfx_lora_apply(const rfx_lora *L, void *ws, size_t ws_bytes, void *stream)
{
    if (!L)
        return fail(RFX_E_INVAL, "rfx_lora_apply: arguments are NULL");
    if (L->type != RFX_F16 && L->type != RFX_BF16)
        return fail(RFX_E_INVAL, "rfx_lora_apply: type %d (RFX_F16 or RFX_BF16)", L->type);
    if (!shape_ok(L->n_tokens, L->rank, L->n_mats, L->cols, L->n_adapters))
        return fail(RFX_E_INVAL, "rfx_lora_apply: n_tokens=%d rank=%d n_mats=%d cols=%d n_adapters=%d (at most 2^19 tokens; rank a "
                    "multiple of 8, at most %d; 1 to %d matrices; cols a multiple of 32, at most 2^20; 1 to 2^20 adapters)",
                    L->n_tokens, L->rank, L->n_mats, L->cols, L->n_adapters, kMaxRank, kMats);
    if (L->x_stride < L->cols || L->x_stride % 4 || L->x_stride > (int64_t)1 << 40)
        return fail(RFX_E_INVAL, "rfx_lora_apply: x_stride=%lld (a multiple of 4, at least cols)", (long long)L->x_stride);
    int st = check_ptr(L->x, 16, "x");
    if (st || (st = check_ptr(L->ids, 4, "ids")))
        return st;
    LoraArgs a{};
    for (int m = 0; m < L->n_mats; m++) {
        const rfx_lora_mat &M = L->mats[m];
        if (M.rows < 1 || M.rows > 1 << 24)
            return fail(RFX_E_INVAL, "rfx_lora_apply: matrix %d of %d rows (1 to 2^24)", m, M.rows);
        if ((st = check_ptr(M.a, 16, "a")) || (st = check_ptr(M.b, 16, "b")) || (st = check_ptr(M.y, 4, "y")) ||
            (M.resid && (st = check_ptr(M.resid, 4, "resid"))) || (M.scale && (st = check_ptr(M.scale, 4, "scale"))))
            return st;
        if (M.rows % 4 == 0 && !((reinterpret_cast<uintptr_t>(M.y) | reinterpret_cast<uintptr_t>(M.resid)) & 15))
            a.vec |= 1 << m;
    }
    if (L->n_tokens == 0)
        return RFX_OK;
    for (int m = 1; m < L->n_mats; m++) // workgroups of both would write there
        for (int j = 0; j < m; j++) {
            const rfx_lora_mat &A = L->mats[j], &B = L->mats[m];
            const uintptr_t ya = reinterpret_cast<uintptr_t>(A.y), yb = reinterpret_cast<uintptr_t>(B.y), each = (uintptr_t)L->n_tokens * 4;
            if (ya < yb + each * B.rows && yb < ya + each * A.rows)
                return fail(RFX_E_INVAL, "rfx_lora_apply: results of matrices %d and %d overlap", j, m);
        }
    const Plan p = plan(L->n_tokens, L->rank, L->n_mats, L->cols, L->n_adapters);
    if (!ws || ws_bytes < p.bytes)
        return fail(RFX_E_WORKSPACE, "rfx_lora_apply: workspace %zu < %zu bytes", ws ? ws_bytes : (size_t)0, p.bytes);
    if ((st = check_ptr(ws, 256, "ws")))
        return st;
    a.l = *L;
    a.R16 = p.R16;
    a.tiles = p.tiles;
    a.groups = p.groups;
    a.splits = p.splits;
    a.slots = p.slots;
    a.T16 = p.T16;
    a.v = static_cast<float *>(ws);
    const hipStream_t hs = (hipStream_t)stream;
    st = L->type == RFX_BF16 ? launch_down<BF16>(a, p.wide, hs) : launch_down<F16>(a, p.wide, hs);
    if (st)
        return st;
    return L->type == RFX_BF16 ? launch_up<BF16>(a, hs) : launch_up<F16>(a, hs);
}

} // extern "C"
