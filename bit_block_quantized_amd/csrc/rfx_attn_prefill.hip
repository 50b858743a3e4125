// Attention of prompts and chunks over the paged cache: o = softmax(scale q
// k^T + mask) v with a causal mask, an optional sliding window and a few
// first tokens that stay visible (sinks).
//
// Bound by the matrix core and by the exponentials beside it. The query
// heads that share a kv head are packed into the rows (row = token * G +
// head of the group), so that a key tile serves all of them and short chunks
// still fill the row tiles. A workgroup of four waves takes 128 rows; key
// tiles of BN keys go through two LDS buffers, the next one's loads in
// flight in registers during the current one's products.
//   S^T = K Q^T on v_mfma_f32_32x32x16: A = 32 keys (LDS), B = the wave's 32
//   rows (registers). A lane holds half of one row's scores, so a row's
//   maximum takes one exchange between lane halves and its sum none.
//   O^T = V^T P^T: S^T's register order is P^T's operand order once the keys
//   of V^T are read in that order (transposed LDS reads), so the weights stay
//   in their lane.
// Tiles outside a wave's rows' window or after their positions are skipped.
// Few row blocks over long sequences: the keys are split over S workgroups
// and a second launch joins the partials in split order.
//
// Rounding: weights are rounded once to the cache's type for a result of
// that type (its own rounding is as large), and the row sums are of the
// rounded ones; for an fp32 result they are carried as the sum of TERMS
// values, and the sums are of the fp32 weights.
#include "rfx_kv.h"

using namespace rfx;
using namespace rfx::dev;

namespace {

constexpr int kWaves = 4;
constexpr int kRows = 32 * kWaves;
constexpr int kThreads = 64 * kWaves;

constexpr int kIds = 1024;

// Pitches (bytes) of the LDS rows: K rows are read 16 bytes per lane down a
// column, so neighbours are 16 bytes apart modulo the 256 bytes of the
// banks; four V rows are read 64 bytes at a time, so theirs are 64 apart.
template <int DP, int THREADS = kThreads>
struct Tile {
    static constexpr int BN = DP <= 128 ? 64 : 32;
    static constexpr int KP = DP * 2 + 16, VP = DP * 2 + 64;
    static constexpr int buf = BN * (KP + VP);
    static constexpr int CH = DP / 8;           // 16-byte chunks per key
    static constexpr int KPI = THREADS / CH;   // keys per load of the workgroup
    static constexpr int NL = BN / KPI;         // loads per thread, K and V each
};

__device__ __forceinline__ float max_halves(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The row's maximum off its scores; nothing where it has seen none.
template <int NK>
__device__ __forceinline__ void subtract_max(f32x16 (&s)[NK], float m)
{
    const float sub = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int k = 0; k < NK; k++)
#pragma unroll
        for (int v = 0; v < 16; v++)
            s[k][v] -= sub;
}

// Heads of 64 fit three waves per SIMD in 168 registers, of 128 two in 256.
// Six prompts with a window, fp16 with an fp32 result: 272 us with two waves,
// 248 with three; with bf16's three terms 65 (2048 tokens) and 71. Heads of 256
// leave room for one: 2048 tokens, 16 heads over 2, bf16, two splits, 109 us
// (315 TFLOP/s; 132 for an fp32 result), the matrix pipe 19 % busy and nothing
// beside the wave that waits.
constexpr int waves_per_simd(int dp, int terms) { return dp <= 64 && terms < 3 ? 3 : dp <= 128 ? 2 : 1; }

template <class T, int DP, int TERMS>
__global__ __launch_bounds__(kThreads, waves_per_simd(DP, TERMS)) void attn_prefill_kernel(AttnArgs a)
{
    using L = Tile<DP>;
    constexpr int BN = L::BN, NC = DP / 16, ND = DP / 32, NK = BN / 32;
    __shared__ __align__(16) char smem[2 * L::buf];
    __shared__ unsigned s_bad[3][2]; // keys of a tile with an unusable page id
    __shared__ int s_ids[kIds];      // page ids of the next tiles, `ept` each

    const int tid = threadIdx.x, lane = tid & 63, r32 = lane & 31, hl = lane >> 5, i16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const KvArgs &kv = a.kv;
    // Splits vary slowest (see the decode kernel). kv heads vary fastest:
    // workgroups go round the XCDs in order, so with eight kv heads each
    // XCD's L2 holds one head's keys and values.
    const int split = a.div_units(blockIdx.x), b = a.div_units.rem(blockIdx.x, split);
    const int us = kv.div_hk(b), hk = kv.div_hk.rem(b, us);
    const int seq = a.div_rb(us), rb = a.row_blocks - 1 - a.div_rb.rem(us, seq); // the longest first
    const int unit = (seq * a.row_blocks + rb) * kv.Hk + hk;
    const int D = kv.D;
    const int window = a.window ? a.window : 1 << 30; // positions are below 2^30

    const Seq sq = load_seq(kv, seq);
    const int nrows = sq.nq * kv.G, row0 = rb * kRows;
    if (row0 >= nrows)
        return;
    const int row_end = min(nrows, row0 + kRows);
    const KeyTiles kt = key_tiles(BN, sq.p0 + kv.div_g(row0), sq.p0 + kv.div_g(row_end - 1), sq.kv, a.window, a.sinks);
    int per, active;
    split_tiles(a, kt.n, per, active);
    if (split >= active)
        return;
    const int t_begin = split * per, t_end = min(kt.n, t_begin + per);

    // the wave's rows
    const int wrow = row0 + 32 * wave;
    const bool wave_on = wrow < nrows;
    const int row = min(wrow + r32, nrows - 1), tok = kv.div_g(row), head = hk * kv.G + kv.div_g.rem(row, tok);
    const bool row_ok = wrow + r32 < nrows;
    const int pos = sq.p0 + tok;
    const int w_lo = sq.p0 + kv.div_g(min(wrow, nrows - 1)), w_hi = sq.p0 + kv.div_g(min(wrow + 31, nrows - 1));
    const size_t at = ((size_t)(sq.t0 + tok) * kv.Hq + head) * D;
    u4 qf[NC];
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int d = 16 * c + 8 * hl;
        const u4 x = *reinterpret_cast<const u4 *>(a.q + at + (d < D ? d : 0));
        qf[c] = d < D ? x : (u4){0, 0, 0, 0};
    }

    f32x16 acc[ND];
#pragma unroll
    for (int i = 0; i < ND; i++)
#pragma unroll
        for (int v = 0; v < 16; v++)
            acc[i][v] = 0.f;
    float m = -INFINITY, l = 0.f;
    bool far = false; // uniform

    // Page ids go through LDS, those of `ids_n` tiles from tile ids_at on, so
    // that a tile's loads need no other global load first.
    const int32_t *table = kv.table + (size_t)seq * kv.stride;
    const int last_key = max(0, kt.hi - 1), ps = kv.page_shift, pm = (1 << ps) - 1;
    const int ept = max(1, BN >> ps), ids_n = kIds / ept;
    int ids_at = t_begin;
    const auto fill_ids = [&](int t) {
        for (int e = tid; e < ids_n * ept; e += kThreads) {
            const int tt = t + e / ept;
            if (tt < t_end)
                s_ids[e] = table[min(tile_key<BN>(kt, tt) + ((e % ept) << ps), last_key) >> ps];
        }
    };

    // staging: this thread's chunk of NL keys of a tile
    const int skey = tid / L::CH, sch = tid % L::CH;
    const unsigned page_elems = (unsigned)kv.Hk * D << ps; // at most 2^30
    const size_t lane_off = ((size_t)hk * D << ps) + (8 * sch < D ? 8 * sch : 0);
    u4 kx[L::NL], vx[L::NL];
    unsigned bad_pages; // loads whose page id is unusable
    const auto load_tile = [&](int t) {
        const int key0 = tile_key<BN>(kt, t), at0 = (t - ids_at) * ept;
        bad_pages = 0;
#pragma unroll
        for (int i = 0; i < L::NL; i++) {
            const int kk = i * L::KPI + skey;
            const int id = s_ids[at0 + (kk >> ps)];
            const bool good = (unsigned)id < (unsigned)kv.n_pages;
            bad_pages |= good ? 0u : 1u << i;
            const size_t off = lane_off + (size_t)(good ? (unsigned)id : 0u) * page_elems + (unsigned)(((key0 + kk) & pm) * D);
            kx[i] = *reinterpret_cast<const u4 *>(kv.k + off);
            vx[i] = *reinterpret_cast<const u4 *>(kv.v + off);
        }
    };
    // Tile t, in the registers, into buffer bf. Keys that no row of the
    // workgroup sees, and elements past D, become zero: their memory may
    // hold anything.
    const auto store_tile = [&](int t, int bf) {
        const int key0 = tile_key<BN>(kt, t);
        char *kb = smem + bf * L::buf, *vb = kb + BN * L::KP;
        if (key0 + BN > kt.hi || (key0 < kt.lo && key0 + BN > kt.sk) || D != DP || __any(bad_pages)) {
#pragma unroll
            for (int i = 0; i < L::NL; i++) {
                const int kk = i * L::KPI + skey, key = key0 + kk;
                const bool good = !(bad_pages >> i & 1);
                if (!good && sch == 0)
                    atomicOr(&s_bad[t % 3][kk >> 5], 1u << (kk & 31));
                if (!(good & (8 * sch < D) & (key < kt.hi) & ((key >= kt.lo) | (key < kt.sk))))
                    kx[i] = vx[i] = (u4){0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int i = 0; i < L::NL; i++) {
            *reinterpret_cast<u4 *>(kb + (i * L::KPI + skey) * L::KP + 16 * sch) = kx[i];
            *reinterpret_cast<u4 *>(vb + (i * L::KPI + skey) * L::VP + 16 * sch) = vx[i];
        }
    };

    if (tid < 6)
        s_bad[tid >> 1][tid & 1] = 0;
    __syncthreads();
    if (t_begin < t_end) {
        fill_ids(t_begin);
        __syncthreads();
        load_tile(t_begin);
        store_tile(t_begin, t_begin & 1);
    }
    __syncthreads();

    for (int t = t_begin; t < t_end; t++) {
        // the next tile's loads (at the end, the last tile's again: on every
        // path, so that nothing waits for them before they are stored)
        const int tn = min(t + 1, t_end - 1);
        if (tn - ids_at >= ids_n) {
            fill_ids(tn); // every thread is past its reads of the old ids
            ids_at = tn;
            __syncthreads();
        }
        load_tile(tn);
        if (tid < 2)
            s_bad[(t + 2) % 3][tid] = 0; // last read for tile t - 1
        const int key0 = tile_key<BN>(kt, t);
        const char *kb = smem + (t & 1) * L::buf, *vb = kb + BN * L::KP;
        const bool seen = wave_on && key0 <= w_hi && (key0 + BN - 1 > w_lo - window || key0 < a.sinks);
        if (seen) {
            f32x16 s[NK];
#pragma unroll
            for (int k = 0; k < NK; k++)
#pragma unroll
                for (int v = 0; v < 16; v++)
                    s[k][v] = 0.f;
#pragma unroll
            for (int c = 0; c < NC; c++)
#pragma unroll
                for (int k = 0; k < NK; k++) {
                    const u4 kf = *reinterpret_cast<const u4 *>(kb + (32 * k + r32) * L::KP + 32 * c + 16 * hl);
                    s[k] = T::mma32(kf, qf[c], s[k]);
                }
            const unsigned bad0 = s_bad[t % 3][0], bad1 = s_bad[t % 3][1];
            const bool edge = key0 + BN - 1 > w_lo || (key0 <= w_hi - window && key0 + BN > a.sinks) || (bad0 | bad1);
            if (edge) {
#pragma unroll
                for (int k = 0; k < NK; k++)
#pragma unroll
                    for (int v = 0; v < 16; v++) {
                        const int kk = 8 * (v >> 2) + 4 * hl + (v & 3), key = key0 + 32 * k + kk;
                        const bool ok = (key <= pos) & ((key > pos - window) | (key < a.sinks)) & !(((k ? bad1 : bad0) >> kk) & 1);
                        s[k][v] = ok ? s[k][v] : -INFINITY;
                    }
            }
            float top = s[0][0];
#pragma unroll
            for (int k = 0; k < NK; k++)
#pragma unroll
                for (int v = 0; v < 16; v++)
                    top = fmaxf(top, s[k][v]);
            top = max_halves(top);
            // Weights may grow to 2^LAG before the sums are rescaled: the
            // largest score rises often by a little, seldom by much.
            if (__any(a.c * (top - m) > T::LAG)) {
                const float mn = fmaxf(m, top), f = m == -INFINITY ? 0.f : fast_exp2(a.c * (m - mn));
                l *= f;
#pragma unroll
                for (int i = 0; i < ND; i++)
                    acc[i] *= f;
                m = mn;
                far = __any((mn != -INFINITY) & (a.c * fabsf(mn) > kFar));
            }
            __builtin_amdgcn_s_setprio(1); // the other wave of the SIMD waits rather than this one: 587 to 572 us
            float off = m == -INFINITY ? 0.f : T::BIAS - a.c * m;
            if (far) {
                off = T::BIAS;
                subtract_max<NK>(s, m);
            }
#pragma unroll
            for (int k = 0; k < NK; k++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    float p[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        p[i] = fast_exp2(fmaf(a.c, s[k][8 * h + i], off));
                        if (TERMS > 1)
                            l += p[i];
                    }
                    u4 pt[TERMS];
                    split_terms<T, TERMS>(p, pt);
                    if (TERMS == 1) // the sum of the weights as they are used
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            l = T::add_pair(pt[0][i], l);
                    // values of keys 32 k + 16 h + 4 hl + 0..3 and + 8..11
                    const char *vr = vb + (32 * k + 16 * h + 4 * hl + (i16 >> 2)) * L::VP + 32 * ((lane >> 4) & 1) + 8 * (i16 & 3);
#pragma unroll
                    for (int i = 0; i < ND; i++) {
                        const u2 x = lds_read_tr(vr + 64 * i), y = lds_read_tr(vr + 8 * L::VP + 64 * i);
                        const u4 vt = {x.x, x.y, y.x, y.y};
#pragma unroll
                        for (int n = 0; n < TERMS; n++)
                            acc[i] = T::mma32(vt, pt[n], acc[i]);
                    }
                }
        }
        __builtin_amdgcn_s_setprio(0);
        store_tile(tn, (t + 1) & 1);
        __syncthreads();
    }

    l += __shfl_xor(l, 32, 64);
    // lane (row r32), register 4 j + v of acc[i]: element 32 i + 8 j + 4 hl + v
    if (active == 1) {
        if (!row_ok)
            return;
        const float inv = l > 0.f ? 1.0f / l : 0.f; // a row that sees nothing is zero
#pragma unroll
        for (int i = 0; i < ND; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int d = 32 * i + 8 * j + 4 * hl;
                if (d >= D)
                    continue;
                const f32x4 o = {acc[i][4 * j] * inv, acc[i][4 * j + 1] * inv, acc[i][4 * j + 2] * inv, acc[i][4 * j + 3] * inv};
                if (a.out_f32)
                    *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + at + d) = o;
                else
                    *reinterpret_cast<u2 *>(static_cast<uint16_t *>(a.out) + at + d) = (u2){T::pack(o[0], o[1]), T::pack(o[2], o[3])};
            }
        return;
    }

    if (!row_ok)
        return;
    const size_t slot = ((size_t)unit * a.S + split) * kRows + 32 * wave + r32;
#pragma unroll
    for (int i = 0; i < ND; i++)
#pragma unroll
        for (int j = 0; j < 4; j++)
            *reinterpret_cast<f32x4 *>(a.part + slot * DP + 32 * i + 8 * j + 4 * hl) =
                (f32x4){acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]};
    if (hl == 0)
        *reinterpret_cast<f2 *>(a.stat + slot * 2) = (f2){m, l};
}

// The same for many rows and heads of up to 128: eight waves and 256 rows,
// in two groups of four (one wave of each on every SIMD) that take turns,
// half a tile apart. While one group's waves run the products of PV (tile j)
// and QK (tile j + 1) with the tiles' staging between them, the other's run
// the softmax of theirs, so that the matrix and the vector pipe of a SIMD
// have one wave each; a barrier ends every phase. A key tile's staging serves
// twice the rows. Three buffers: a tile is in LDS a tile ahead of its
// products, so that their first operands are read during the softmax before
// (514 us with two buffers and those reads at the start of the products).
// 8192 tokens of 32 heads of 128 over 8, bf16: 500 us (1100 TFLOP/s), 586 with
// the kernel above, whose two waves per SIMD meet on the same pipe as often
// as not. Where the staging and the packing of weights stand, and a shorter
// path for tiles without a mask, move this by less than 1 %. By counters the
// matrix pipe is busy 58 % and the vector pipe 50 % of the time; what holds the
// rest was not found (a large library product reaches 1371 TFLOP/s; power was
// not recorded). An fp32 result (three terms, twice the products in all) takes
// 864 us, the matrix pipe 74 % busy.
__device__ __forceinline__ void phase_end()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F); // lgkmcnt(0): LDS writes are done; global loads stay in flight
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

template <class T, int TERMS>
__global__ __launch_bounds__(512, 2) void attn_pair_kernel(AttnArgs a)
{
    constexpr int DP = 128;
    using L = Tile<DP, 512>;
    constexpr int BN = L::BN, NC = DP / 16, ND = DP / 32, NK = BN / 32, ROWS = kPairRows;
    __shared__ __align__(16) char smem[3 * L::buf];
    __shared__ int s_ids[kPairIds];  // page ids of the tiles, `ept` each, 0 for unusable ones
    __shared__ unsigned s_bad[kPairIds / 32]; // a bit for each of those
    __shared__ unsigned s_any_bad;

    const int tid = threadIdx.x, lane = tid & 63, r32 = lane & 31, hl = lane >> 5, i16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), grp = wave >> 2;
    const KvArgs &kv = a.kv;
    const int split = a.div_units(blockIdx.x), b = a.div_units.rem(blockIdx.x, split);
    const int us = kv.div_hk(b), hk = kv.div_hk.rem(b, us);
    const int seq = a.div_rb(us), rb = a.row_blocks - 1 - a.div_rb.rem(us, seq); // the longest first
    const int unit = (seq * a.row_blocks + rb) * kv.Hk + hk;
    const int D = kv.D;
    const int window = a.window ? a.window : 1 << 30;

    const Seq sq = load_seq(kv, seq);
    const int nrows = sq.nq * kv.G, row0 = rb * ROWS;
    if (row0 >= nrows)
        return;
    const int row_end = min(nrows, row0 + ROWS);
    const KeyTiles kt = key_tiles(BN, sq.p0 + kv.div_g(row0), sq.p0 + kv.div_g(row_end - 1), sq.kv, a.window, a.sinks);
    int per, active;
    split_tiles(a, kt.n, per, active);
    if (split >= active)
        return;
    const int t0 = split * per, n = min(kt.n, t0 + per) - t0;

    const int wrow = row0 + 32 * wave;
    const int row = min(wrow + r32, nrows - 1), tok = kv.div_g(row), head = hk * kv.G + kv.div_g.rem(row, tok);
    const bool row_ok = wrow + r32 < nrows;
    const int pos = sq.p0 + tok;
    const int w_lo = sq.p0 + kv.div_g(min(wrow, nrows - 1)), w_hi = sq.p0 + kv.div_g(min(wrow + 31, nrows - 1));
    const size_t at = ((size_t)(sq.t0 + tok) * kv.Hq + head) * D;
    u4 qf[NC];
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int d = 16 * c + 8 * hl;
        const u4 x = *reinterpret_cast<const u4 *>(a.q + at + (d < D ? d : 0));
        qf[c] = d < D ? x : (u4){0, 0, 0, 0};
    }

    f32x16 acc[ND];
#pragma unroll
    for (int i = 0; i < ND; i++)
#pragma unroll
        for (int v = 0; v < 16; v++)
            acc[i][v] = 0.f;
    float m = -INFINITY, l = 0.f;
    bool far = false; // uniform

    const int32_t *table = kv.table + (size_t)seq * kv.stride;
    const int last_key = max(0, kt.hi - 1), ps = kv.page_shift, pm = (1 << ps) - 1;
    const int ept = max(1, BN >> ps);
    if (tid < kPairIds / 32)
        s_bad[tid] = 0;
    if (tid == 0)
        s_any_bad = 0;
    __syncthreads();
    for (int e = tid; e < n * ept; e += 512) {
        const int id = table[min(tile_key<BN>(kt, t0 + e / ept) + ((e % ept) << ps), last_key) >> ps];
        const bool good = (unsigned)id < (unsigned)kv.n_pages;
        s_ids[e] = good ? id : 0;
        if (!good) {
            atomicOr(&s_bad[e >> 5], 1u << (e & 31));
            s_any_bad = 1;
        }
    }
    __syncthreads();
    const bool any_bad = __builtin_amdgcn_readfirstlane(s_any_bad) != 0;
    const auto key_bad = [&](int jj, int kk) {
        const int e = jj * ept + (kk >> ps);
        return s_bad[e >> 5] >> (e & 31) & 1;
    };

    // staging: this thread's chunk of NL keys of a tile; keys and values of
    // different tiles
    const int skey = tid / L::CH, sch = tid % L::CH;
    const unsigned page_elems = (unsigned)kv.Hk * D << ps; // at most 2^30
    const size_t lane_off = ((size_t)hk * D << ps) + (8 * sch < D ? 8 * sch : 0);
    u4 kx[L::NL], vx[L::NL];
    size_t at_k[L::NL], at_v[L::NL]; // elements
    unsigned ids[L::NL];
    const auto read_ids = [&](int j) {
#pragma unroll
        for (int i = 0; i < L::NL; i++)
            ids[i] = (unsigned)s_ids[min(j, n - 1) * ept + ((i * L::KPI + skey) >> ps)];
    };
    const auto load_keys = [&](int j) { // after read_ids(j)
        const int key0 = tile_key<BN>(kt, t0 + min(j, n - 1));
#pragma unroll
        for (int i = 0; i < L::NL; i++) {
            const int kk = i * L::KPI + skey;
            at_k[i] = (uint64_t)ids[i] * page_elems + (lane_off + (unsigned)(((key0 + kk) & pm) * D));
            kx[i] = *reinterpret_cast<const u4 *>(kv.k + at_k[i]);
        }
    };
    const auto load_values = [&] { // of the tile whose keys came last but one
#pragma unroll
        for (int i = 0; i < L::NL; i++)
            vx[i] = *reinterpret_cast<const u4 *>(kv.v + at_v[i]);
    };
    // Keys that no row of the workgroup sees, and elements past D, become
    // zero.
    const auto clear_rows = [&](int j, u4 (&x)[L::NL]) {
        const int jj = min(j, n - 1), key0 = tile_key<BN>(kt, t0 + jj);
        if (key0 + BN > kt.hi || (key0 < kt.lo && key0 + BN > kt.sk) || D != DP || any_bad) {
#pragma unroll
            for (int i = 0; i < L::NL; i++) {
                const int kk = i * L::KPI + skey, key = key0 + kk;
                if (!((8 * sch < D) & (key < kt.hi) & ((key >= kt.lo) | (key < kt.sk)) & !key_bad(jj, kk)))
                    x[i] = (u4){0, 0, 0, 0};
            }
        }
    };
    char *const kbase = smem, *const vbase = smem + BN * L::KP;
    const auto store_rows = [&](char *base, int pitch, const u4 (&x)[L::NL]) {
#pragma unroll
        for (int i = 0; i < L::NL; i++)
            *reinterpret_cast<u4 *>(base + (i * L::KPI + skey) * pitch + 16 * sch) = x[i];
    };
    // Tile j lives in buffer j % 3. Staging beside the products of tile j:
    // keys of j + 2 and values of j + 1 to LDS, the next ones' loads.
    const auto stage_clear = [&](int j) {
        clear_rows(j + 2, kx);
        clear_rows(j + 1, vx);
    };
    const auto stage = [&](int j, int part, int kbuf, int vbuf) {
        if (part == 0)
            store_rows(kbase + kbuf, L::KP, kx);
        if (part == 1) {
            store_rows(vbase + vbuf, L::VP, vx);
            read_ids(j + 3);
        }
        if (part == 2) {
#pragma unroll
            for (int i = 0; i < L::NL; i++)
                at_v[i] = at_k[i];
            load_values();
        }
        if (part == 3)
            load_keys(j + 3);
    };

    f32x16 s[NK];
    u4 pt[2][TERMS];
    // Fragments are read one step of four products ahead.
    u4 fr[2][4];
    const auto read_k = [&](int buf, int st, u4 (&f)[4]) {
        const char *kb = kbase + buf + r32 * L::KP + 16 * hl;
#pragma unroll
        for (int i = 0; i < 4; i++)
            f[i] = *reinterpret_cast<const u4 *>(kb + 32 * (i & 1) * L::KP + 32 * (2 * st + (i >> 1)));
    };
    const auto read_v = [&](int buf, int st, u4 (&f)[4]) {
        const char *vr = vbase + buf + (16 * st + 4 * hl + (i16 >> 2)) * L::VP + 32 * ((lane >> 4) & 1) + 8 * (i16 & 3);
#pragma unroll
        for (int i = 0; i < ND; i++) {
            const u2 x = lds_read_tr(vr + 64 * i), y = lds_read_tr(vr + 8 * L::VP + 64 * i);
            f[i] = (u4){x.x, x.y, y.x, y.y};
        }
    };
    // a step's products with whatever else is in its region between them
    const auto mix = [&](int products) {
#pragma unroll
        for (int i = 0; i < products; i++) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002 | 0x020 | 0x100 | 0x200, 4, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    // Tile j's, with its staging (to the keys' buffer kbuf and the values'
    // vbuf); read_k(buf, 0, fr[0]) is done.
    const auto scores = [&](int buf, int j, int kbuf, int vbuf) {
#pragma unroll
        for (int k = 0; k < NK; k++)
#pragma unroll
            for (int v = 0; v < 16; v++)
                s[k][v] = 0.f;
#pragma unroll
        for (int st = 0; st < NC / 2; st++) {
            if (st + 1 < NC / 2)
                read_k(buf, st + 1, fr[~st & 1]);
#pragma unroll
            for (int i = 0; i < 4; i++)
                s[i & 1] = T::mma32(fr[st & 1][i], qf[2 * st + (i >> 1)], s[i & 1]);
            stage(j, st, kbuf, vbuf);
            mix(4);
        }
    };
    // weights of 16 keys as operands, and their sums: beside the products of
    // the 16 before
    const auto pack = [&](int st) {
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            p[i] = s[st >> 1][8 * (st & 1) + i];
            if (TERMS > 1)
                l += p[i];
        }
        split_terms<T, TERMS>(p, pt[st & 1]);
        if (TERMS == 1) // the sum of the weights as they are used
#pragma unroll
            for (int i = 0; i < 4; i++)
                l = T::add_pair(pt[st & 1][0][i], l);
    };
    const auto weights = [&](int j) {
        const int key0 = tile_key<BN>(kt, t0 + j);
        unsigned bad0 = 0, bad1 = 0;
        if (any_bad) {
#pragma unroll 1
            for (int kk = 0; kk < 32; kk++) {
                bad0 |= key_bad(j, kk) << kk;
                bad1 |= key_bad(j, 32 + kk) << kk;
            }
        }
        bad0 >>= 4 * hl;
        bad1 >>= 4 * hl;
        const bool edge = any_bad || key0 + BN - 1 > w_lo || (key0 <= w_hi - window && key0 + BN > a.sinks);
        if (edge) {
            int first = key0 + 4 * hl; // opaque: else the compiler keeps the keys' numbers in registers around the loop
            asm volatile("" : "+v"(first));
#pragma unroll
            for (int k = 0; k < NK; k++)
#pragma unroll
                for (int v = 0; v < 16; v++) {
                    const int kk = 8 * (v >> 2) + (v & 3), key = first + 32 * k + kk;
                    const bool ok = (key <= pos) & ((key > pos - window) | (key < a.sinks)) & !(((k ? bad1 : bad0) >> kk) & 1);
                    s[k][v] = ok ? s[k][v] : -INFINITY;
                }
        }
        float top = s[0][0];
#pragma unroll
        for (int k = 0; k < NK; k++)
#pragma unroll
            for (int v = 0; v < 16; v++)
                top = fmaxf(top, s[k][v]);
        top = max_halves(top);
        if (__any(a.c * (top - m) > T::LAG)) {
            const float mn = fmaxf(m, top), f = m == -INFINITY ? 0.f : fast_exp2(a.c * (m - mn));
            l *= f;
#pragma unroll
            for (int i = 0; i < ND; i++)
                acc[i] *= f;
            m = mn;
            far = __any((mn != -INFINITY) & (a.c * fabsf(mn) > kFar));
        }
        float off = m == -INFINITY ? 0.f : T::BIAS - a.c * m;
        if (far) {
            off = T::BIAS;
            subtract_max<NK>(s, m);
        }
#pragma unroll
        for (int k = 0; k < NK; k++)
#pragma unroll
            for (int v = 0; v < 16; v++)
                s[k][v] = fast_exp2(fmaf(a.c, s[k][v], off));
        pack(0);
    };
    // Tile j's, buffer b0, the next tile's b1; read_v(b0, 0, fr[0]) is done.
    const auto results = [&](int b0, int b1) {
#pragma unroll
        for (int st = 0; st < 2 * NK; st++) {
            if (st + 1 < 2 * NK) {
                read_v(b0, st + 1, fr[~st & 1]);
                pack(st + 1);
            } else
                read_k(b1, 0, fr[0]); // for the scores that follow (at the end unused)
#pragma unroll
            for (int i = 0; i < ND; i++)
#pragma unroll
                for (int t = 0; t < TERMS; t++)
                    acc[i] = T::mma32(fr[st & 1][i], pt[st & 1][t], acc[i]);
            mix(ND * TERMS);
        }
    };

    if (n > 0) {
        int b0 = 0, b1 = L::buf, b2 = 2 * L::buf;
        read_ids(0);
        load_keys(0);
        clear_rows(0, kx);
        store_rows(kbase + b0, L::KP, kx);
        stage(-2, 2, 0, 0); // values of tile 0
        read_ids(1);
        load_keys(1);
        clear_rows(0, vx);
        store_rows(vbase + b0, L::VP, vx);
        clear_rows(1, kx);
        store_rows(kbase + b1, L::KP, kx);
        stage(-1, 2, 0, 0); // values of tile 1
        read_ids(2);
        load_keys(2);
        phase_end();
        if (grp) // group 1 runs one phase behind
            phase_end();
        stage_clear(0);
        read_k(b0, 0, fr[0]);
        scores(b0, 0, b2, b1);
        for (int j = 0; j + 1 < n; j++) {
            phase_end();
            read_v(b0, 0, fr[0]);
            weights(j);
            stage_clear(j + 1);
            phase_end();
            __builtin_amdgcn_s_setprio(1);
            results(b0, b1);
            scores(b1, j + 1, b0, b2);
            __builtin_amdgcn_s_setprio(0);
            const int t = b0;
            b0 = b1;
            b1 = b2;
            b2 = t;
        }
        phase_end();
        read_v(b0, 0, fr[0]);
        weights(n - 1);
        phase_end();
        results(b0, b1);
        if (grp == 0)
            phase_end();
    }

    l += __shfl_xor(l, 32, 64);
    if (active == 1) {
        if (!row_ok)
            return;
        const float inv = l > 0.f ? 1.0f / l : 0.f;
#pragma unroll
        for (int i = 0; i < ND; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int d = 32 * i + 8 * j + 4 * hl;
                if (d >= D)
                    continue;
                const f32x4 o = {acc[i][4 * j] * inv, acc[i][4 * j + 1] * inv, acc[i][4 * j + 2] * inv, acc[i][4 * j + 3] * inv};
                if (a.out_f32)
                    *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + at + d) = o;
                else
                    *reinterpret_cast<u2 *>(static_cast<uint16_t *>(a.out) + at + d) = (u2){T::pack(o[0], o[1]), T::pack(o[2], o[3])};
            }
        return;
    }
    if (!row_ok)
        return;
    const size_t slot = ((size_t)unit * a.S + split) * ROWS + 32 * wave + r32;
#pragma unroll
    for (int i = 0; i < ND; i++)
#pragma unroll
        for (int j = 0; j < 4; j++)
            *reinterpret_cast<f32x4 *>(a.part + slot * DP + 32 * i + 8 * j + 4 * hl) =
                (f32x4){acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]};
    if (hl == 0)
        *reinterpret_cast<f2 *>(a.stat + slot * 2) = (f2){m, l};
}

template <class T, int DP>
int launch(const AttnArgs &a, hipStream_t st)
{
    const unsigned grid = (unsigned)a.kv.n_seq * a.kv.Hk * a.row_blocks * a.S;
    if constexpr (DP == 128)
        if (a.rows == kPairRows) {
            if (a.out_f32)
                hipLaunchKernelGGL((attn_pair_kernel<T, T::TERMS>), dim3(grid), dim3(512), 0, st, a);
            else
                hipLaunchKernelGGL((attn_pair_kernel<T, 1>), dim3(grid), dim3(512), 0, st, a);
            return hip_status("attn prefill launch");
        }
    if (a.out_f32)
        hipLaunchKernelGGL((attn_prefill_kernel<T, DP, T::TERMS>), dim3(grid), dim3(kThreads), 0, st, a);
    else
        hipLaunchKernelGGL((attn_prefill_kernel<T, DP, 1>), dim3(grid), dim3(kThreads), 0, st, a);
    return hip_status("attn prefill launch");
}

template <class T>
int launch_dim(const AttnArgs &a, hipStream_t st)
{
    return a.kv.D <= 64 ? launch<T, 64>(a, st) : a.kv.D <= 128 ? launch<T, 128>(a, st) : launch<T, 256>(a, st);
}

} // namespace

namespace rfx {

int attn_prefill_launch(const AttnArgs &a, int type, hipStream_t st)
{
    return type == RFX_BF16 ? launch_dim<BF16>(a, st) : launch_dim<F16>(a, st);
}

} // namespace rfx
