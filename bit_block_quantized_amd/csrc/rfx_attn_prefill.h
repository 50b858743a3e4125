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
// With SharedArgs the rows are those of a whole group of sequences and the
// keys the prefix that they share, which all rows see (rfx_attn_shared).
// Few row blocks over long sequences: the keys are split over S workgroups
// and a second launch joins the partials in split order.
//
// Rounding: weights are rounded once to the cache's type for a result of
// that type (its own rounding is as large), and the row sums are of the
// rounded ones; for an fp32 result, and for a shared prefix, they are carried as
// the sum of TERMS values, and the sums are of the fp32 weights.
#pragma once

#include <type_traits>

#include "rfx_kv.h"

namespace rfx {
namespace dev {
namespace prefill {

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

__device__ __forceinline__ const AttnArgs &launch_of(const AttnArgs &a) { return a; }
__device__ __forceinline__ const AttnArgs &launch_of(const SharedArgs &a) { return a.group; }

// Workgroup `block` of the launch. smem: 2 * Tile<DP>::buf bytes; s_bad: keys of
// a tile with an unusable page id; s_ids: kIds page ids of the next tiles.
template <class T, int DP, int TERMS, class Args>
__device__ __forceinline__ void attention(const Args &args, int block, char *smem, unsigned (*s_bad)[2], int *s_ids)
{
    constexpr bool SHARED = std::is_same_v<Args, SharedArgs>;
    const AttnArgs &a = launch_of(args);
    using L = Tile<DP>;
    constexpr int BN = L::BN, NC = DP / 16, ND = DP / 32, NK = BN / 32;
    const int tid = threadIdx.x, lane = tid & 63, r32 = lane & 31, hl = lane >> 5, i16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const KvArgs &kv = a.kv;
    // Splits vary slowest (see the decode kernel). kv heads vary fastest:
    // workgroups go round the XCDs in order, so with eight kv heads each
    // XCD's L2 holds one head's keys and values.
    const int split = a.div_units(block), b = a.div_units.rem(block, split);
    const int us = kv.div_hk(b), hk = kv.div_hk.rem(b, us);
    int seq = a.div_rb(us);
    const int rb = a.row_blocks - 1 - a.div_rb.rem(us, seq); // the longest first
    const int unit = (seq * a.row_blocks + rb) * kv.Hk + hk;
    const int D = kv.D;
    const int window = !SHARED && a.window ? a.window : 1 << 30; // positions are below 2^30
    const int sinks = SHARED ? 0 : a.sinks;

    Seq sq;
    if constexpr (SHARED) {
        const Group gr = load_group(kv, args.pre, seq);
        seq = gr.s0;
        sq = {gr.t0, gr.nt, gr.len - 1, gr.len}; // as if at the last key
    } else {
        sq = load_seq(kv, seq);
    }
    const int nrows = sq.nq * kv.G, row0 = rb * kRows;
    if (row0 >= nrows)
        return;
    const int row_end = min(nrows, row0 + kRows);
    const KeyTiles kt = SHARED ? range_tiles(BN, 0, sq.kv)
                               : key_tiles(BN, sq.p0 + kv.div_g(row0), sq.p0 + kv.div_g(row_end - 1), sq.kv, a.window, a.sinks);
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
    // every key of a shared prefix is before every row
    const int pos = SHARED ? sq.p0 : sq.p0 + tok;
    const int w_lo = SHARED ? pos : sq.p0 + kv.div_g(min(wrow, nrows - 1)), w_hi = SHARED ? pos : sq.p0 + kv.div_g(min(wrow + 31, nrows - 1));
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
        const bool seen = wave_on && key0 <= w_hi && (key0 + BN - 1 > w_lo - window || key0 < sinks);
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
            const bool edge = key0 + BN - 1 > w_lo || (key0 <= w_hi - window && key0 + BN > sinks) || (bad0 | bad1);
            if (edge) {
#pragma unroll
                for (int k = 0; k < NK; k++)
#pragma unroll
                    for (int v = 0; v < 16; v++) {
                        const int kk = 8 * (v >> 2) + 4 * hl + (v & 3), key = key0 + 32 * k + kk;
                        const bool ok = (key <= pos) & ((key > pos - window) | (key < sinks)) & !(((k ? bad1 : bad0) >> kk) & 1);
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
    if (!SHARED && active == 1) {
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

} // namespace prefill
} // namespace dev
} // namespace rfx
