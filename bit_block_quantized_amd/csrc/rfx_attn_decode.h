// Attention of few new tokens per sequence over the paged cache (decode and
// speculative verification): o = softmax(scale q k^T + mask) v for the up to
// 32 query rows (tokens x query heads of a group) that share a kv head.
//
// Bound by the cache's bytes where there are many of them (1.6 GB at 5.9
// TB/s): every visible key and value is read once, for all rows of its kv
// head. Smaller calls are bound by latency: four tokens of eight sequences of
// 4000 to 8192 keys, 32 rows, take 22 us (and 4.5 for the join) for 90 MB with
// the matrix pipe 11 % and the vector pipe 21 % busy; a wave's four tiles come
// after three dependent loads, one in flight at a time. A wave takes tiles of
// 32 keys; its keys and values of the next tile are in flight while it
// computes the current one.
//   S^T = K Q^T on v_mfma_f32_16x16x32: A = 16 keys straight from memory, B =
//   the rows' queries (registers, loaded once). A lane ends with scores of one
//   row. The keys' order inside a tile is chosen so that they are 8 (l / 16)
//   .. + 7, which is the B operand's order of
//   O^T = V^T P^T: the weights go from S to the next product without leaving
//   their lane. V^T comes from LDS (each wave its own 32 x D piece, no
//   barrier) by transposed reads.
// Each wave keeps a running maximum and sum per row (fp32); waves are joined
// through LDS, and where few rows have long sequences the keys are split
// over S workgroups whose partials a second launch joins in split order.
//
// The same kernel serves rfx_attn_shared, with SharedArgs: some workgroups
// take the rows of a whole group of sequences against the prefix that they
// share, the others a sequence's rows against its own keys behind the prefix;
// both leave partials for the join.
#pragma once

#include <type_traits>

#include "rfx_kv.h"

namespace rfx {
namespace dev {
namespace decode {

constexpr int kWaves = 4;
constexpr int BN = 32;                  // keys per wave and tile
constexpr int kWaitVmcnt0 = 0x0F70;     // s_waitcnt vmcnt(0)

// LDS bytes: each wave's V piece, reused for the waves' join
// ([wave][16 rows][DP + 4] floats).
template <int DP>
constexpr int lds_bytes()
{
    constexpr int v = kWaves * BN * (DP * 2 + 32), o = kWaves * 16 * (DP + 4) * 4;
    return v > o ? v : o;
}

// Key (of a tile's 32) that sits in row r of the wave's V piece: the four
// rows that a group of 16 lanes reads at once are neighbours, so that with a
// pitch of 2 D + 32 bytes the groups' rows fall on different banks.
__device__ __forceinline__ int row_key(int r) { return (r & 3) + 8 * ((r >> 2) & 3) + 4 * (r >> 4); }

// The largest of the four lanes l % 16, one of each group of 16.
__device__ __forceinline__ float max_groups(float x)
{
    auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// How a tile's keys lie in pages. kOne: pages of 32 tokens or more, a tile
// in one; kTwo: pages of 16, two per tile; both with heads of exactly DP
// elements, so that a tile's addresses are one or two uniform bases, offsets
// that the lane keeps, and immediates (few waves run at once in a small
// call, and one wave issues an instruction every 8 cycles: the loop's length
// in instructions is its time). kAny: smaller pages, or heads that do not
// fill DP.
enum Pages { kOne, kTwo, kAny };

// The launch that a workgroup belongs to.
__device__ __forceinline__ const AttnArgs &launch_of(const AttnArgs &a, bool) { return a; }
__device__ __forceinline__ const AttnArgs &launch_of(const SharedArgs &a, bool group) { return group ? a.group : a.own; }

// Workgroup `block` of the launch. smem: lds_bytes<DP>() bytes; s_m, s_l: each
// wave's maxima and sums of NR * 16 rows.
template <class T, int DP, int NR, Pages PG, class Args>
__device__ __forceinline__ void attention(const Args &args, int block, char *smem, float (*s_m)[NR * 16], float (*s_l)[NR * 16])
{
    constexpr bool SHARED = std::is_same_v<Args, SharedArgs>;
    constexpr int NC = DP / 32;         // K steps of the score product
    constexpr int NV = DP / 16;         // 16-byte loads per lane and V tile; also 16-row tiles of O^T
    constexpr int CH = DP / 8;          // 16-byte chunks per key
    constexpr int RPI = 64 / CH;        // keys per V load instruction
    constexpr int VP = DP * 2 + 32;     // pitch of the V piece
    constexpr int TERMS = T::TERMS;
    const int lane = threadIdx.x & 63, r16 = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    bool group = false; // the rows of a group of sequences
    if constexpr (SHARED) {
        group = block < args.group_blocks;
        block -= group ? 0 : args.group_blocks;
    }
    const AttnArgs &a = launch_of(args, group);
    const KvArgs &kv = a.kv;
    // splits vary slowest: those that a short sequence leaves empty are the
    // last of the launch, and the others spread over all compute units (18 to
    // 14 us at 8192 keys with the splits of one unit side by side)
    const int split = a.div_units(block), unit = a.div_units.rem(block, split);
    int seq = kv.div_hk(unit);
    const int hk = kv.div_hk.rem(unit, seq);
    const int D = PG == kAny ? kv.D : DP;
    const int window = !SHARED && a.window ? a.window : 1 << 30; // positions are below 2^30

    Seq sq;
    int row0 = 0;        // of the block
    bool alone = true;   // no prefix beside these keys
    KeyTiles kt;
    if constexpr (SHARED) {
        Group gr;
        if (group) { // all of its keys are before all of its rows
            const int g = a.div_rb(seq);
            row0 = a.div_rb.rem(seq, g) * NR * 16;
            gr = load_group(kv, args.pre, g);
            seq = gr.s0;
            sq = {gr.t0, gr.nt, gr.len - 1, gr.len}; // as if at the last key
            kt = range_tiles(BN, 0, gr.len);
        } else {
            int g;
            sq = load_seq_prefix(kv, args.pre, seq, g, gr);
            kt = range_tiles(BN, gr.len, min(sq.kv, sq.p0 + sq.nq));
            if (split == 0 && threadIdx.x == 0) {
                int per, n_own, n_group = 0;
                split_tiles(a, kt.n, per, n_own);
                if (gr.len)
                    split_tiles(args.group, range_tiles(args.group.bn, 0, gr.len).n, per, n_group);
                args.units[unit] = {sq.t0, sq.nq, n_own, n_group, g, (sq.t0 - gr.t0) * kv.G};
            }
        }
        alone = !group && gr.len == 0;
    } else {
        sq = load_seq(kv, seq);
    }
    const int nrows = min(sq.nq * kv.G - row0, NR * 16);
    if (nrows <= 0)
        return;
    const int p_lo = sq.p0, p_hi = group ? sq.p0 : sq.p0 + kv.div_g(nrows - 1);
    if constexpr (!SHARED)
        kt = key_tiles(BN, p_lo, p_hi, sq.kv, a.window, a.sinks);
    int per, active;
    split_tiles(a, kt.n, per, active);
    if (split >= active)
        return;
    const int t_begin = split * per + wave, t_end = min(kt.n, (split + 1) * per);

    // this lane's row of each row tile: its query as the B operand (lane l:
    // row l % 16, elements 32 c + 8 (l / 16) .. + 7) and its position
    u4 qf[NR][NC];
    int pos[NR];
#pragma unroll
    for (int n = 0; n < NR; n++) {
        const int row = 16 * n + r16, rr = row0 + min(row, nrows - 1), tok = kv.div_g(rr), head = hk * kv.G + kv.div_g.rem(rr, tok);
        pos[n] = group ? sq.p0 : sq.p0 + tok;
        const uint16_t *qp = a.q + ((size_t)(sq.t0 + tok) * kv.Hq + head) * D;
#pragma unroll
        for (int c = 0; c < NC; c++) {
            const int d = 32 * c + 8 * g4;
            const u4 x = *reinterpret_cast<const u4 *>(qp + (d < D ? d : 0));
            qf[n][c] = d < D ? x : (u4){0, 0, 0, 0};
        }
    }

    f32x4 acc[NR][NV];
    float m[NR], l[NR];
    bool far[NR]; // uniform
#pragma unroll
    for (int n = 0; n < NR; n++) {
        far[n] = false;
        m[n] = -INFINITY;
        l[n] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; i++)
            acc[n][i] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }

    const int32_t *table = kv.table + (size_t)seq * kv.stride;
    const int last_key = max(0, kt.hi - 1);
    const int ps = kv.page_shift, pm = (1 << ps) - 1;
    const unsigned page_elems = (unsigned)kv.Hk * D << ps;  // at most 2^30
    const size_t head_off = (size_t)hk * D << ps;
    const int ka = 8 * (r16 >> 2) + (r16 & 3);              // the lane's keys of a tile: ka and ka + 4
    const int vrow = lane / CH, vch = 8 * (lane % CH) < D ? 8 * (lane % CH) : 0;
    char *vbuf = smem + wave * (BN * VP);
    const auto usable = [&](int id) { return (unsigned)id < (unsigned)kv.n_pages; };

    // Page ids. kOne, kTwo: lane i holds the i-th id of the wave's next
    // tiles, refilled when they run out; id[h] is uniform. kAny: lane i holds
    // the id of key i % 32 of one tile.
    constexpr int HALVES = PG == kTwo ? 2 : 1;
    struct Ids {
        int id[HALVES];
    };
    int ids = 0, ids_at = 0;   // ids of tiles ids_at, ids_at + kWaves, ...
    const auto fill_ids = [&](int t) {
        const int key = min(tile_key<BN>(kt, min(t + kWaves * (lane / HALVES), kt.n - 1)) + 16 * (lane % HALVES), last_key);
        ids = table[key >> ps];
        ids_at = t;
    };
    const auto uniform_ids = [&](int t) {
        Ids u;
#pragma unroll
        for (int h = 0; h < HALVES; h++)
            u.id[h] = __builtin_amdgcn_readlane(ids, HALVES * ((t - ids_at) / kWaves) + h);
        return u;
    };
    const auto lane_ids = [&](int t) { return Ids{{table[min(tile_key<BN>(kt, t) + (lane & 31), last_key) >> ps]}}; };
    // the first element of this head in the page, and of the tile's slots there
    const auto base = [&](const uint16_t *cache, int id, int key0) {
        return cache + head_off + (size_t)(unsigned)(usable(id) ? id : 0) * page_elems + (PG == kAny ? 0 : (key0 & pm) * D);
    };

    u4 kf[2][NC], vf[NV];
    // The loads of a tile; addresses are always inside the cache.
    const auto load_k = [&](int key0, const Ids &u) {
        const uint16_t *p;
        if constexpr (PG == kOne)
            p = base(kv.k, u.id[0], key0) + (unsigned)(ka * D + 8 * g4);
        else if constexpr (PG == kTwo)
            p = (r16 < 8 ? base(kv.k, u.id[0], 0) : base(kv.k, u.id[1], 0)) + (unsigned)((ka & 15) * D + 8 * g4);
#pragma unroll
        for (int j = 0; j < 2; j++) {
            if constexpr (PG == kAny)
                p = base(kv.k, __shfl(u.id[0], ka + 4 * j, 64), 0) + (unsigned)(((key0 + ka + 4 * j) & pm) * D);
#pragma unroll
            for (int c = 0; c < NC; c++) {
                const int d = 32 * c + 8 * g4;
                kf[j][c] = *reinterpret_cast<const u4 *>(p + (PG == kAny ? (d < D ? d : 0) : 4 * j * D + 32 * c));
            }
        }
    };
    // Values are read once and not kept in the caches (the keys are, whose
    // lines two loads share): 301 to 277 us on a 1.6 GB cache.
    const auto load_v = [&](int key0, const Ids &u) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            // the key's part that the lane decides and the load's own
            const int kl = row_key(vrow), ki = row_key(i * RPI);
            const uint16_t *p;
            if constexpr (PG == kOne)
                p = base(kv.v, u.id[0], key0) + ki * D + (unsigned)(kl * D + vch);
            else if constexpr (PG == kTwo)
                p = base(kv.v, u.id[ki >> 4], 0) + (ki & 15) * D + (unsigned)(kl * D + vch);
            else
                p = base(kv.v, __shfl(u.id[0], kl + ki, 64), 0) + (unsigned)(((key0 + kl + ki) & pm) * D + vch);
            vf[i] = __builtin_nontemporal_load(reinterpret_cast<const u4 *>(p));
        }
    };

    Ids cur{}, nxt{};          // ids of the tile in the registers, and of the next
    if (t_begin < t_end) {
        if constexpr (PG == kAny) {
            cur = lane_ids(t_begin);
            nxt = lane_ids(min(t_begin + kWaves, t_end - 1));
        } else {
            fill_ids(t_begin);
            cur = uniform_ids(t_begin);
        }
        load_k(tile_key<BN>(kt, t_begin), cur);
        load_v(tile_key<BN>(kt, t_begin), cur);
    }
    for (int t = t_begin; t < t_end; t += kWaves) {
        const int key0 = tile_key<BN>(kt, t);
        const int tn = t + kWaves < t_end ? t + kWaves : t; // the next tile, or this one again
        const int key_n = tile_key<BN>(kt, tn);
        Ids nn{}; // kAny: the ids after next, ahead of the loads they must not wait for
        if constexpr (PG == kAny) {
            nn = lane_ids(min(t + 2 * kWaves, t_end - 1));
        } else {
            if ((tn - ids_at) / kWaves >= 64 / HALVES) {
                fill_ids(tn);
                // waited for here, or the compiler waits for every load of
                // the loop wherever it reads an id
                __builtin_amdgcn_s_waitcnt(kWaitVmcnt0);
            }
            nxt = uniform_ids(tn);
        }

        // scores: register v of s[n][j] is key key0 + 8 (l / 16) + 4 j + v
        f32x4 s[NR][2];
        if (PG == kAny && D != DP) { // elements past D in the last K steps
#pragma unroll
            for (int c = 0; c < NC; c++)
                if (32 * c + 8 * g4 >= D)
                    kf[0][c] = kf[1][c] = (u4){0, 0, 0, 0};
        }
#pragma unroll
        for (int n = 0; n < NR; n++)
#pragma unroll
            for (int j = 0; j < 2; j++)
                s[n][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < NC; c++)
#pragma unroll
            for (int n = 0; n < NR; n++)
#pragma unroll
                for (int j = 0; j < 2; j++)
                    s[n][j] = T::mma16(kf[j][c], qf[n][c], s[n][j]);
        load_k(key_n, nxt);

        // a tile that some row sees only in part, or whose page ids are not
        // all good (in the small-page case every tile is checked for that)
        bool page_bad = !usable(cur.id[0]);
        if constexpr (PG == kTwo)
            page_bad |= !usable(cur.id[1]);
        if constexpr (PG == kAny)
            page_bad = __ballot(page_bad) != 0;
        const auto page_good = [&](int kk) { // kk < 32: key of the tile
            if constexpr (PG == kOne)
                return usable(cur.id[0]);
            else if constexpr (PG == kTwo)
                return kk < 16 ? usable(cur.id[0]) : usable(cur.id[1]);
            else
                return usable(__shfl(cur.id[0], kk, 64));
        };
        const int sinks = SHARED ? 0 : a.sinks;
        const bool edge = (key0 + BN - 1 > p_lo) | (key0 + BN > kt.hi) | ((key0 <= p_hi - window) & (key0 + BN > sinks)) |
                          (SHARED & (key0 < kt.lo)) | page_bad;
        if (edge) { // no branches inside: the compiler's waits for the loads in flight would cover all of them
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int v = 0; v < 4; v++) {
                    const int kk = 8 * g4 + 4 * j + v, key = key0 + kk;
                    const bool good = page_good(kk) & (key < kt.hi) & (!SHARED | (key >= kt.lo));
#pragma unroll
                    for (int n = 0; n < NR; n++) {
                        const bool seen = good & (key <= pos[n]) & ((key > pos[n] - window) | (key < sinks));
                        s[n][j][v] = seen ? s[n][j][v] : -INFINITY;
                    }
                }
            // values of keys that no row sees may be anything: zero
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int kk = row_key(i * RPI + vrow), key = key0 + kk;
                const bool any = page_good(kk) & (key < kt.hi) & ((key >= kt.lo) | (key < kt.sk));
                const uint32_t keep = any ? ~0u : 0u;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    vf[i][e] &= keep;
            }
        }

        u4 pt[NR][TERMS];
#pragma unroll
        for (int n = 0; n < NR; n++) {
            float top = fmaxf(fmaxf(fmaxf(s[n][0][0], s[n][0][1]), fmaxf(s[n][0][2], s[n][0][3])),
                              fmaxf(fmaxf(s[n][1][0], s[n][1][1]), fmaxf(s[n][1][2], s[n][1][3])));
            top = max_groups(top);
            // weights may grow to 2^LAG before the sums are rescaled
            if (__any(a.c * (top - m[n]) > T::LAG)) {
                // nothing seen yet: the sums are zero, and so is the factor
                const float mn = fmaxf(m[n], top), f = m[n] == -INFINITY ? 0.f : fast_exp2(a.c * (m[n] - mn));
                l[n] *= f;
#pragma unroll
                for (int i = 0; i < NV; i++)
                    acc[n][i] *= f;
                m[n] = mn;
                far[n] = __any((mn != -INFINITY) & (a.c * fabsf(mn) > kFar));
            }
            float off = m[n] == -INFINITY ? 0.f : T::BIAS - a.c * m[n];
            if (far[n]) {
                const float sub = m[n] == -INFINITY ? 0.f : m[n];
                off = T::BIAS;
#pragma unroll
                for (int i = 0; i < 8; i++)
                    s[n][i >> 2][i & 3] -= sub;
            }
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                p[i] = fast_exp2(fmaf(a.c, s[n][i >> 2][i & 3], off));
                l[n] += p[i];
            }
            split_terms<T, TERMS>(p, pt[n]);
        }

        // V through the wave's LDS piece: its previous reads are done (in
        // order within a wave), then this tile's rows, then the transposed
        // reads
#pragma unroll
        for (int i = 0; i < NV; i++)
            *reinterpret_cast<u4 *>(vbuf + (i * RPI + vrow) * VP + 16 * (lane % CH)) = vf[i];
        load_v(key_n, nxt);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const char *vr = vbuf + (4 * g4 + (r16 >> 2)) * VP + 8 * (r16 & 3);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const u2 lo = lds_read_tr(vr + 32 * i), hi = lds_read_tr(vr + 16 * VP + 32 * i);
            const u4 vt = {lo.x, lo.y, hi.x, hi.y}; // element 16 i + l % 16 of keys 8 (l / 16) .. + 7
#pragma unroll
            for (int n = 0; n < NR; n++)
#pragma unroll
                for (int k = 0; k < TERMS; k++)
                    acc[n][i] = T::mma16(vt, pt[n][k], acc[n][i]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        cur = nxt;
        if constexpr (PG == kAny)
            nxt = nn;
    }

    // the waves' sums joined in wave order
#pragma unroll
    for (int n = 0; n < NR; n++) {
        l[n] += __shfl_xor(l[n], 16, 64);
        l[n] += __shfl_xor(l[n], 32, 64);
        if (g4 == 0) {
            s_m[wave][16 * n + r16] = m[n];
            s_l[wave][16 * n + r16] = l[n];
        }
    }
    const size_t slot = ((size_t)unit * a.S + split) * (NR * 16);
    const bool joined = active == 1 && alone;
    float *o_lds = reinterpret_cast<float *>(smem);
    constexpr int OP = DP + 4;
#pragma unroll
    for (int n = 0; n < NR; n++) {
        __syncthreads();
        float top = s_m[0][16 * n + r16];
#pragma unroll
        for (int w = 1; w < kWaves; w++)
            top = fmaxf(top, s_m[w][16 * n + r16]);
        const float f = m[n] == -INFINITY ? 0.f : fast_exp2(a.c * (m[n] - top));
#pragma unroll
        for (int i = 0; i < NV; i++)
            *reinterpret_cast<f32x4 *>(o_lds + (wave * 16 + r16) * OP + 16 * i + 4 * g4) = acc[n][i] * f;
        __syncthreads();
        // 16 threads per row, four elements each at a time
        const int r = threadIdx.x >> 4, row = 16 * n + r;
        float rm = s_m[0][16 * n + r], rl = 0.f;
#pragma unroll
        for (int w = 1; w < kWaves; w++)
            rm = fmaxf(rm, s_m[w][16 * n + r]);
#pragma unroll
        for (int w = 0; w < kWaves; w++)
            rl += s_m[w][16 * n + r] == -INFINITY ? 0.f : s_l[w][16 * n + r] * fast_exp2(a.c * (s_m[w][16 * n + r] - rm));
        if (row >= nrows)
            continue;
        const float inv = rl > 0.f ? 1.0f / rl : 0.f; // a row that sees nothing is zero
        const int tok = kv.div_g(row);
        const size_t at = ((size_t)(sq.t0 + tok) * kv.Hq + hk * kv.G + kv.div_g.rem(row, tok)) * D;
        for (int d = 4 * (threadIdx.x & 15); d < D; d += 64) {
            f32x4 o = *reinterpret_cast<const f32x4 *>(o_lds + r * OP + d);
#pragma unroll
            for (int w = 1; w < kWaves; w++)
                o += *reinterpret_cast<const f32x4 *>(o_lds + (w * 16 + r) * OP + d);
            if (joined) {
                o *= inv;
                if (a.out_f32)
                    *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + at + d) = o;
                else
                    *reinterpret_cast<u2 *>(static_cast<uint16_t *>(a.out) + at + d) = (u2){T::pack(o[0], o[1]), T::pack(o[2], o[3])};
            } else {
                *reinterpret_cast<f32x4 *>(a.part + (slot + row) * DP + d) = o;
            }
        }
        if (!joined && (threadIdx.x & 15) == 0)
            *reinterpret_cast<f2 *>(a.stat + (slot + row) * 2) = (f2){rm, rl};
    }
}

} // namespace decode
} // namespace dev
} // namespace rfx
