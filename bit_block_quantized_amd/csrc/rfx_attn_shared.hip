// Attention of sequences that share a prefix: the keys and values of the
// prefix are read once for all new tokens of a group of sequences, those
// behind it once for each sequence's.
//
// Softmax over both parts: each leaves its rows' maximum m, sum l and
// unnormalised result o (per split of its keys), and
//   out = sum_i e^(m_i - M) o_i / sum_i e^(m_i - M) l_i,   M = max m_i,
// added in a fixed order. The parts are rfx_attn's kernels: to the prefix a
// group is a sequence whose new tokens, which are neighbours, all come after
// its keys, so with 64 sequences of four heads per kv head a key tile serves
// 256 rows instead of four.
//
// Two launches, the parts and the join (rfx_kv.h: AttnArgs, SharedArgs).
// Bound by latency where prefixes are short, by the own keys' bytes and the
// matrix pipe where there is much: 32 heads of 128, four sequences behind 500
// keys (8 kv heads) 10 us; two groups of twelve with up to four new tokens each
// behind 3001 and 1606 keys (4) 23; 64 sequences of up to 700 keys behind 16384
// (8) 69 (60 and the join's 9; the bytes take 23, the prefix with hardly an own
// key 58 with its join, the own keys with hardly a prefix 27).
#include <algorithm>
#include <cmath>

#include "rfx_attn_decode.h"
#include "rfx_attn_prefill.h"

using namespace rfx;
using namespace rfx::dev;

namespace {

constexpr int kMaxSplits = 64; // one lane of the join each

// The prefix of many rows on the prefill kernel's tiles and the sequences' own
// keys on the decode kernel's, in one launch: the one is bound by the matrix
// pipe, the other by latency and memory, and a compute unit has both at a time
// (64 sequences of up to 700 keys behind 16384, weights of one term: 54 us with
// the join, 72 with the two one after the other).
// Weights of the prefix are carried as all of their terms, whatever the result's
// type, as those of a sequence's own keys and of small groups are: what a
// request gets does not depend on how many are in its group.
template <class T, int DP, int NR, decode::Pages PG>
__global__ __launch_bounds__(256, prefill::waves_per_simd(DP, T::TERMS) > 2 ? 2 : prefill::waves_per_simd(DP, T::TERMS))
void shared_both_kernel(SharedArgs args)
{
    constexpr int A = 2 * prefill::Tile<DP>::buf, B = decode::lds_bytes<DP>();
    __shared__ __align__(16) char smem[A > B ? A : B];
    // the smaller arrays of either
    constexpr int kBad = 3 * 2 * 4, kSmall = std::max(kBad + prefill::kIds * 4, 2 * decode::kWaves * NR * 16 * 4);
    __shared__ __align__(16) char small[kSmall];
    const int block = blockIdx.x;
    if (block < args.group_blocks) {
        prefill::attention<T, DP, T::TERMS>(args, block, smem, reinterpret_cast<unsigned (*)[2]>(small), reinterpret_cast<int *>(small + kBad));
    } else {
        float(*m)[NR * 16] = reinterpret_cast<float(*)[NR * 16]>(small);
        decode::attention<T, DP, NR, PG>(args, block, smem, m, m + decode::kWaves);
    }
}

template <class T, int DP, int NR>
void both_pages(const SharedArgs &a, hipStream_t st)
{
    const KvArgs &kv = a.own.kv;
    const dim3 grid(a.group_blocks + (unsigned)kv.n_seq * kv.Hk * a.own.S), block(256);
    if (kv.D != DP || kv.page_shift < 4)
        hipLaunchKernelGGL((shared_both_kernel<T, DP, NR, decode::kAny>), grid, block, 0, st, a);
    else if (kv.page_shift == 4)
        hipLaunchKernelGGL((shared_both_kernel<T, DP, NR, decode::kTwo>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((shared_both_kernel<T, DP, NR, decode::kOne>), grid, block, 0, st, a);
}

template <class T>
int both(const SharedArgs &a, hipStream_t st)
{
    const int D = a.own.kv.D;
    const bool one = a.own.rows == 16;
    if (D > 128)
        both_pages<T, 256, 1>(a, st);
    else if (D > 64)
        one ? both_pages<T, 128, 1>(a, st) : both_pages<T, 128, 2>(a, st);
    else
        one ? both_pages<T, 64, 1>(a, st) : both_pages<T, 64, 2>(a, st);
    return hip_status("attn shared launch");
}

// The first eight partials of a row, `stride` elements apart, past the last
// (of most) the last again.
template <class V>
__device__ __forceinline__ void first_partials(V (&x)[8], const float *p, size_t stride, int most)
{
#pragma unroll
    for (int i = 0; i < 8; i++)
        x[i] = *reinterpret_cast<const V *>(p + (size_t)min(i, most - 1) * stride);
}

// Adds the n partials of a row by their factors (lane i: the i-th's); x: the
// first of them.
template <class V>
__device__ __forceinline__ void add_partials(V &sum, V (&x)[8], const float *p, size_t stride, int n, float factor)
{
    for (int s = 0; s < n; s += 8) {
        V y[8];
#pragma unroll
        for (int i = 0; i < 8; i++)
            y[i] = x[i];
        if (s + 8 < n) // the next ones' loads
#pragma unroll
            for (int i = 0; i < 8; i++)
                x[i] = *reinterpret_cast<const V *>(p + (size_t)min(s + 8 + i, n - 1) * stride);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(factor), min(s + i, 63)));
            if (s + i < n)
                sum += y[i] * w;
        }
    }
}

// One wave per row of a sequence's new tokens. The sequence's own partials are
// read beside the unit's record, which says where the prefix's are.
template <class T, int DP>
__global__ __launch_bounds__(256) void shared_join_kernel(SharedArgs args)
{
    constexpr int PER = DP / 64; // elements per lane
    typedef float fp __attribute__((ext_vector_type(PER)));
    const AttnArgs &o = args.own, &g = args.group;
    const KvArgs &kv = o.kv;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int quads = o.rows / 4, unit = blockIdx.x >> __builtin_ctz(quads), row = (blockIdx.x & (quads - 1)) * 4 + wave;
    const int seq = kv.div_hk(unit), hk = kv.div_hk.rem(unit, seq);
    const size_t own = (size_t)unit * o.S * o.rows + row, so = (size_t)o.rows * DP, sg = (size_t)g.rows * DP;
    const float *po = o.part + own * DP + PER * lane;
    const f2 any = *reinterpret_cast<const f2 *>(o.stat + (own + (size_t)min(lane, o.S - 1) * o.rows) * 2);
    fp xo[8], xg[8];
    xo[0] = *reinterpret_cast<const fp *>(po);
    const SharedArgs::Unit u = args.units[unit];
    if (row >= u.nq * kv.G || (!u.n_group && u.n_own == 1)) // none, or done already
        return;
    const int r = u.row0 + row, shift = __builtin_ctz(g.rows); // rows: a power of two
    const size_t pre = u.n_group ? ((size_t)(u.g * g.row_blocks + (r >> shift)) * kv.Hk + hk) * g.S * g.rows + (r & (g.rows - 1)) : 0;
    const float *pg = g.part + pre * DP + PER * lane;
    // what no split wrote may be anything and is selected away
    const f2 none = {-INFINITY, 0.f};
    const f2 stg = lane < u.n_group ? *reinterpret_cast<const f2 *>(g.stat + (pre + (size_t)lane * g.rows) * 2) : none;
    if (u.n_group)
        first_partials(xg, pg, sg, u.n_group);
    if (u.n_own > 1)
        first_partials(xo, po, so, u.n_own);
    const f2 sto = lane < u.n_own ? any : none;
    float m = fmaxf(sto.x, stg.x);
#pragma unroll
    for (int i = 32; i > 0; i >>= 1)
        m = fmaxf(m, __shfl_xor(m, i, 64));
    const float fo = sto.x == -INFINITY ? 0.f : fast_exp2(o.c * (sto.x - m)), fg = stg.x == -INFINITY ? 0.f : fast_exp2(o.c * (stg.x - m));
    float l = sto.y * fo + stg.y * fg;
#pragma unroll
    for (int i = 32; i > 0; i >>= 1)
        l += __shfl_xor(l, i, 64);
    fp sum;
#pragma unroll
    for (int i = 0; i < PER; i++)
        sum[i] = 0.f;
    if (u.n_group)
        add_partials(sum, xg, pg, sg, u.n_group, fg);
    if (u.n_own > 1)
        add_partials(sum, xo, po, so, u.n_own, fo);
    else
        sum += xo[0] * __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(fo)));
    const int d = PER * lane;
    if (d >= kv.D)
        return;
    const float inv = l > 0.f ? 1.0f / l : 0.f; // a row that sees nothing is zero
    const int tok = kv.div_g(row);
    const size_t at = ((size_t)(u.t0 + tok) * kv.Hq + hk * kv.G + kv.div_g.rem(row, tok)) * kv.D + d;
    if (o.out_f32) {
        *reinterpret_cast<fp *>(static_cast<float *>(o.out) + at) = sum * inv;
    } else {
        uint16_t *p = static_cast<uint16_t *>(o.out) + at;
        if constexpr (PER == 1)
            *p = (uint16_t)T::pack(sum[0] * inv, 0.f);
        else
#pragma unroll
            for (int i = 0; i < PER; i += 2)
                *reinterpret_cast<uint32_t *>(p + i) = T::pack(sum[i] * inv, sum[i + 1] * inv);
    }
}

template <class T>
int join(const SharedArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)a.own.kv.n_seq * a.own.kv.Hk * (a.own.rows / 4)), block(256);
    if (a.own.kv.D <= 64)
        hipLaunchKernelGGL((shared_join_kernel<T, 64>), grid, block, 0, st, a);
    else if (a.own.kv.D <= 128)
        hipLaunchKernelGGL((shared_join_kernel<T, 128>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((shared_join_kernel<T, 256>), grid, block, 0, st, a);
    return hip_status("attn shared join launch");
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

struct Part {
    int rows, row_blocks, bn, S, min_tiles, one_tiles, cap_shift;
    int64_t units;
    size_t part, stat;
};

struct Plan {
    bool shared;     // else rfx_attn
    bool tall;       // the prefix on the prefill kernel's tiles
    Part group, own;
    size_t units, bytes;
};

void sizes(Part &p, int dp)
{
    p.part = align256((size_t)p.units * p.S * p.rows * dp * sizeof(float));
    p.stat = align256((size_t)p.units * p.S * p.rows * 2 * sizeof(float));
}

int splits(int64_t units, int64_t tiles, const Part &p, int places = 512)
{
    const int64_t want = places / (units < places ? units : places), most = tiles <= p.one_tiles ? 1 : ceil_div(tiles, p.min_tiles);
    const int64_t s = want < most ? want : most;
    return (int)(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
}

// Sequences of more rows than the decode kernel takes are left to rfx_attn,
// whose prefill tiles already have 128 rows of one sequence per key. The
// prefix of a group of few rows is the decode kernel's, which reads it once
// per 32 (16) rows, mostly from L2: 128 rows of 3001 keys of 8 kv heads 22.3 us,
// on the prefill kernel's tiles 24.6, of 8000 27.6 and 30.2. With more rows it is
// the other way round: 256 rows of 500 keys 27.3 and 21.8, of 8000 41.5 and 40.0,
// 384 of 8000 65 and 51.
constexpr int64_t kTallRows = 128;

Plan plan(const rfx_kv_cache *C, const rfx_kv_batch *B, const rfx_kv_prefix *P, int n_heads)
{
    Plan p{};
    const int G = n_heads / C->n_kv_heads, dp = C->head_dim <= 64 ? 64 : C->head_dim <= 128 ? 128 : 256;
    const int64_t rows = (int64_t)B->max_q * G, all = (int64_t)P->max_tokens * G;
    const int most = dp == 256 ? 16 : 32;
    p.shared = rows <= most;
    if (!p.shared)
        return p;
    p.tall = all > kTallRows;
    p.own.rows = rows > 16 || (!p.tall && all > 16 && most > 16) ? 32 : 16;
    p.own.row_blocks = 1;
    p.own.bn = 32;
    p.own.min_tiles = 4;
    p.own.one_tiles = 16;
    p.own.cap_shift = p.own.rows == 16 ? 5 : 3;
    p.own.units = (int64_t)B->n_seq * C->n_kv_heads;
    const int64_t room = (int64_t)B->table_stride * C->page_size;
    p.own.S = splits(p.own.units, ceil_div(room, 32), p.own);
    p.group.rows = p.tall ? 128 : p.own.rows;
    p.group.row_blocks = (int)ceil_div(all, p.group.rows);
    p.group.bn = p.tall && dp < 256 ? 64 : 32;
    p.group.min_tiles = p.tall ? 2 : 4;
    p.group.one_tiles = p.tall ? 4 : 8;
    p.group.cap_shift = 5;
    p.group.units = (int64_t)P->n_groups * C->n_kv_heads * p.group.row_blocks;
    const int64_t tiles = ceil_div(P->max_len < room ? P->max_len : room, p.group.bn);
    p.group.S = splits(p.group.units, tiles, p.group, p.tall ? 384 : 256);
    // Partials of more splits cost the join more than they save, unless the
    // chip is not full without them (64 sequences behind 16384 keys, 256 rows of
    // 8 kv heads: 16 splits 69 us, 32 76; 80 behind 16000, 320 rows of 2: 37, with
    // 16 splits 52), and past eight a split wants four tiles (256 rows, 2000 keys:
    // 39.6 us, else 44.4). Beside the own keys' workgroups 384 are enough (48
    // sequences of up to four tokens behind 16000: 85, with 512 90, with 256 96).
    const int64_t full = 256 / (p.group.units < 256 ? p.group.units : 256);
    const int64_t cap = p.tall ? std::min(std::max<int64_t>(full, 16), std::max<int64_t>(8, ceil_div(tiles, 4))) : 32;
    p.group.S = (int)std::min<int64_t>(p.group.S, cap);
    sizes(p.group, dp);
    sizes(p.own, dp);
    p.units = align256((size_t)p.own.units * sizeof(SharedArgs::Unit));
    p.bytes = p.group.part + p.group.stat + p.own.part + p.own.stat + p.units;
    return p;
}

void fill(AttnArgs &a, const Part &p, char *&ws)
{
    a.S = p.S;
    a.row_blocks = p.row_blocks;
    a.rows = p.rows;
    a.bn = p.bn;
    a.min_tiles = p.min_tiles;
    a.one_tiles = p.one_tiles;
    a.cap_shift = p.cap_shift;
    a.div_s = Div(p.S);
    a.div_rb = Div(p.row_blocks);
    a.div_units = Div((uint32_t)p.units);
    a.part = reinterpret_cast<float *>(ws);
    a.stat = reinterpret_cast<float *>(ws + p.part);
    ws += p.part + p.stat;
}

bool prefix_ok(const rfx_kv_prefix *P)
{
    return P->n_groups >= 1 && P->n_groups <= kMaxTokens && P->max_tokens >= 1 && P->max_tokens <= kMaxTokens && P->max_len >= 1;
}

} // namespace

extern "C" {

size_t rfx_attn_shared_workspace_bytes(const rfx_kv_cache *C, const rfx_kv_batch *B, const rfx_kv_prefix *P, int n_heads)
{
    if (!C || !B || !P || C->n_kv_heads < 1 || n_heads < 1 || n_heads % C->n_kv_heads || C->head_dim < 8 ||
        C->head_dim > kMaxHeadDim || C->page_size < 1 || B->n_seq < 1 || B->max_q < 1 || B->max_q > kMaxTokens ||
        B->table_stride < 1 || !prefix_ok(P))
        return 0;
    const Plan p = plan(C, B, P, n_heads);
    return p.shared ? p.bytes : rfx_attn_workspace_bytes(C, B, n_heads);
}

int rfx_attn_shared(const void *q, const rfx_kv_cache *C, const rfx_kv_batch *B, const rfx_kv_prefix *P, int n_heads,
                    float scale, void *out, int out_type, void *ws, size_t ws_bytes, void *stream)
{
    int st = check_kv(C, B, n_heads, "rfx_attn_shared");
    if (st)
        return st;
    if (!P)
        return fail(RFX_E_INVAL, "rfx_attn_shared: prefix descriptor is NULL");
    if (!prefix_ok(P))
        return fail(RFX_E_INVAL, "rfx_attn_shared: n_groups=%d max_tokens=%d max_len=%d", P->n_groups, P->max_tokens, P->max_len);
    if ((st = check_ptr(P->seq_off, 4, "seq_off")) || (st = check_ptr(P->len, 4, "len")))
        return st;
    const Plan p = plan(C, B, P, n_heads);
    if (!p.shared)
        return rfx_attn(q, C, B, n_heads, scale, 0, 0, out, out_type, ws, ws_bytes, stream);
    if (!(scale > 0.0f) || scale > 0x1p127f)
        return fail(RFX_E_INVAL, "rfx_attn_shared: scale=%g (positive, at most 2^127)", (double)scale);
    if (out_type != RFX_F32 && out_type != C->type)
        return fail(RFX_E_INVAL, "rfx_attn_shared: out_type=%d (RFX_F32 or the cache's type)", out_type);
    if ((st = check_ptr(q, 16, "q")) || (st = check_ptr(out, 16, "out")))
        return st;
    // workgroups of each launch, the join's among them
    if (p.group.units * p.group.S + p.own.units * p.own.S >= (int64_t)kMaxTokens || p.own.units * (p.own.rows / 4) >= (int64_t)kMaxTokens)
        return fail(RFX_E_INVAL, "rfx_attn_shared: %d sequences in %d groups of up to %d new tokens need more than %d workgroups",
                    B->n_seq, P->n_groups, P->max_tokens, kMaxTokens);
    if (!ws || ws_bytes < p.bytes)
        return fail(RFX_E_WORKSPACE, "rfx_attn_shared: workspace %zu < %zu bytes", ws ? ws_bytes : (size_t)0, p.bytes);
    if ((st = check_ptr(ws, 256, "ws")))
        return st;
    if (B->n_tokens == 0)
        return RFX_OK;
    SharedArgs a{};
    a.pre = {P->seq_off, P->len, P->n_groups, P->max_tokens};
    a.own.kv = kv_args(C, B, n_heads);
    a.own.q = static_cast<const uint16_t *>(q);
    a.own.out = out;
    a.own.out_f32 = out_type == RFX_F32;
    a.own.c = scale * 1.4426950408889634f; // finite
    a.group = a.own;
    char *w = static_cast<char *>(ws);
    fill(a.group, p.group, w);
    fill(a.own, p.own, w);
    a.units = reinterpret_cast<SharedArgs::Unit *>(w);
    a.group_blocks = (int)(p.group.units * p.group.S);
    const hipStream_t hs = (hipStream_t)stream;
    if (p.tall)
        st = C->type == RFX_BF16 ? both<BF16>(a, hs) : both<F16>(a, hs);
    else
        st = attn_decode_launch(a, C->type, p.own.rows / 16, hs);
    if (st)
        return st;
    return C->type == RFX_BF16 ? join<BF16>(a, hs) : join<F16>(a, hs);
}

} // extern "C"
