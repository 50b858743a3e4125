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
#include <cmath>

#include "rfx_kv.h"

using namespace rfx;
using namespace rfx::dev;

namespace {

constexpr int kMaxSplits = 64; // one lane of the join each

// Adds the n partials of one row, `stride` elements apart, by their factors
// (lane i: the i-th's), eight loads at a time.
template <class V>
__device__ __forceinline__ void add_partials(V &sum, const float *p, size_t stride, int n, float factor)
{
    for (int s = 0; s < n; s += 8) {
        V x[8];
#pragma unroll
        for (int i = 0; i < 8; i++)
            x[i] = *reinterpret_cast<const V *>(p + (size_t)min(s + i, n - 1) * stride);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(factor), min(s + i, 63)));
            if (s + i < n)
                sum += x[i] * w;
        }
    }
}

// One wave per row of a sequence's new tokens.
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
    const Seq sq = load_seq(kv, seq);
    if (row >= sq.nq * kv.G)
        return;
    Group gr;
    const int gi = prefix_of(kv, args.pre, seq, sq, gr);
    int per, n_own, n_group = 0;
    split_tiles(o, range_tiles(o.bn, gr.len, min(sq.kv, sq.p0 + sq.nq)).n, per, n_own);
    if (!gr.len && n_own == 1)
        return; // done already
    const int tok = kv.div_g(row), head = kv.div_g.rem(row, tok);
    const size_t own = (size_t)unit * o.S * o.rows + row;
    size_t pre = 0;
    if (gr.len) {
        split_tiles(g, range_tiles(g.bn, 0, gr.len).n, per, n_group);
        const int r = (sq.t0 + tok - gr.t0) * kv.G + head, shift = __builtin_ctz(g.rows); // rows: a power of two
        pre = ((size_t)(gi * g.row_blocks + (r >> shift)) * kv.Hk + hk) * g.S * g.rows + (r & (g.rows - 1));
    }
    // what no split wrote may be anything and is selected away
    const f2 none = {-INFINITY, 0.f};
    const f2 so = lane < n_own ? *reinterpret_cast<const f2 *>(o.stat + (own + (size_t)lane * o.rows) * 2) : none;
    const f2 sg = lane < n_group ? *reinterpret_cast<const f2 *>(g.stat + (pre + (size_t)lane * g.rows) * 2) : none;
    float m = fmaxf(so.x, sg.x);
#pragma unroll
    for (int i = 32; i > 0; i >>= 1)
        m = fmaxf(m, __shfl_xor(m, i, 64));
    const float fo = so.x == -INFINITY ? 0.f : fast_exp2(o.c * (so.x - m)), fg = sg.x == -INFINITY ? 0.f : fast_exp2(o.c * (sg.x - m));
    float l = so.y * fo + sg.y * fg;
#pragma unroll
    for (int i = 32; i > 0; i >>= 1)
        l += __shfl_xor(l, i, 64);
    fp sum;
#pragma unroll
    for (int i = 0; i < PER; i++)
        sum[i] = 0.f;
    add_partials(sum, g.part + pre * DP + PER * lane, (size_t)g.rows * DP, n_group, fg);
    add_partials(sum, o.part + own * DP + PER * lane, (size_t)o.rows * DP, n_own, fo);
    const int d = PER * lane;
    if (d >= kv.D)
        return;
    const float inv = l > 0.f ? 1.0f / l : 0.f; // a row that sees nothing is zero
    const size_t at = ((size_t)(sq.t0 + tok) * kv.Hq + hk * kv.G + head) * kv.D + d;
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
    bool tall;       // the prefix on the prefill kernel
    Part group, own;
};

void sizes(Part &p, int dp)
{
    p.part = align256((size_t)p.units * p.S * p.rows * dp * sizeof(float));
    p.stat = align256((size_t)p.units * p.S * p.rows * 2 * sizeof(float));
}

int splits(int64_t units, int64_t tiles, const Part &p)
{
    const int64_t want = 512 / (units < 512 ? units : 512), most = tiles <= p.one_tiles ? 1 : ceil_div(tiles, p.min_tiles);
    const int64_t s = want < most ? want : most;
    return (int)(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
}

// Sequences of more rows than the decode kernel takes are left to rfx_attn,
// whose prefill tiles already have 128 rows of one sequence per key. A group
// of up to kTallRows rows stays on the decode kernel, in the launch of the
// sequences' own keys; more go to the prefill kernel.
constexpr int kTallRows = 64;

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
    p.group.S = splits(p.group.units, ceil_div(P->max_len < room ? P->max_len : room, p.group.bn), p.group);
    sizes(p.group, dp);
    sizes(p.own, dp);
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
    return p.shared ? p.group.part + p.group.stat + p.own.part + p.own.stat : rfx_attn_workspace_bytes(C, B, n_heads);
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
    const size_t need = p.group.part + p.group.stat + p.own.part + p.own.stat;
    if (!ws || ws_bytes < need)
        return fail(RFX_E_WORKSPACE, "rfx_attn_shared: workspace %zu < %zu bytes", ws ? ws_bytes : (size_t)0, need);
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
    a.group_blocks = (int)(p.group.units * p.group.S);
    const hipStream_t hs = (hipStream_t)stream;
    if (p.tall) {
        if ((st = attn_prefill_launch(a, C->type, hs)))
            return st;
        a.group_blocks = 0;
    }
    if ((st = attn_decode_launch(a, C->type, p.own.rows / 16, hs)))
        return st;
    return C->type == RFX_BF16 ? join<BF16>(a, hs) : join<F16>(a, hs);
}

} // extern "C"
