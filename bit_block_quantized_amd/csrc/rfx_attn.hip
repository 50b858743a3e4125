// Host side of the paged-cache entry points (argument checks, the choice of
// kernel and split, workspace sizes), and the launch that joins split keys.
#include <cmath>

#include "rfx_kv.h"

namespace rfx {

int check_kv(const rfx_kv_cache *C, const rfx_kv_batch *B, int n_heads, const char *who)
{
    if (!C || !B)
        return fail(RFX_E_INVAL, "%s: cache or batch descriptor is NULL", who);
    if (C->type != RFX_F16 && C->type != RFX_BF16)
        return fail(RFX_E_INVAL, "%s: cache type %d (RFX_F16 or RFX_BF16)", who, C->type);
    if (C->head_dim < 8 || C->head_dim > kMaxHeadDim || C->head_dim % 8)
        return fail(RFX_E_INVAL, "%s: head_dim=%d (a multiple of 8 from 8 to %d)", who, C->head_dim, kMaxHeadDim);
    if (C->n_kv_heads < 1 || n_heads < 1 || n_heads > kMaxHeads || n_heads % C->n_kv_heads)
        return fail(RFX_E_INVAL, "%s: %d heads over %d kv heads (at most %d, a multiple)", who, n_heads, C->n_kv_heads,
                    kMaxHeads);
    if (C->page_size < 1 || C->page_size > kMaxPage || (C->page_size & (C->page_size - 1)))
        return fail(RFX_E_INVAL, "%s: page_size=%d (a power of two from 1 to %d)", who, C->page_size, kMaxPage);
    if (C->n_pages < 1)
        return fail(RFX_E_INVAL, "%s: n_pages=%d", who, C->n_pages);
    if (B->n_seq < 1 || B->n_tokens < 0 || B->max_q < 1 || B->table_stride < 1)
        return fail(RFX_E_INVAL, "%s: n_seq=%d n_tokens=%d max_q=%d table_stride=%d", who, B->n_seq, B->n_tokens,
                    B->max_q, B->table_stride);
    if ((int64_t)B->table_stride * C->page_size > (int64_t)1 << 30)
        return fail(RFX_E_INVAL, "%s: table_stride=%d pages of %d tokens (at most 2^30 tokens)", who, B->table_stride,
                    C->page_size);
    if (B->n_tokens > kMaxTokens || B->max_q > kMaxTokens)
        return fail(RFX_E_INVAL, "%s: n_tokens=%d max_q=%d (at most %d)", who, B->n_tokens, B->max_q, kMaxTokens);
    int st = check_ptr(C->k, 16, "cache k");
    if (!st)
        st = check_ptr(C->v, 16, "cache v");
    if (!st)
        st = check_ptr(B->q_off, 4, "q_off");
    if (!st)
        st = check_ptr(B->kv_len, 4, "kv_len");
    if (!st)
        st = check_ptr(B->page_table, 4, "page_table");
    return st;
}

namespace {

using namespace dev;

constexpr int kMaxSplits = 64; // one lane of the join each

// Joins the splits of one row per wave: lane s holds the factor of split s,
// exp2(c (m_s - max m)), and the partials are added in split order, so
// the result does not depend on timing. Reads S partials per row once;
// blocks that one split covered are done already.
template <class T, int DP>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a)
{
    constexpr int PER = DP / 64; // elements per lane
    typedef float fp __attribute__((ext_vector_type(PER)));
    const KvArgs &kv = a.kv;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int quads = a.rows / 4, unit = blockIdx.x >> __builtin_ctz(quads), r = (blockIdx.x & (quads - 1)) * 4 + wave;
    const int u = kv.div_hk(unit), hk = kv.div_hk.rem(unit, u), seq = a.div_rb(u), rb = a.div_rb.rem(u, seq);
    // The first partials and the statistics of all splits are read before it
    // is known how many there are, beside the lengths (one round trip to
    // memory where each waiting for the one before made three). What no split
    // wrote may be anything and is selected away, not multiplied.
    const size_t slot = (size_t)unit * a.S * a.rows + r;
    const float *p = a.part + slot * DP + PER * lane;
    const size_t stride = (size_t)a.rows * DP;
    const f2 any = *reinterpret_cast<const f2 *>(a.stat + (slot + (size_t)min(lane, a.S - 1) * a.rows) * 2);
    fp x[8];
#pragma unroll
    for (int i = 0; i < 8; i++)
        x[i] = *reinterpret_cast<const fp *>(p + min(i, a.S - 1) * stride);
    const Seq sq = load_seq(kv, seq);
    const int nrows = sq.nq * kv.G, row0 = rb * a.rows, row = row0 + r;
    const int row_end = min(nrows, row0 + a.rows);
    const KeyTiles kt = key_tiles(a.bn, sq.p0 + kv.div_g(row0), sq.p0 + kv.div_g(max(0, row_end - 1)), sq.kv, a.window, a.sinks);
    int per, active;
    split_tiles(a, kt.n, per, active);
    const f2 st = {lane < active ? any.x : -INFINITY, lane < active ? any.y : 0.f};
    float m = st.x;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor(m, o, 64));
    const float f = st.x == -INFINITY ? 0.f : fast_exp2(a.c * (st.x - m));
    float l = st.y * f;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        l += __shfl_xor(l, o, 64);
    fp sum;
#pragma unroll
    for (int i = 0; i < PER; i++)
        sum[i] = 0.f;
    for (int s = 0; s < active; s += 8) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), min(s + i, 63)));
            if (s + i < active)
                sum += x[i] * w;
        }
        // eight partials' loads at a time; past the last, the last again
        if (s + 8 < active)
#pragma unroll
            for (int i = 0; i < 8; i++)
                x[i] = *reinterpret_cast<const fp *>(p + min(s + 8 + i, active - 1) * stride);
    }
    if (row >= nrows || active == 1)
        return;
    const int d = PER * lane;
    if (d >= kv.D)
        return;
    const float inv = l > 0.f ? 1.0f / l : 0.f;
    const int tok = kv.div_g(row);
    const size_t at = ((size_t)(sq.t0 + tok) * kv.Hq + hk * kv.G + kv.div_g.rem(row, tok)) * kv.D + d;
    if (a.out_f32) {
        *reinterpret_cast<fp *>(static_cast<float *>(a.out) + at) = sum * inv;
    } else {
        uint16_t *o = static_cast<uint16_t *>(a.out) + at;
        if constexpr (PER == 1)
            *o = (uint16_t)T::pack(sum[0] * inv, 0.f);
        else
#pragma unroll
            for (int i = 0; i < PER; i += 2)
                *reinterpret_cast<uint32_t *>(o + i) = T::pack(sum[i] * inv, sum[i + 1] * inv);
    }
}

template <class T>
int join(const AttnArgs &a, int64_t units, hipStream_t st)
{
    const dim3 grid((unsigned)(units * (a.rows / 4)));
    if (a.kv.D <= 64)
        hipLaunchKernelGGL((attn_join_kernel<T, 64>), grid, dim3(256), 0, st, a);
    else if (a.kv.D <= 128)
        hipLaunchKernelGGL((attn_join_kernel<T, 128>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((attn_join_kernel<T, 256>), grid, dim3(256), 0, st, a);
    return hip_status("attn join launch");
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

struct Plan {
    bool decode;
    int row_tiles;   // decode: 16-row tiles per workgroup
    int row_blocks;
    int S, min_tiles, one_tiles;
    int rows, bn;    // rows of a block, keys of a tile
    int64_t units;   // (sequence, row block, kv head)
    size_t part, stat;
};

// The two-group prefill kernel (rows of 256, heads of 65 to 128 elements)
// wants two workgroups per compute unit in turn or long runs of key tiles:
// it starts and ends slower, alone on its compute unit. Measured in us, 32
// heads of 128 over 8, against the four-wave kernel: 8192 tokens (1024
// workgroups) 500 and 586, 4096 (512) 145 and 171, 1000 after 30000 (four
// splits of 121 tiles) 466 and 547; but 2048 (256) 90 and 69, 256 after
// 8000 (sixteen splits of 9 tiles) 62 and 57. Its list of page ids has to
// fit the LDS. The host knows the table's width, not the lengths, and a width
// far beyond them misleads it: 2048 tokens with a table for 131072 take this
// kernel, 89 us where the exact table takes 64; and with pages of 16 a table
// past 65536 tokens rules it out (8192 tokens 597 us, 515 with the exact one).
bool pair_rows(const rfx_kv_cache *C, const rfx_kv_batch *B, int64_t rows, int dp)
{
    const int64_t keys = (int64_t)B->table_stride * C->page_size;
    if (dp != 128 || ceil_div(keys, C->page_size < 64 ? C->page_size : 64) > kPairIds)
        return false;
    const int64_t units = (int64_t)B->n_seq * C->n_kv_heads * ceil_div(rows, kPairRows);
    return units >= 512 || ceil_div(keys, 64) / (512 / units) >= 64;
}

// The decode kernel serves up to 32 rows (new tokens x query heads of a kv
// head) in one pass over the keys, 16 with heads over 128 elements (its
// accumulators would not fit the registers); more rows go to the prefill
// kernel, whose matrix-core tiles have 32. Keys are split as far as needed
// for about two workgroups per compute unit, by the table's width: where it
// could hold enough to be split the join is launched, for short sequences too
// (one token, 400 keys: 8.1 us, 10.5 with a table for 131072).
Plan plan(const rfx_kv_cache *C, const rfx_kv_batch *B, int n_heads)
{
    Plan p{};
    const int64_t rows = (int64_t)B->max_q * (n_heads / C->n_kv_heads);
    const int dp = C->head_dim <= 64 ? 64 : C->head_dim <= 128 ? 128 : 256;
    p.decode = rows <= (dp == 256 ? 16 : 32);
    p.rows = p.decode ? (rows <= 16 ? 16 : 32) : pair_rows(C, B, rows, dp) ? kPairRows : 128;
    p.row_tiles = p.rows / 16;
    p.row_blocks = (int)((rows + p.rows - 1) / p.rows);
    p.bn = p.decode || dp == 256 ? 32 : 64;
    // measured in us, one sequence, 8 kv heads, 512 / 700 / 1537 keys: 16
    // tiles (of 32 keys) unsplit 8.9 and as two splits 10.0; 22 tiles 9.0 as
    // six splits and 11.3 unsplit; 49 tiles 9.8 as 13 splits, 10.6 as seven.
    // Prompt chunks of 300 new tokens: 5 tiles (of 64) 15.5 unsplit, 20.2 split.
    p.min_tiles = p.decode ? 4 : 2;
    // The join reads every row of every split: 256 new tokens after 200 (64
    // units, 8 tiles) 20.4 unsplit and 27.0 as four splits, 12 after 500 (8
    // units, 8 tiles) 17.9 and 12.2.
    p.units = (int64_t)B->n_seq * C->n_kv_heads * p.row_blocks;
    p.one_tiles = p.decode ? 16 : p.units >= 64 ? 8 : 6;
    const int64_t tiles = ceil_div((int64_t)B->table_stride * C->page_size, p.bn);
    const int64_t want = 2 * 256 / (p.units < 512 ? p.units : 512);
    const int64_t most = tiles <= p.one_tiles ? 1 : ceil_div(tiles, p.min_tiles);
    p.S = (int)(want < most ? want : most);
    p.S = p.S < 1 ? 1 : p.S > kMaxSplits ? kMaxSplits : p.S;
    if (p.S > 1) {
        const size_t n = (size_t)p.units * p.S * p.rows;
        p.part = align256(n * dp * sizeof(float));
        p.stat = align256(n * 2 * sizeof(float));
    }
    return p;
}

} // namespace

int attn_join_launch(const AttnArgs &a, int type, int64_t units, hipStream_t st)
{
    return type == RFX_BF16 ? join<BF16>(a, units, st) : join<F16>(a, units, st);
}

} // namespace rfx

using namespace rfx;

extern "C" {

size_t rfx_attn_workspace_bytes(const rfx_kv_cache *C, const rfx_kv_batch *B, int n_heads)
{
    if (!C || !B || C->n_kv_heads < 1 || n_heads < 1 || n_heads % C->n_kv_heads || C->head_dim < 8 ||
        C->head_dim > kMaxHeadDim || C->page_size < 1 || B->n_seq < 1 || B->max_q < 1 || B->max_q > kMaxTokens || B->table_stride < 1)
        return 0;
    const Plan p = plan(C, B, n_heads);
    return p.part + p.stat;
}

int rfx_attn(const void *q, const rfx_kv_cache *C, const rfx_kv_batch *B, int n_heads, float scale, int window,
             int sinks, void *out, int out_type, void *ws, size_t ws_bytes, void *stream)
{
    int st = check_kv(C, B, n_heads, "rfx_attn");
    if (st)
        return st;
    if (!(scale > 0.0f) || scale > 0x1p127f)
        return fail(RFX_E_INVAL, "rfx_attn: scale=%g (positive, at most 2^127)", (double)scale);
    if (window < 0 || sinks < 0)
        return fail(RFX_E_INVAL, "rfx_attn: window=%d sinks=%d", window, sinks);
    if (out_type != RFX_F32 && out_type != C->type)
        return fail(RFX_E_INVAL, "rfx_attn: out_type=%d (RFX_F32 or the cache's type)", out_type);
    if ((st = check_ptr(q, 16, "q")) || (st = check_ptr(out, 16, "out")))
        return st;
    const Plan p = plan(C, B, n_heads);
    if (p.units * p.S >= (int64_t)kMaxTokens)
        return fail(RFX_E_INVAL, "rfx_attn: %d sequences of up to %d new tokens need more than %d workgroups",
                    B->n_seq, B->max_q, kMaxTokens);
    if (p.part + p.stat) {
        if (!ws || ws_bytes < p.part + p.stat)
            return fail(RFX_E_WORKSPACE, "rfx_attn: workspace %zu < %zu bytes", ws ? ws_bytes : (size_t)0, p.part + p.stat);
        if ((st = check_ptr(ws, 256, "ws")))
            return st;
    }
    if (B->n_tokens == 0)
        return RFX_OK;
    AttnArgs a{};
    a.kv = kv_args(C, B, n_heads);
    a.q = static_cast<const uint16_t *>(q);
    a.out = out;
    a.out_f32 = out_type == RFX_F32;
    a.c = scale * 1.4426950408889634f; // finite
    a.window = window < 1 << 30 ? window : 1 << 30; // positions are below 2^30: differences stay in 32 bits
    a.sinks = sinks;
    a.S = p.S;
    a.row_blocks = p.row_blocks;
    a.rows = p.rows;
    a.bn = p.bn;
    a.min_tiles = p.min_tiles;
    a.one_tiles = p.one_tiles;
    a.cap_shift = p.rows == 16 ? 5 : 3;
    a.div_s = Div(p.S);
    a.div_rb = Div(p.row_blocks);
    a.div_units = Div((uint32_t)p.units);
    if (p.S > 1) {
        a.part = static_cast<float *>(ws);
        a.stat = reinterpret_cast<float *>(static_cast<char *>(ws) + p.part);
    }
    st = p.decode ? attn_decode_launch(a, C->type, p.row_tiles, (hipStream_t)stream)
                  : attn_prefill_launch(a, C->type, (hipStream_t)stream);
    return st || p.S == 1 ? st : attn_join_launch(a, C->type, p.units, (hipStream_t)stream);
}

} // extern "C"
