// Host side of the paged-cache entry points: argument checks, the choice of
// kernel and split, workspace sizes.
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

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

struct Plan {
    bool decode;
    int row_tiles;   // decode: 16-row tiles per workgroup
    int row_blocks;
    int S, min_tiles;
    int64_t units;   // (sequence, kv head, row block)
    size_t part, cnt;
};

// The decode kernel serves up to 32 rows (new tokens x query heads of a kv
// head) in one pass over the keys, 16 with heads over 128 elements (its
// accumulators would not fit the registers); more rows go to the prefill
// kernel, whose matrix-core tiles have 32. Keys are split as far as needed
// for about two workgroups per compute unit.
Plan plan(const rfx_kv_cache *C, const rfx_kv_batch *B, int n_heads)
{
    Plan p{};
    const int64_t rows = (int64_t)B->max_q * (n_heads / C->n_kv_heads);
    const int dp = C->head_dim <= 64 ? 64 : C->head_dim <= 128 ? 128 : 256;
    p.decode = rows <= (dp == 256 ? 16 : 32);
    const int per_block = p.decode ? (rows <= 16 ? 16 : 32) : 128;
    p.row_tiles = per_block / 16;
    p.row_blocks = (int)((rows + per_block - 1) / per_block);
    const int bn = p.decode ? 32 : dp == 256 ? 32 : 64;
    p.min_tiles = p.decode ? 8 : 4;
    const int64_t tiles = ceil_div((int64_t)B->table_stride * C->page_size, bn);
    p.units = (int64_t)B->n_seq * C->n_kv_heads * p.row_blocks;
    const int64_t want = 2 * 256 / (p.units < 512 ? p.units : 512);
    const int64_t most = ceil_div(tiles, p.min_tiles);
    p.S = (int)(want < most ? want : most);
    if (p.S < 1)
        p.S = 1;
    if (p.S > 64)
        p.S = 64;
    if (p.S > 1) {
        p.part = align256((size_t)p.units * p.S * per_block * (dp + 2) * sizeof(float));
        p.cnt = align256((size_t)p.units * sizeof(unsigned));
    }
    return p;
}

} // namespace
} // namespace rfx

using namespace rfx;

extern "C" {

size_t rfx_attn_workspace_bytes(const rfx_kv_cache *C, const rfx_kv_batch *B, int n_heads)
{
    if (!C || !B || C->n_kv_heads < 1 || n_heads < 1 || n_heads % C->n_kv_heads || C->head_dim < 8 ||
        C->head_dim > kMaxHeadDim || C->page_size < 1 || B->n_seq < 1 || B->max_q < 1 || B->max_q > kMaxTokens || B->table_stride < 1)
        return 0;
    const Plan p = plan(C, B, n_heads);
    return p.part + p.cnt;
}

int rfx_attn(const void *q, const rfx_kv_cache *C, const rfx_kv_batch *B, int n_heads, float scale, int window,
             int sinks, void *out, int out_type, void *ws, size_t ws_bytes, void *stream)
{
    int st = check_kv(C, B, n_heads, "rfx_attn");
    if (st)
        return st;
    if (!(scale > 0.0f) || std::isinf(scale))
        return fail(RFX_E_INVAL, "rfx_attn: scale=%g (positive and finite)", (double)scale);
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
    if (p.part + p.cnt) {
        if (!ws || ws_bytes < p.part + p.cnt)
            return fail(RFX_E_WORKSPACE, "rfx_attn: workspace %zu < %zu bytes", ws ? ws_bytes : (size_t)0, p.part + p.cnt);
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
    a.c = scale * 1.4426950408889634f;
    a.window = window;
    a.sinks = sinks;
    a.S = p.S;
    a.row_blocks = p.row_blocks;
    a.min_tiles = p.min_tiles;
    a.cnt = static_cast<unsigned *>(ws);
    a.part = reinterpret_cast<float *>(static_cast<char *>(ws) + p.cnt);
    return p.decode ? attn_decode_launch(a, C->type, p.row_tiles, (hipStream_t)stream)
                    : attn_prefill_launch(a, C->type, (hipStream_t)stream);
}

} // extern "C"
