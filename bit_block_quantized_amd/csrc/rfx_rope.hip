// Per-head RMS norms of queries and keys, the rotation by position, and the
// append of keys and values to the paged cache, in one pass.
//
//   y = x w / sqrt(mean(x^2) + eps)     (no weight given: y = x)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),   t = position * inv_freq
//
// Bound by memory: 4 bytes read and 2 written per element, each once. A
// head's vector sits in the registers of LPH lanes, eight elements each, so
// the norm's sum is a shuffle tree and both elements of every rotated pair
// are in one lane. A lane turns the same four pairs in every head of its
// token, so it evaluates its four angles once: position * inv_freq / 2 pi in
// fp64, of which the whole turns are dropped before the rest goes to fp32
// (at position 2^20 an fp32 product would be off by 0.06 rad) and to the
// hardware's sine and cosine of turns (off by at most 2^-22, measured
// over 2^24 arguments; the result is rounded to 8 or 11 bits).
#include <type_traits>

#include "rfx_kv.h"

using namespace rfx;
using namespace rfx::dev;

namespace {

struct RopeArgs {
    KvArgs kv;
    const float *q, *k, *v;
    int64_t qs, ks, vs; // row strides, elements
    const double *inv_freq;
    const float *wq, *wk;
    float eps;
    int rot, pairs;
    uint16_t *qo;
};

// Sequence of row t: the last s with q_off[s] <= t, or -1 for rows before
// the first and behind the last sequence. 64 lanes probe at a time.
__device__ __forceinline__ int find_seq(const int32_t *q_off, int n, int t)
{
    const int lane = threadIdx.x & 63;
    const int first = q_off[0], last = q_off[n];
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 64) / 65;
        const int i = lo + (lane + 1) * step;
        const bool le = i < hi && q_off[min(i, n)] <= t;
        const int c = __popcll(__ballot(le));
        hi = min(hi, lo + (c + 1) * step);
        lo += c * step;
    }
    return t >= first && t < last ? lo : -1;
}

// Sum over the LPH (8, 16 or 32) lanes of a head: neighbours, pairs and
// halves by the vector pipe's own lane exchanges.
template <int LPH>
__device__ __forceinline__ float head_sum(float x)
{
    const auto add = [&](auto ctrl) {
        x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xf, 0xf, true));
    };
    add(std::integral_constant<int, 0xB1>{});  // lanes 1 0 3 2
    add(std::integral_constant<int, 0x4E>{});  // lanes 2 3 0 1
    add(std::integral_constant<int, 0x141>{}); // 7 - i of 8
    if (LPH >= 16)
        add(std::integral_constant<int, 0x140>{}); // 15 - i of 16
    if (LPH == 32) {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    return x;
}

// One workgroup of four waves per token and share (blockIdx.y) of its
// heads; a wave takes 64 / LPH heads at a time: queries, keys, then values.
template <class T, int LPH, bool NT>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a)
{
    constexpr int HPW = 64 / LPH;
    const int lane = threadIdx.x & 63, l = lane & (LPH - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = blockIdx.x;
    const int Hq = a.kv.Hq, Hk = a.kv.Hk, D = a.kv.D, H = Hq + 2 * Hk;
    const bool on = 8 * l < D;
    const bool turned = 8 * l < a.rot;
    // the lane's two groups of four elements: both halves of its pairs, or
    // (adjacent pairs, and elements that are not turned) eight in a row
    const bool halves = !a.pairs && turned;
    const int e0 = halves ? 4 * l : 8 * l, e1 = halves ? a.rot / 2 + 4 * l : 8 * l + 4;
    const int step = 4 * HPW * gridDim.y;
    int h = (blockIdx.y * 4 + wave) * HPW + lane / LPH;

    const auto source = [&](int h) {
        return h < Hq ? a.q + t * a.qs + h * D : h < Hq + Hk ? a.k + t * a.ks + (h - Hq) * D : a.v + t * a.vs + (h - Hq - Hk) * D;
    };
    const float *p = source(min(h, H - 1));
    const auto load = [&](int e) {
        const f32x4 *q = reinterpret_cast<const f32x4 *>(p + (on ? e : 0));
        return NT ? __builtin_nontemporal_load(q) : *q;
    };
    const auto store = [&](uint16_t *q, auto v) {
        if (NT)
            __builtin_nontemporal_store(v, reinterpret_cast<decltype(v) *>(q));
        else
            *reinterpret_cast<decltype(v) *>(q) = v;
    };
    f32x4 x0 = load(e0), x1 = load(e1);

    const int s = find_seq(a.kv.q_off, a.kv.n_seq, t);
    if (s < 0)
        return; // rows of no sequence stay as they are
    const Seq sq = load_seq(a.kv, s);
    if (sq.nq <= 0)
        return;
    const int pos = sq.p0 + (t - sq.t0);
    // the cache row of the new token: none before the first position
    const int pg = pos >> a.kv.page_shift;
    const int id = pos >= 0 && pg < a.kv.stride ? a.kv.table[(size_t)s * a.kv.stride + pg] : -1;
    const bool put = id >= 0 && id < a.kv.n_pages;
    const size_t slot = (size_t)(pos & ((1 << a.kv.page_shift) - 1));

    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    f32x4 wq0 = {1.f, 1.f, 1.f, 1.f}, wq1 = wq0, wk0 = wq0, wk1 = wq0;
    if (turned && on) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const double turns = (double)pos * a.inv_freq[4 * l + i] * 0.15915494309189533577;
            const float f = (float)(turns - rint(turns)); // -0.5 .. 0.5
            sn[i] = __builtin_amdgcn_sinf(f); // of turns
            cs[i] = __builtin_amdgcn_cosf(f);
        }
    }
    if (on && a.wq) {
        wq0 = *reinterpret_cast<const f32x4 *>(a.wq + e0);
        wq1 = *reinterpret_cast<const f32x4 *>(a.wq + e1);
    }
    if (on && a.wk) {
        wk0 = *reinterpret_cast<const f32x4 *>(a.wk + e0);
        wk1 = *reinterpret_cast<const f32x4 *>(a.wk + e1);
    }

    const float inv_d = 1.0f / (float)D;
    for (int base = h - lane / LPH; base < H; base += step, h += step) {
        f32x4 y0 = x0, y1 = x1;
        const int hn = min(h + step, H - 1); // the next head's loads, always in bounds
        p = source(hn);
        x0 = load(e0);
        x1 = load(e1);
        const bool is_q = h < Hq, is_v = h >= Hq + Hk;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 4; i++)
            ss += on ? y0[i] * y0[i] + y1[i] * y1[i] : 0.f;
        ss = head_sum<LPH>(ss);
        if (!is_v) {
            const bool norm = is_q ? a.wq != nullptr : a.wk != nullptr;
            const float r = norm ? __builtin_amdgcn_rsqf(ss * inv_d + a.eps) : 1.0f; // to 2^-22
            const f32x4 w0 = is_q ? wq0 : wk0, w1 = is_q ? wq1 : wk1;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                y0[i] *= r * w0[i];
                y1[i] *= r * w1[i];
            }
            if (halves) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float u = y0[i], w = y1[i];
                    y0[i] = u * cs[i] - w * sn[i];
                    y1[i] = w * cs[i] + u * sn[i];
                }
            } else if (turned) {
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const float u = y0[2 * i], w = y0[2 * i + 1], u1 = y1[2 * i], w1b = y1[2 * i + 1];
                    y0[2 * i] = u * cs[i] - w * sn[i];
                    y0[2 * i + 1] = w * cs[i] + u * sn[i];
                    y1[2 * i] = u1 * cs[2 + i] - w1b * sn[2 + i];
                    y1[2 * i + 1] = w1b * cs[2 + i] + u1 * sn[2 + i];
                }
            }
        }
        if (!on || h >= H || (!is_q && !put))
            continue;
        const int hk = is_v ? h - Hq - Hk : h - Hq;
        uint16_t *o = is_q ? a.qo + ((size_t)t * Hq + h) * D
                           : (is_v ? a.kv.v : a.kv.k) + ((((size_t)id * Hk + hk) << a.kv.page_shift) + slot) * D;
        // one rounding to the cache's type, to nearest even
        const u2 r0 = {T::pack(y0[0], y0[1]), T::pack(y0[2], y0[3])}, r1 = {T::pack(y1[0], y1[1]), T::pack(y1[2], y1[3])};
        if (halves) {
            store(o + e0, r0);
            store(o + e1, r1);
        } else {
            store(o + e0, (u4){r0.x, r0.y, r1.x, r1.y});
        }
    }
}

template <class T>
int launch(const RopeArgs &a, hipStream_t st)
{
    const int D = a.kv.D, H = a.kv.Hq + 2 * a.kv.Hk;
    const int lph = D <= 64 ? 8 : D <= 128 ? 16 : 32;
    const int per = 4 * 64 / lph; // heads of one pass of a workgroup
    // few tokens: a token's heads over several workgroups, one pass each;
    // with many, one workgroup per token evaluates the angles once per wave
    const int passes = (H + per - 1) / per;
    const bool few = a.kv.n_tokens < 512;
    const dim3 grid(a.kv.n_tokens, few ? passes : 1), block(256);
    // Many tokens' rows are more than the caches hold until they are used:
    // past them (79 to 71 us for 10858 tokens of 48 heads of 128, the only
    // size it was measured at; 512 tokens, 19 MB, would fit them).
#define RFX_ROPE(LPH)                                                               \
    if (few)                                                                        \
        hipLaunchKernelGGL((rope_kernel<T, LPH, false>), grid, block, 0, st, a);    \
    else                                                                            \
        hipLaunchKernelGGL((rope_kernel<T, LPH, true>), grid, block, 0, st, a);
    if (lph == 8) {
        RFX_ROPE(8)
    } else if (lph == 16) {
        RFX_ROPE(16)
    } else {
        RFX_ROPE(32)
    }
#undef RFX_ROPE
    return hip_status("qk_norm_rope launch");
}

} // namespace

extern "C" int rfx_qk_norm_rope(const rfx_qk_rope *R, const rfx_kv_cache *C, const rfx_kv_batch *B, void *q_out,
                                void *stream)
{
    if (!R)
        return fail(RFX_E_INVAL, "rfx_qk_norm_rope: arguments are NULL");
    int st = check_kv(C, B, R->n_heads, "rfx_qk_norm_rope");
    if (st)
        return st;
    const int D = C->head_dim;
    if (R->rot_dim < 0 || R->rot_dim > D || R->rot_dim % 8)
        return fail(RFX_E_INVAL, "rfx_qk_norm_rope: rot_dim=%d (a multiple of 8 from 0 to head_dim=%d)", R->rot_dim, D);
    if (!(R->eps >= 0.0f) || R->eps > 1e30f)
        return fail(RFX_E_INVAL, "rfx_qk_norm_rope: eps=%g", (double)R->eps);
    const struct {
        int64_t stride;
        int heads;
        const char *name;
    } rows[3] = {{R->q_stride, R->n_heads, "q"}, {R->k_stride, C->n_kv_heads, "k"}, {R->v_stride, C->n_kv_heads, "v"}};
    for (const auto &r : rows)
        if (r.stride < (int64_t)r.heads * D || r.stride % 4 || r.stride > (int64_t)1 << 40)
            return fail(RFX_E_INVAL, "rfx_qk_norm_rope: %s_stride=%lld (a multiple of 4, at least heads * head_dim)",
                        r.name, (long long)r.stride);
    if ((st = check_ptr(R->q, 16, "q")) || (st = check_ptr(R->k, 16, "k")) || (st = check_ptr(R->v, 16, "v")) ||
        (st = check_ptr(q_out, 16, "q_out")))
        return st;
    if (R->rot_dim && (st = check_ptr(R->inv_freq, 8, "inv_freq")))
        return st;
    if ((R->q_weight && (st = check_ptr(R->q_weight, 16, "q_weight"))) ||
        (R->k_weight && (st = check_ptr(R->k_weight, 16, "k_weight"))))
        return st;
    if (B->n_tokens == 0)
        return RFX_OK;
    RopeArgs a{};
    a.kv = kv_args(C, B, R->n_heads);
    a.q = R->q;
    a.k = R->k;
    a.v = R->v;
    a.qs = R->q_stride;
    a.ks = R->k_stride;
    a.vs = R->v_stride;
    a.inv_freq = R->inv_freq;
    a.wq = R->q_weight;
    a.wk = R->k_weight;
    a.eps = R->eps;
    a.rot = R->rot_dim;
    a.pairs = R->interleaved != 0;
    a.qo = static_cast<uint16_t *>(q_out);
    return C->type == RFX_BF16 ? launch<BF16>(a, (hipStream_t)stream) : launch<F16>(a, (hipStream_t)stream);
}
