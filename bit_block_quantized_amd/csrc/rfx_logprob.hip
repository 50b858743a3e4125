// Log probabilities of tokens from logits z [q][V]: the row's log sum of
// exponentials, its entropy, the given token's log probability and rank, and
// the k largest logits in order, ties to the lower index.
//
//   lse = M + log(s),  s = sum e^(z - M),  entropy = log(s) - sum e^(z - M) (z - M) / s
//
// Bound by memory where there are many rows: every logit is read once, by the
// first launch, in which a workgroup takes a chunk of a row into registers
// and leaves the chunk's maximum, sums, count and k best keys. A second
// launch, one workgroup per row, joins the chunks in 64 bits.
//
// The elements equal to the maximum are counted and the others' sum is kept
// apart from that count, so that a row with one likely token keeps the small
// rest (1 + 1e-9 is 1 in fp32), which its log probability and entropy are.
//
// The k best: an element is a key of 64 bits, the value's order above the
// complement of its index, so that no two are equal and ties are decided. In
// a set of 256 threads the ceil(k / 4)-th largest of a wave's 64 thread
// maxima is exceeded by that many elements of the wave; the least of the four
// waves' is a bound that at least k elements reach and, in random
// data, few more (k = 20 of 8192: about 40). They are compacted and ranked by
// counting. Where more than 256 reach it (equal logits, sorted
// ones), the k are taken out one after the other.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "rfx.h"
#include "rfx_internal.h"

using namespace rfx;

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kMaxTop = 64;
constexpr int kMaxVocab = 1 << 19;
constexpr int kLong = 32, kShort = 8;   // elements per thread of a chunk
constexpr int kJoinKeys = 32;           // keys per thread of the join
constexpr float kLog2e = 1.4426950408889634f;

// What a chunk leaves: its maximum, how many elements equal it, and over the
// others sum e^(z - m); sum e^(z - m) (z - m) over all; elements above the token's.
struct Stat {
    float m, n, rest, dot, above, pad[3];
};

struct LogpArgs {
    const void *z;
    int64_t stride;
    int q, V, k, S, chunk;
    const int32_t *tokens;
    Stat *stat;      // [q][S]
    uint64_t *keys;  // [q][S][k]
    rfx_logprob out;
};

// Keys order as values do, equal values by the lower index first; 0 is below
// every key. The two zeros are equal.
__device__ __forceinline__ uint32_t ordered(float v)
{
    const uint32_t u = __float_as_uint(v + 0.0f); // -0 becomes 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint64_t key)
{
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ uint64_t make_key(float v, int index) { return (uint64_t)ordered(v) << 32 | (uint32_t)~index; }
__device__ __forceinline__ int index_of(uint64_t key) { return (int)~(uint32_t)key; }

__device__ __forceinline__ uint64_t shfl64(uint64_t v, int o)
{
    return (uint64_t)__shfl_xor((uint32_t)(v >> 32), o, 64) << 32 | (uint32_t)__shfl_xor((uint32_t)v, o, 64);
}

struct Shared {
    uint64_t list[kThreads];
    uint64_t wave[kWaves];
    int count;
};

// The n-th largest (n >= 1) of a wave's 64 values, uniform: its bits one
// after the other, from the highest, by counting who reaches them.
__device__ __forceinline__ uint32_t nth_largest(uint32_t v, int n)
{
    uint32_t t = 0;
#pragma unroll 4
    for (int b = 31; b >= 0; b--) {
        const uint32_t u = t | 1u << b;
        if (__popcll(__ballot(v >= u)) >= n)
            t = u;
    }
    return t;
}
__device__ __forceinline__ uint64_t nth_largest(uint64_t v, int n)
{
    const uint32_t hi = (uint32_t)(v >> 32), h = nth_largest(hi, n);
    const int above = __popcll(__ballot(hi > h));
    const uint32_t lo = nth_largest(hi == h ? (uint32_t)v : 0u, n - above);
    return (uint64_t)h << 32 | lo;
}

// The k largest keys of the workgroup's to out[0..k), in descending order,
// 0 where there are fewer; key(j) is this thread's j-th of N, 0 for none;
// best: the largest of them. All threads call it.
template <int N, class Key>
__device__ __forceinline__ void top_keys(Shared &sh, int k, uint64_t best, Key &&key, uint64_t *out)
{
    const int tid = threadIdx.x, wave = tid >> 6;
    const uint64_t bound = nth_largest(best, (k + kWaves - 1) / kWaves);
    if ((tid & 63) == 0)
        sh.wave[wave] = bound;
    if (tid == 0)
        sh.count = 0;
    __syncthreads();
    uint64_t t = sh.wave[0];
#pragma unroll
    for (int w = 1; w < kWaves; w++)
        t = sh.wave[w] < t ? sh.wave[w] : t;
    t = t ? t : 1; // 0 is no key
    if (best >= t)
#pragma unroll
        for (int j = 0; j < N; j++) {
            const uint64_t v = key(j);
            if (v >= t) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < kThreads)
                    sh.list[at] = v;
            }
        }
    __syncthreads();
    const int n = sh.count;
    if (n <= kThreads) {
        const uint64_t mine = tid < n ? sh.list[tid] : 0;
        int rank = 0;
        for (int i = 0; i < n; i++)
            rank += sh.list[i] > mine;
        if (tid < n && rank < k)
            out[rank] = mine;
        if (tid >= n && tid < k)
            out[tid] = 0;
        return;
    }
    // one after the other: the largest key below the last
    uint64_t last = ~0ull;
    for (int i = 0; i < k; i++) {
        uint64_t m = 0;
#pragma unroll
        for (int j = 0; j < N; j++) {
            const uint64_t v = key(j);
            m = v < last && v > m ? v : m;
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const uint64_t v = shfl64(m, o);
            m = v > m ? v : m;
        }
        __syncthreads();
        if ((tid & 63) == 0)
            sh.wave[wave] = m;
        __syncthreads();
        m = sh.wave[0];
#pragma unroll
        for (int w = 1; w < kWaves; w++)
            m = sh.wave[w] > m ? sh.wave[w] : m;
        if (tid == 0)
            out[i] = m;
        last = m; // 0 once there are no more
    }
}

__device__ __forceinline__ float wave_sum(float x)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        x += __shfl_xor(x, o, 64);
    return x;
}
__device__ __forceinline__ float wave_max(float x)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        x = fmaxf(x, __shfl_xor(x, o, 64));
    return x;
}

template <int TYPE>
__device__ __forceinline__ float logit(const void *row, int i)
{
    if (TYPE == RFX_F32)
        return static_cast<const float *>(row)[i];
    if (TYPE == RFX_F16)
        return (float)static_cast<const _Float16 *>(row)[i];
    return __uint_as_float((uint32_t)static_cast<const uint16_t *>(row)[i] << 16);
}

// One workgroup per (row, chunk of E elements per thread). A thread's 16-byte
// loads are aligned, so that the row's elements start `lead` elements into
// the first; a load that the row fills only in part goes element by element.
template <int TYPE, int E>
__global__ __launch_bounds__(kThreads) void logprob_chunk_kernel(LogpArgs a)
{
    constexpr int PER = TYPE == RFX_F32 ? 4 : 8, LOADS = E / PER, SIZE = 16 / PER;
    __shared__ Shared sh;
    __shared__ Stat ws[kWaves];
    const int tid = threadIdx.x, wave = tid >> 6;
    const int row = blockIdx.x / a.S, c = blockIdx.x - row * a.S;
    const char *zr = static_cast<const char *>(a.z) + (int64_t)row * a.stride * SIZE;
    const int lead = (int)((reinterpret_cast<uintptr_t>(zr) & 15) / SIZE);
    const int token = a.tokens ? a.tokens[row] : -1;
    const bool known = (unsigned)token < (unsigned)a.V;

    float z[E];
    const auto index = [&](int l) { return c * a.chunk + (l * kThreads + tid) * PER - lead; }; // of a load's first element
#pragma unroll
    for (int l = 0; l < LOADS; l++) {
        const int i = index(l);
        if (i >= 0 && i + PER <= a.V) {
            const u32x4 u = *reinterpret_cast<const u32x4 *>(zr + (int64_t)i * SIZE);
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const uint32_t w = u[e]; // a bit cast of the vector's element itself reads another one
                if (TYPE == RFX_F32) {
                    z[l * PER + e] = __uint_as_float(w);
                } else if (TYPE == RFX_BF16) {
                    z[l * PER + 2 * e] = __uint_as_float(w << 16);
                    z[l * PER + 2 * e + 1] = __uint_as_float(w & 0xffff0000u);
                } else {
                    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
                    const h2 h = __builtin_bit_cast(h2, w);
                    z[l * PER + 2 * e] = (float)h[0];
                    z[l * PER + 2 * e + 1] = (float)h[1];
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < PER; e++)
                z[l * PER + e] = i + e >= 0 && i + e < a.V ? logit<TYPE>(zr, i + e) : -INFINITY;
        }
    }
    const float zt = known ? logit<TYPE>(zr, token) : INFINITY;

    // the thread's largest, the first of equal ones
    float top = -INFINITY, mx = -INFINITY;
    int at = 0;
#pragma unroll
    for (int j = 0; j < E; j++) {
        if (z[j] > top) {
            top = z[j];
            at = j;
        }
        mx = fmaxf(mx, z[j]);
    }
    const float m = wave_max(mx), base = m == -INFINITY ? 0.f : m;
    float rest = 0.f, dot = 0.f;
    int n = 0, above = 0;
#pragma unroll
    for (int j = 0; j < E; j++) {
        const float d = z[j] - base;
        const float e = __builtin_amdgcn_exp2f(d * kLog2e);
        const bool is_one = e == 1.0f;
        n += __popcll(__ballot(is_one));
        rest += is_one ? 0.f : e;
        dot = fmaf(e, fmaxf(d, -1e30f), dot); // 0 * -inf where nothing is left
        above += __popcll(__ballot(z[j] > zt));
    }
    rest = wave_sum(rest);
    dot = wave_sum(dot);
    if ((tid & 63) == 0)
        ws[wave] = Stat{m, (float)n, rest, dot, (float)above};
    __syncthreads();
    if (tid == 0) {
        Stat s = ws[0];
#pragma unroll
        for (int w = 1; w < kWaves; w++)
            s.m = fmaxf(s.m, ws[w].m);
        s.n = s.rest = s.dot = s.above = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; w++) {
            const Stat &p = ws[w];
            const float d = p.m == -INFINITY ? 0.f : fmaxf(p.m - s.m, -1e30f); // times the mass stays finite
            const float f = p.m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(d * kLog2e);
            const bool first = p.m == s.m;
            s.n += first ? p.n : 0.f;
            s.rest += first ? p.rest : f * (p.n + p.rest);
            s.dot += f * (p.dot + d * (p.n + p.rest));
            s.above += p.above;
        }
        a.stat[(size_t)row * a.S + c] = s;
    }
    if (a.k)
        top_keys<E>(sh, a.k, top > -INFINITY ? make_key(top, index(at / PER) + at % PER) : 0,
                    [&](int j) { return z[j] > -INFINITY ? make_key(z[j], index(j / PER) + j % PER) : 0; },
                    a.keys + ((size_t)row * a.S + c) * a.k);
}

// One workgroup per row.
__global__ __launch_bounds__(kThreads) void logprob_join_kernel(LogpArgs a)
{
    __shared__ Shared sh;
    __shared__ uint64_t best_keys[kMaxTop];
    __shared__ double part[kWaves][4];
    __shared__ float tops[kWaves];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const size_t row = blockIdx.x;
    const Stat *st = a.stat + row * a.S;

    float m = -INFINITY;
    for (int i = tid; i < a.S; i += kThreads)
        m = fmaxf(m, st[i].m);
    m = wave_max(m);
    if (lane == 0)
        tops[wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    double ones = 0.0, rest = 0.0, dot = 0.0, above = 0.0;
    for (int i = tid; i < a.S; i += kThreads) {
        const Stat p = st[i];
        above += p.above;
        if (p.m == -INFINITY && p.n + p.rest == 0.f)
            continue;
        const double d = (double)p.m - (double)m, f = p.m == m ? 1.0 : exp(d), mass = (double)p.n + (double)p.rest;
        ones += p.m == m ? (double)p.n : 0.0;
        rest += p.m == m ? (double)p.rest : f * mass;
        dot += f * ((double)p.dot + (p.m == m ? 0.0 : d * mass));
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        ones += __shfl_xor(ones, o, 64);
        rest += __shfl_xor(rest, o, 64);
        dot += __shfl_xor(dot, o, 64);
        above += __shfl_xor(above, o, 64);
    }
    if (lane == 0) {
        part[wave][0] = ones;
        part[wave][1] = rest;
        part[wave][2] = dot;
        part[wave][3] = above;
    }
    __syncthreads();
    ones = rest = dot = above = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
        ones += part[w][0];
        rest += part[w][1];
        dot += part[w][2];
        above += part[w][3];
    }
    const double s = ones + rest;
    const bool any = !(s == 0.0); // a row that nothing is left of: -inf, entropy 0
    const double ls = any ? log1p(ones - 1.0 + rest) : 0.0, lse = any ? (double)m + ls : -INFINITY;
    const auto logp = [&](float z) { return z == -INFINITY && ls == ls ? -INFINITY : (float)((double)z - (double)m - ls); };
    if (tid == 0) {
        const rfx_logprob &o = a.out;
        if (o.lse)
            o.lse[row] = (float)lse;
        if (o.entropy)
            o.entropy[row] = any ? (float)(ls - dot / s) : 0.f;
        const int token = a.tokens ? a.tokens[row] : -1;
        const bool known = (unsigned)token < (unsigned)a.V;
        if (o.rank)
            o.rank[row] = known ? (int)above : -1;
        if (o.logprob) {
            const int size = o.type == RFX_F32 ? 4 : 2;
            const char *zr = static_cast<const char *>(a.z) + (int64_t)row * a.stride * size;
            float z = 0.f;
            if (known)
                z = o.type == RFX_F32 ? logit<RFX_F32>(zr, token) : o.type == RFX_F16 ? logit<RFX_F16>(zr, token) : logit<RFX_BF16>(zr, token);
            o.logprob[row] = known ? logp(z) : 0.f;
        }
    }
    if (!a.k)
        return;
    // S lists of k: neighbouring threads of a wave take every fourth key
    const uint64_t *keys = a.keys + row * a.S * a.k;
    const int n = a.S * a.k, first = lane * kWaves + wave;
    uint64_t mine[kJoinKeys], best = 0;
#pragma unroll
    for (int j = 0; j < kJoinKeys; j++) {
        const int i = j * kThreads + first;
        mine[j] = i < n ? keys[i] : 0;
        best = mine[j] > best ? mine[j] : best;
    }
    top_keys<kJoinKeys>(sh, a.k, best, [&](int j) { return mine[j]; }, best_keys);
    __syncthreads();
    if (tid < a.k) {
        const uint64_t key = best_keys[tid];
        if (a.out.top_index)
            a.out.top_index[row * a.k + tid] = key ? index_of(key) : -1;
        if (a.out.top_logprob)
            a.out.top_logprob[row * a.k + tid] = key ? logp(value_of(key)) : -INFINITY;
    }
}

struct Plan {
    int E, chunk, S;
    size_t stat, keys;
};

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Chunks of 8192 logits, or of 2048 where the long ones would leave compute
// units idle and the join still holds the short ones' keys.
Plan plan(int q, int V, int k)
{
    Plan p{};
    // a row may start up to seven elements into its first 16 bytes
    const auto chunks = [&](int E) { return (int)ceil_div((int64_t)V + 7, (int64_t)E * kThreads); };
    const int fine = chunks(kShort);
    p.E = (int64_t)q * chunks(kLong) < 512 && (int64_t)fine * (k ? k : 1) <= kJoinKeys * kThreads ? kShort : kLong;
    p.chunk = p.E * kThreads;
    p.S = chunks(p.E);
    p.stat = align256((size_t)q * p.S * sizeof(Stat));
    p.keys = align256((size_t)q * p.S * k * sizeof(uint64_t));
    return p;
}

static_assert((kMaxVocab + 7 + kLong * kThreads - 1) / (kLong * kThreads) * kMaxTop <= kJoinKeys * kThreads, "the join holds all keys");

bool shape_ok(int q, int V, int k) { return q >= 0 && q <= RFX_LOGPROB_MAX_Q && V >= 1 && V <= kMaxVocab && k >= 0 && k <= kMaxTop; }

template <int E>
void launch(const LogpArgs &a, int type, hipStream_t st)
{
    const dim3 grid((unsigned)a.q * a.S), block(kThreads);
    if (type == RFX_F32)
        hipLaunchKernelGGL((logprob_chunk_kernel<RFX_F32, E>), grid, block, 0, st, a);
    else if (type == RFX_F16)
        hipLaunchKernelGGL((logprob_chunk_kernel<RFX_F16, E>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((logprob_chunk_kernel<RFX_BF16, E>), grid, block, 0, st, a);
}

} // namespace

extern "C" {

size_t rfx_token_logprobs_workspace_bytes(int q, int n_vocab, int top_k)
{
    if (!shape_ok(q, n_vocab, top_k))
        return 0;
    const Plan p = plan(q, n_vocab, top_k);
    return p.stat + p.keys;
}

int rfx_token_logprobs(const void *logits, int64_t stride, const int32_t *tokens, const rfx_logprob *O, void *ws, size_t ws_bytes,
                       void *stream)
{
    if (!O)
        return fail(RFX_E_INVAL, "rfx_token_logprobs: arguments are NULL");
    if (O->type != RFX_F32 && O->type != RFX_F16 && O->type != RFX_BF16)
        return fail(RFX_E_INVAL, "rfx_token_logprobs: type %d", O->type);
    if (!shape_ok(O->q, O->n_vocab, O->top_k))
        return fail(RFX_E_INVAL, "rfx_token_logprobs: q=%d n_vocab=%d top_k=%d (at most %d rows of 1 to %d, top_k from 0 to %d)",
                    O->q, O->n_vocab, O->top_k, RFX_LOGPROB_MAX_Q, kMaxVocab, kMaxTop);
    if (stride < O->n_vocab || stride > (int64_t)1 << 40)
        return fail(RFX_E_INVAL, "rfx_token_logprobs: stride=%lld (at least n_vocab=%d)", (long long)stride, O->n_vocab);
    int st = check_ptr(logits, O->type == RFX_F32 ? 4 : 2, "logits");
    if (st)
        return st;
    const struct {
        const void *p;
        const char *name;
    } optional[] = {{tokens, "tokens"}, {O->logprob, "logprob"}, {O->lse, "lse"}, {O->entropy, "entropy"}, {O->rank, "rank"},
                    {O->top_index, "top_index"}, {O->top_logprob, "top_logprob"}};
    for (const auto &o : optional)
        if (o.p && (st = check_ptr(o.p, 4, o.name)))
            return st;
    if (!tokens && (O->logprob || O->rank))
        return fail(RFX_E_INVAL, "rfx_token_logprobs: logprob and rank want tokens");
    if (!O->top_k && (O->top_index || O->top_logprob))
        return fail(RFX_E_INVAL, "rfx_token_logprobs: top_index and top_logprob want top_k");
    if (!O->logprob && !O->lse && !O->entropy && !O->rank && !O->top_index && !O->top_logprob)
        return fail(RFX_E_INVAL, "rfx_token_logprobs: no output");
    const Plan p = plan(O->q, O->n_vocab, O->top_k);
    if (!ws || ws_bytes < p.stat + p.keys) {
        if (O->q)
            return fail(RFX_E_WORKSPACE, "rfx_token_logprobs: workspace %zu < %zu bytes", ws ? ws_bytes : (size_t)0, p.stat + p.keys);
    } else if ((st = check_ptr(ws, 256, "ws"))) {
        return st;
    }
    if (O->q == 0)
        return RFX_OK;
    LogpArgs a{};
    a.z = logits;
    a.stride = stride;
    a.q = O->q;
    a.V = O->n_vocab;
    a.k = O->top_index || O->top_logprob ? O->top_k : 0;
    a.S = p.S;
    a.chunk = p.chunk;
    a.tokens = tokens;
    a.stat = static_cast<Stat *>(ws);
    a.keys = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) + p.stat);
    a.out = *O;
    const hipStream_t hs = (hipStream_t)stream;
    if (p.E == kShort)
        launch<kShort>(a, O->type, hs);
    else
        launch<kLong>(a, O->type, hs);
    if ((st = hip_status("token_logprobs chunk launch")))
        return st;
    hipLaunchKernelGGL(logprob_join_kernel, dim3(a.q), dim3(kThreads), 0, hs, a);
    return hip_status("token_logprobs join launch");
}

} // extern "C"
