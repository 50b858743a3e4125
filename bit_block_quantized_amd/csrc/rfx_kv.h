// What the paged key-value cache's kernels share: the launch arguments that
// describe cache and batch, their host checks, and the device-side types
// (16-bit elements, matrix-core products of them, transposed LDS reads).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "rfx.h"
#include "rfx_internal.h"

namespace rfx {

constexpr int kMaxHeadDim = 256;
constexpr int kMaxHeads = 1024;
constexpr int kMaxPage = 4096;
constexpr int kMaxTokens = 1 << 23; // a launch of one 256-thread workgroup per token stays below 2^32 threads

// Host checks of the two descriptors (no HIP calls); `who` names the entry
// point in the message. n_heads: query heads.
int check_kv(const rfx_kv_cache *C, const rfx_kv_batch *B, int n_heads, const char *who);


// Division of 0 <= n < 2^31 by a number known at launch, as a multiplication
// (the compiler's sequence for an unknown divisor is some 30 operations, and
// the kernels' setup has several in a row).
struct Div {
    uint32_t d, mul, shift;
    Div() = default;
    explicit Div(uint32_t v) : d(v), shift(v > 1 ? 32 - __builtin_clz(v - 1) : 0)
    {
        mul = (uint32_t)((((1ull << shift) - v) << 32) / v + 1);
    }
    __device__ __forceinline__ int operator()(int n) const { return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift); }
    __device__ __forceinline__ int rem(int n, int q) const { return n - q * (int)d; }
};

// Cache and batch as the kernels take them.
struct KvArgs {
    uint16_t *k, *v; // [n_pages][Hk][page][D]
    const int32_t *q_off, *kv_len, *table;
    int n_seq, n_tokens, max_q, stride;
    int n_pages, page_shift;
    int Hq, Hk, G, D;
    Div div_g, div_hk; // by G and Hk
};

inline KvArgs kv_args(const rfx_kv_cache *C, const rfx_kv_batch *B, int n_heads)
{
    KvArgs a{};
    a.k = static_cast<uint16_t *>(C->k);
    a.v = static_cast<uint16_t *>(C->v);
    a.q_off = B->q_off;
    a.kv_len = B->kv_len;
    a.table = B->page_table;
    a.n_seq = B->n_seq;
    a.n_tokens = B->n_tokens;
    a.max_q = B->max_q;
    a.stride = B->table_stride;
    a.n_pages = C->n_pages;
    a.page_shift = __builtin_ctz((unsigned)C->page_size);
    a.Hq = n_heads;
    a.Hk = C->n_kv_heads;
    a.G = n_heads / C->n_kv_heads;
    a.D = C->head_dim;
    a.div_g = Div(a.G);
    a.div_hk = Div(a.Hk);
    return a;
}

// Arguments of the attention kernels.
struct AttnArgs {
    KvArgs kv;
    const uint16_t *q; // [n_tokens][Hq][D]
    void *out;         // [n_tokens][Hq][D], fp32 or the cache's type
    int out_f32;
    float c;           // scale * log2(e)
    int window, sinks; // window 0: none
    int S;             // splits of a sequence's keys (grid)
    int row_blocks;    // row blocks of a (sequence, kv head) (grid)
    int rows;          // rows of a block
    int bn;            // keys of a tile
    int min_tiles;     // key tiles a split takes at least
    int one_tiles;     // up to so many key tiles are not split
    int cap_shift;     // see split_tiles
    Div div_s, div_rb, div_units; // by S, row_blocks and units
    // workspace, where S > 1, by unit = (seq * row_blocks + block) * Hk + hk:
    float *part;       // [unit][split][rows][DP] unnormalized results
    float *stat;       // [unit][split][rows][2] their maxima and sums
};

// The two-group prefill kernel: rows of a block, and the page ids that its
// LDS holds (for 64 keys one of each page they touch).
constexpr int kPairRows = 256, kPairIds = 4096;

int attn_decode_launch(const AttnArgs &a, int type, int row_tiles, hipStream_t st);
int attn_prefill_launch(const AttnArgs &a, int type, hipStream_t st);
int attn_join_launch(const AttnArgs &a, int type, int64_t units, hipStream_t st);

namespace dev {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef float f2 __attribute__((ext_vector_type(2)));

// The two 16-bit element types. TERMS: how many of them carry a softmax
// weight where the result is fp32 (fp16 11 + 11 bits, bf16 8 + 8 + 8: about
// fp32's 24). BIAS: power of two that weights are scaled by, so that the
// small ones stay clear of fp16's subnormals (it cancels in the division by
// the sum); bf16 has fp32's exponents. LAG: power of two that weights may
// grow beyond the running maximum's before sums are rescaled (2^(BIAS + LAG)
// stays below fp16's largest value).
struct F16 {
    static constexpr int TERMS = 2;
    static constexpr float BIAS = 10.0f, LAG = 5.0f;
    static __device__ __forceinline__ float add_pair(uint32_t u, float x)
    {
        return __builtin_amdgcn_fdot2(__builtin_bit_cast(h2, u), (h2){(_Float16)1.0f, (_Float16)1.0f}, x, false);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, h2));
    }
    static __device__ __forceinline__ f2 unpack(uint32_t u)
    {
        return __builtin_convertvector(__builtin_bit_cast(h2, u), f2);
    }
    static __device__ __forceinline__ f32x4 mma16(u4 a, u4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mma32(u4 a, u4 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
    }
};

struct BF16 {
    static constexpr int TERMS = 3;
    static constexpr float BIAS = 0.0f, LAG = 8.0f;
    static __device__ __forceinline__ float add_pair(uint32_t u, float x)
    {
        return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2, u), (b2){(__bf16)1.0f, (__bf16)1.0f}, x, false);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){a, b}, b2));
    }
    static __device__ __forceinline__ f2 unpack(uint32_t u)
    {
        return (f2){__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)};
    }
    static __device__ __forceinline__ f32x4 mma16(u4 a, u4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mma32(u4 a, u4 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
    }
};

// Eight fp32 weights as N operands of 16-bit terms that sum to them: the
// first is the rounded value, each next the rounded remainder.
template <class T, int N>
__device__ __forceinline__ void split_terms(const float (&p)[8], u4 (&t)[N])
{
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; i++)
        r[i] = p[i];
#pragma unroll
    for (int n = 0; n < N; n++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t u = T::pack(r[2 * i], r[2 * i + 1]);
            t[n][i] = u;
            if (n + 1 < N) {
                const f2 back = T::unpack(u);
                r[2 * i] -= back.x;
                r[2 * i + 1] -= back.y;
            }
        }
}

// ds_read_b64_tr_b16: in each group of 16 lanes, lane i's address names 4
// consecutive elements of row i / 4 (columns 4 (i % 4) ..) of a 4 x 16
// block; it receives column i's four rows.
__device__ __forceinline__ u2 lds_read_tr(const char *p)
{
    typedef short s4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4 *lptr;
    return __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lptr)(uint32_t)(uintptr_t)p));
}

// A weight is exp2(c s - c m + BIAS), one fused operation per score. Where c m
// is large its rounding (2^-24 of it) moves all of a row's weights by one
// factor, which overflows fp16 from c m = 2^26 on, and by another one once m
// rises. From here on (an error of 2^-12 up to here) m is subtracted from the
// scores first.
constexpr float kFar = 4096.0f;

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// One sequence as a workgroup sees it, for the append and for attention. nq
// new tokens (rows t0 .., at most max_q), the first at position p0; kv cached
// tokens. nq = 0: none, or its rows leave the arrays, or its tokens the table
// (a position that was moved inside would overwrite an older token's slot).
struct Seq {
    int t0, nq, p0, kv;
};

__device__ __forceinline__ Seq load_seq(const KvArgs &a, int s)
{
    Seq q;
    const int t0 = __builtin_amdgcn_readfirstlane(a.q_off[s]);
    const int t1 = __builtin_amdgcn_readfirstlane(a.q_off[s + 1]);
    const int len = __builtin_amdgcn_readfirstlane(a.kv_len[s]);
    const int room = a.stride << a.page_shift;
    q.t0 = t0;
    q.kv = max(0, min(len, room));
    const bool ok = t0 >= 0 && t1 > t0 && t1 <= a.n_tokens && len <= room;
    q.nq = ok ? min(t1 - t0, a.max_q) : 0;
    q.p0 = ok ? q.kv - (t1 - t0) : 0;
    return q;
}

// The key tiles of bn keys that rows with first position p_lo and last
// position p_hi can see: the sinks' tiles, then those of the window.
struct KeyTiles {
    int hi;    // keys from hi on are after every row
    int lo;    // keys below lo are outside every row's window
    int sk;    // ... except the first sk
    int nst;   // tiles of the sinks
    int wt;    // first tile after them
    int n;     // tiles in all
};

__device__ __forceinline__ KeyTiles key_tiles(int bn, int p_lo, int p_hi, int kv, int window, int sinks)
{
    KeyTiles t;
    t.hi = max(0, min(kv, p_hi + 1));
    t.lo = window ? max(0, min(p_lo - window + 1, t.hi)) : 0;
    t.sk = min(sinks, t.lo);
    t.nst = (t.sk + bn - 1) / bn;
    t.wt = max(t.lo / bn, t.nst);
    t.n = t.nst + max(0, (t.hi + bn - 1) / bn - t.wt);
    return t;
}

// How a block's n key tiles are split: `per` tiles each over `active` of the
// grid's S splits. Few tiles are not split (joining costs more), and a split
// takes n / 2^cap_shift tiles, though not fewer than min_tiles nor, for
// that, more than 16: joining costs by splits and rows.
__device__ __forceinline__ void split_tiles(const AttnArgs &a, int n, int &per, int &active)
{
    if (n <= a.one_tiles || a.S == 1) {
        per = n;
        active = 1;
        return;
    }
    per = max(a.div_s(n + a.S - 1), max(a.min_tiles, min((n + (1 << a.cap_shift) - 1) >> a.cap_shift, 16)));
    active = (n + per - 1) / per;
}

// First key of the i-th tile.
template <int BN>
__device__ __forceinline__ int tile_key(const KeyTiles &t, int i)
{
    return (i < t.nst ? i : i - t.nst + t.wt) * BN;
}

} // namespace dev
} // namespace rfx
