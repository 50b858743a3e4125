// Log probabilities of tokens from logits z [q][V]: the row's log sum of
// exponentials, its entropy, the given token's log probability and rank, and
// the k largest logits in order, ties to the lower index.
//
//   lse = M + log(s),  s = sum e^(z - M),  entropy = log(s) - sum e^(z - M) (z - M) / s
//
// Every logit is read once, by the first launch, in which a workgroup takes a
// chunk of a row into registers and leaves the chunk's maximum, sums, count and
// k best keys. A second launch, one workgroup per row, joins the chunks in 64
// bits.
//
// Measured (both launches): one row of 32000 fp32 logits and five alternatives
// 7 us, latency; 64 rows of 131072, half of them -inf, and 20 alternatives 17,
// of which the join is 5 and reading takes 5; 1021 rows of 100003 bf16 logits
// 51 (204 MB, 4.0 TB/s; 30 at the rate of a large read). There the vector pipe
// is busy all the time: an element is some ten operations, an exponential
// among them, and there is nothing that the matrix pipe could take.
//
// Where little is beside the maximum, the elements equal to it are counted
// and the others' sum is kept apart from that count, so that a row with one
// likely token keeps the small rest (1 + 1e-9 is 1 in fp32), which its log
// probability and entropy are.
//
// The k best: an element is a key of 64 bits, the value's order above the
// complement of its index, so that no two are equal and ties are decided. In
// a workgroup the k-th largest of the threads' maxima is a bound that at least
// k elements reach and, in random data, few more (64 of 8192: about 75). They
// are listed and ranked by counting. Where more than 512 of a wave reach it
// (equal logits, sorted ones), the k are taken out one after the other.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "rfx.h"
#include "rfx_internal.h"

using namespace rfx;

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kMaxTop = 64;
constexpr int kList = 512; // 63 threads' eight elements fit: fewer than 64 that have any, at a row's end
constexpr int kMaxVocab = 1 << 19;
constexpr int kShort = 8;               // elements per thread of a short chunk
constexpr int kWaveTop = 8;            // up to so many alternatives a chunk is one wave's
constexpr int kLoads = 6;               // 16-byte loads per thread of a long one
constexpr int kJoinKeys = 32;           // keys per thread of the join
constexpr int kFewKeys = 8;             // of a join by one wave
constexpr float kLog2e = 1.4426950408889634f;

// What a wave's part of a chunk leaves: its maximum m; sum e^(z - m), as the number of elements
// that equal the maximum and the rest's sum where that is little, else all in
// `rest`; sum e^(z - m) (z - m); elements above the token's.
struct Stat {
    float m, n, rest, dot, above, pad[3];
};

struct LogpArgs {
    const void *z;
    int64_t stride;
    int q, V, k, S;
    int waves;       // of a chunk
    const int32_t *tokens;
    Stat *stat;      // [q][S][wave]
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

// Wave reductions by the vector pipe's lane exchanges: pairs, fours, eights,
// sixteens inside a row of 16, then rows and halves.
template <class V, class Op>
__device__ __forceinline__ V wave_reduce(V x, Op op)
{
    const auto dpp = [&](auto ctrl) {
        constexpr int N = sizeof(V) / 4;
        uint32_t u[N];
        __builtin_memcpy(u, &x, sizeof(V));
#pragma unroll
        for (int i = 0; i < N; i++)
            u[i] = __builtin_amdgcn_update_dpp(0, (int)u[i], decltype(ctrl)::value, 0xf, 0xf, true);
        V y;
        __builtin_memcpy(&y, u, sizeof(V));
        x = op(x, y);
    };
    dpp(std::integral_constant<int, 0xB1>{});  // lanes 1 0 3 2
    dpp(std::integral_constant<int, 0x4E>{});  // lanes 2 3 0 1
    dpp(std::integral_constant<int, 0x141>{}); // 7 - i of 8
    dpp(std::integral_constant<int, 0x140>{}); // 15 - i of 16
    constexpr int N = sizeof(V) / 4;
    uint32_t u[N], v[N];
    V y;
#pragma unroll
    for (int half = 0; half < 2; half++) {
        __builtin_memcpy(u, &x, sizeof(V));
#pragma unroll
        for (int i = 0; i < N; i++) {
            const auto r = half ? __builtin_amdgcn_permlane32_swap(u[i], u[i], false, false)
                                : __builtin_amdgcn_permlane16_swap(u[i], u[i], false, false);
            u[i] = r[0];
            v[i] = r[1];
        }
        __builtin_memcpy(&x, u, sizeof(V));
        __builtin_memcpy(&y, v, sizeof(V));
        x = op(x, y);
    }
    return x;
}
// A value that all lanes have, for branches that a wave takes as one.
__device__ __forceinline__ float uniform(float x) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x))); }

template <class V>
__device__ __forceinline__ V wave_sum(V x)
{
    return wave_reduce(x, [](V p, V q) { return p + q; });
}
__device__ __forceinline__ float wave_max(float x)
{
    return wave_reduce(x, [](float p, float q) { return fmaxf(p, q); });
}

template <int WAVES>
struct Shared {
    uint64_t list[WAVES][kList];
    uint64_t wave[WAVES];
    uint32_t top[64 * WAVES];
    int count[WAVES];
    int larger[WAVES > 1 ? kList * WAVES / 2 : 1]; // two counts of 16 bits each
    // The i-th of all lists' keys, which are `counts` long.
    __device__ __forceinline__ uint64_t at(int i, const int (&counts)[WAVES]) const
    {
        int w = 0;
#pragma unroll
        for (int u = 0; u < WAVES - 1; u++)
            if (w == u && i >= counts[u]) {
                i -= counts[u];
                w++;
            }
        return list[w][i];
    }
};

// The upper 16 bits of the n-th largest (n >= 1) of 64 N values, N per lane,
// the lower ones zero, uniform: its bits one after the other, from the highest,
// by counting who reaches them. 0: fewer than n values are not 0.
template <int N>
__device__ __forceinline__ uint32_t nth_largest(const uint32_t (&v)[N], int n)
{
    uint32_t t = 0;
#pragma unroll
    for (int b = 31; b >= 16; b--) {
        const uint32_t u = t | 1u << b;
        int count = 0;
#pragma unroll
        for (int i = 0; i < N; i++)
            count += __popcll(__ballot(v[i] >= u));
        t = count >= n ? u : t;
    }
    return t;
}

// The k largest keys of the workgroup's to out[0..k), in descending order,
// 0 where there are fewer. This thread's N elements are key(j), where reach(1)(j);
// best: the largest's upper half; reach(t)(j) for t > 0: whether the upper
// half of key(j) is t or more; anew(j) has the compiler forget what it knows
// of them. All threads call it.
template <int N, int WAVES, class Anew, class Reach, class Key>
__device__ __forceinline__ void top_keys(Shared<WAVES> &sh, int k, uint32_t best, Anew &&anew, Reach &&reach, Key &&key, uint64_t *out)
{
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    // the k-th largest of the threads' largest, which at least k elements reach
    uint32_t tops[WAVES], t;
    if constexpr (WAVES > 1) {
        sh.top[tid] = best;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; w++)
            tops[w] = sh.top[64 * w + lane];
    } else {
        tops[0] = best;
    }
    if (k == 1) {
        t = tops[0];
#pragma unroll
        for (int w = 1; w < WAVES; w++)
            t = max(t, tops[w]);
        t = __builtin_amdgcn_readfirstlane(wave_reduce(t, [](uint32_t p, uint32_t q) { return max(p, q); }));
    } else {
        t = nth_largest(tops, k);
    }
    t = max(t, 1u);
    const auto from = reach(t);
    // each wave lists its own, four elements a thread at a time
    uint64_t *list = sh.list[wave];
    int n = 0;
#pragma unroll
    for (int j0 = 0; j0 < N; j0 += 4) {
        uint64_t in[4];
#pragma unroll
        for (int j = 0; j < 4; j++)
            in[j] = __ballot(from(j0 + j));
        if (in[0] | in[1] | in[2] | in[3])
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (in[j]) {
                    const int at = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(in[j] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)in[j], 0));
                    if (from(j0 + j) && at < kList)
                        list[at] = key(j0 + j);
                    n += (int)__popcll(in[j]);
                }
    }
    if (lane == 0)
        sh.count[wave] = n;
    if constexpr (WAVES > 1)
        for (int i = tid; i < kList * WAVES / 2; i += 64 * WAVES)
            sh.larger[i] = 0;
    __syncthreads();
    int counts[WAVES], all = 0, most = 0;
#pragma unroll
    for (int w = 0; w < WAVES; w++) {
        counts[w] = __builtin_amdgcn_readfirstlane(sh.count[w]);
        all += counts[w];
        most = max(most, counts[w]);
    }
    if (most <= kList) {
        // each wave counts, for all, who of its own is larger
        for (int i = lane; i < all; i += 64) {
            const uint64_t mine = sh.at(i, counts);
            int larger = 0;
#pragma unroll 4
            for (int v = 0; v < n; v++)
                larger += list[v] > mine;
            if constexpr (WAVES > 1)
                atomicAdd(&sh.larger[i / 2], larger << (16 * (i & 1)));
            else if (larger < k)
                out[larger] = mine;
        }
        if constexpr (WAVES > 1) {
            __syncthreads();
            for (int i = tid; i < all; i += 64 * WAVES) {
                const int rank = sh.larger[i / 2] >> (16 * (i & 1)) & 0xffff;
                if (rank < k)
                    out[rank] = sh.at(i, counts);
            }
        }
        if (tid >= all && tid < k)
            out[tid] = 0;
        return;
    }
    // one after the other: the largest key below the last
    const auto any = reach(1u);
    uint64_t last = ~0ull;
    for (int i = 0; i < k; i++) {
        uint64_t m = 0;
#pragma unroll
        for (int j = 0; j < N; j++) {
            anew(j);
            const uint64_t v = any(j) ? key(j) : 0;
            m = v < last && v > m ? v : m;
            if (j % 4 == 3)
                asm volatile("" : "+v"(m));  // no more of them side by side
        }
        m = wave_reduce(m, [](uint64_t p, uint64_t q) { return p > q ? p : q; });
        __syncthreads();
        if ((tid & 63) == 0)
            sh.wave[wave] = m;
        __syncthreads();
        m = sh.wave[0];
#pragma unroll
        for (int w = 1; w < WAVES; w++)
            m = sh.wave[w] > m ? sh.wave[w] : m;
        if (tid == 0)
            out[i] = m;
        last = m; // 0 once there are no more
    }
}

template <int TYPE>
__device__ __forceinline__ uint32_t bits(const void *row, int i)
{
    return TYPE == RFX_F32 ? static_cast<const uint32_t *>(row)[i] : static_cast<const uint16_t *>(row)[i];
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

// The logit of a 32-bit word, of two the lower or the upper one.
template <int TYPE>
__device__ __forceinline__ float widen(uint32_t u, int upper)
{
    if (TYPE == RFX_F32)
        return __uint_as_float(u);
    if (TYPE == RFX_F16)
        return (float)__builtin_bit_cast(_Float16, (uint16_t)(upper ? u >> 16 : u));
    return __uint_as_float(upper ? u & 0xffff0000u : u << 16);
}

// One workgroup per (row, chunk of E elements per thread). A thread's 16-byte
// loads are aligned, so that the row's elements start `lead` elements into the
// first; a load that the row fills only in part goes element by element.
template <int TYPE, int E, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void logprob_chunk_kernel(LogpArgs a)
{
    constexpr int PER = TYPE == RFX_F32 ? 4 : 8, LOADS = E / PER, SIZE = 16 / PER;
    constexpr int CHUNK = E * 64 * WAVES;
    __shared__ Shared<WAVES> sh;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int row = blockIdx.x / a.S, c = blockIdx.x - row * a.S;
    const char *zr = static_cast<const char *>(a.z) + (int64_t)row * a.stride * SIZE;
    const int lead = (int)((reinterpret_cast<uintptr_t>(zr) & 15) / SIZE);
    const int token = a.tokens ? a.tokens[row] : -1;
    const bool known = (unsigned)token < (unsigned)a.V;

    int first = c * CHUNK + tid * PER - lead;
    const auto index = [&](int l) { return first + l * 64 * WAVES * PER; }; // of a load's first element
    const bool whole = c * CHUNK >= lead && (c + 1) * CHUNK - lead <= a.V; // uniform
    u32x4 raw[LOADS];
    if (whole) {
        const char *p = zr + ((int64_t)c * CHUNK - lead) * SIZE;
#pragma unroll
        for (int l = 0; l < LOADS; l++)
            raw[l] = *reinterpret_cast<const u32x4 *>(p + 16 * (unsigned)(l * 64 * WAVES + tid));
    } else { // what the row does not fill reads the workspace instead
#pragma unroll
        for (int l = 0; l < LOADS; l++) {
            const int i = index(l);
            const bool full = i >= 0 && i + PER <= a.V;
            raw[l] = *reinterpret_cast<const u32x4 *>(full ? zr + (int64_t)i * SIZE : reinterpret_cast<const char *>(a.stat));
        }
    }
    const float zt = uniform(known ? logit<TYPE>(zr, token) : INFINITY);

    if (!whole)
#pragma unroll
        for (int l = 0; l < LOADS; l++) {
            const int i = index(l);
            if (i < 0 || i + PER > a.V) {
                constexpr uint32_t none = TYPE == RFX_F32 ? 0xff800000u : TYPE == RFX_F16 ? 0xfc00u : 0xff80u; // -inf
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    uint32_t w = 0;
#pragma unroll
                    for (int h = 0; h < PER / 4; h++) {
                        const int at = i + e * (PER / 4) + h;
                        w |= (at >= 0 && at < a.V ? bits<TYPE>(zr, at) : none) << (16 * h);
                    }
                    raw[l][e] = w;
                }
            }
        }
    // 16-bit logits stay packed and are widened anew by each pass, and keys are
    // made anew: in half the registers or less a SIMD holds up to eight waves
    // instead of four (78 -> 70 us for 1021 rows of 100003 and eight
    // alternatives)
    uint32_t w[4 * LOADS];
#pragma unroll
    for (int i = 0; i < 4 * LOADS; i++)
        w[i] = raw[i / 4][i % 4]; // a bit cast of the vector's element itself reads another one
    const auto anew = [&](int j) { asm volatile("" : "+v"(w[j / (PER / 4)]), "+v"(first)); };
    const auto pass = [&]() {
        if constexpr (PER == 8)
#pragma unroll
            for (int i = 0; i < 4 * LOADS; i++)
                anew(2 * i);
    };
    const auto z = [&](int j) { return widen<TYPE>(w[j / (PER / 4)], j & 1); };

    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < E; j++)
        top = fmaxf(top, z(j));
    // e^(z - m) = 2^(c z - c m), one fused operation: c m is rounded, by
    // the same for all, and what it lacks is made up for below
    const float m = uniform(wave_max(top)), base = m == -INFINITY ? 0.f : m;
    const float off = base * kLog2e, lack = fmaf(base, kLog2e, -off);
    // two sums each: half the roundings on either
    float rests[2] = {0.f, 0.f}, dots[2] = {0.f, 0.f};
    pass();
#pragma unroll
    for (int j = 0; j < E; j++) {
        const float x = fmaf(z(j), kLog2e, -off), e = __builtin_amdgcn_exp2f(x);
        rests[j & 1] += e; // NaN where x is
        dots[j & 1] = fmaf(e, fmaxf(x, -1e30f), dots[j & 1]); // not 0 * -inf
    }
    const float fix = __builtin_amdgcn_exp2f(-lack), s = uniform(wave_sum(rests[0] + rests[1]));
    float rest = s * fix, dot = (wave_sum(dots[0] + dots[1]) - lack * s) * fix;
    int n = 0, above = 0;
    // Little beside the largest: the others alone. So too where c m lacks more
    // than 1 (from |m| of about 1e7 on, and where c m is past fp32's range): 2^lack
    // and 2^-lack would leave that range, and their product what it stands for.
    if (rest < 1.25f || !(fabsf(lack) <= 1.f)) {
        rests[0] = rests[1] = dots[0] = dots[1] = 0.f;
        pass();
#pragma unroll
        for (int j = 0; j < E; j++) {
            const float x = fmaxf((z(j) - m) * kLog2e, -1e30f), e = z(j) == m ? 0.f : __builtin_amdgcn_exp2f((z(j) - m) * kLog2e);
            rests[j & 1] += e;
            dots[j & 1] = fmaf(e, x, dots[j & 1]);
            n += z(j) == m;
            if (j % 4 == 3) // no more of them side by side: registers that the other passes would have to leave free
                asm volatile("" : "+v"(rests[0]), "+v"(rests[1]), "+v"(dots[0]), "+v"(dots[1]), "+v"(n));
        }
        rest = m == INFINITY ? NAN : wave_sum(rests[0] + rests[1]);
        dot = wave_sum(dots[0] + dots[1]);
        n = m == -INFINITY ? 0 : wave_sum(n);
    }
    if (m > zt) {
        pass();
#pragma unroll
        for (int j = 0; j < E; j++)
            above += __popcll(__ballot(z(j) > zt));
    }
    if (lane == 0) // from powers of two
        a.stat[((size_t)row * a.S + c) * WAVES + wave] = Stat{m, (float)n, rest, dot * 0.69314718055994531f, (float)above};
    if (!a.k)
        return;
    pass();
    const auto key = [&](int j) { return make_key(z(j), index(j / PER) + j % PER); };
    const auto reach = [&](uint32_t t) {
        const float from = fmaxf(value_of((uint64_t)t << 32), -3.4028234663852886e38f); // not -inf, which is no element
        return [&z, from](int j) { return z(j) >= from; };
    };
    top_keys<E, WAVES>(sh, a.k, top > -INFINITY ? ordered(top) : 0u, anew, reach, key, a.keys + ((size_t)row * a.S + c) * a.k);
}

// One workgroup per row, KEYS keys a thread.
template <int WAVES, int KEYS>
__global__ __launch_bounds__(64 * WAVES) void logprob_join_kernel(LogpArgs a)
{
    constexpr int THREADS = 64 * WAVES;
    __shared__ Shared<WAVES> sh;
    __shared__ uint64_t best_keys[kMaxTop];
    __shared__ double part[WAVES][4];
    __shared__ float tops[WAVES];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const size_t row = blockIdx.x;
    const rfx_logprob &o = a.out;
    const int parts = a.S * a.waves;
    const Stat *st = a.stat + row * parts;

    // Everything is read before it is waited for: the first statistics, the
    // keys, the token. Keys are S ordered lists of k, taken across the lists, all
    // first ones, all second ones, so that every thread has some of the best (a
    // bound from threads of which some have none lets most keys pass).
    const Stat none = {-INFINITY, 0.f, 0.f, 0.f, 0.f}, own = tid < parts ? st[tid] : none;
    const uint64_t *keys = a.keys + row * a.S * a.k;
    uint64_t mine[KEYS];
    {
        const int n = a.S * a.k, first = lane * WAVES + wave, step_pos = THREADS / a.S, step_list = THREADS - step_pos * a.S;
        int pos = first / a.S, list = first - pos * a.S;
#pragma unroll
        for (int j = 0; j < KEYS; j++) {
            mine[j] = 0;
            if (j * THREADS < n) { // uniform
                mine[j] = pos < a.k ? keys[list * a.k + pos] : 0;
                pos += step_pos;
                list += step_list;
                if (list >= a.S) {
                    list -= a.S;
                    pos++;
                }
            }
        }
    }
    const int token = a.tokens ? a.tokens[row] : -1;
    const bool known = (unsigned)token < (unsigned)a.V;
    float zt = 0.f;
    if (known) {
        const char *zr = static_cast<const char *>(a.z) + (int64_t)row * a.stride * (o.type == RFX_F32 ? 4 : 2);
        zt = o.type == RFX_F32 ? logit<RFX_F32>(zr, token) : o.type == RFX_F16 ? logit<RFX_F16>(zr, token) : logit<RFX_BF16>(zr, token);
    }

    float m = own.m;
    for (int i = tid + THREADS; i < parts; i += THREADS)
        m = fmaxf(m, st[i].m);
    m = wave_max(m);
    if (lane == 0)
        tops[wave] = m;
    __syncthreads();
    m = tops[0];
#pragma unroll
    for (int w = 1; w < WAVES; w++)
        m = fmaxf(m, tops[w]);
    m = uniform(m);
    double ones = 0.0, rest = 0.0, dot = 0.0, above = 0.0;
    const auto add = [&](const Stat &p) {
        above += p.above;
        if (p.m == -INFINITY && p.n + p.rest == 0.f)
            return;
        const float d = fmaxf(p.m - m, -1e30f);
        const double f = p.m == m ? 1.f : __builtin_amdgcn_exp2f(d * kLog2e), mass = (double)p.n + (double)p.rest;
        ones += p.m == m ? (double)p.n : 0.0;
        rest += p.m == m ? (double)p.rest : f * mass;
        dot += f * ((double)p.dot + (p.m == m ? 0.0 : (double)d * mass));
    };
    add(own);
    for (int i = tid + THREADS; i < parts; i += THREADS)
        add(st[i]);
    ones = wave_sum(ones);
    rest = wave_sum(rest);
    dot = wave_sum(dot);
    above = wave_sum(above);
    if (lane == 0) {
        part[wave][0] = ones;
        part[wave][1] = rest;
        part[wave][2] = dot;
        part[wave][3] = above;
    }
    __syncthreads();
    ones = rest = dot = above = 0.0;
#pragma unroll
    for (int w = 0; w < WAVES; w++) {
        ones += part[w][0];
        rest += part[w][1];
        dot += part[w][2];
        above += part[w][3];
    }
    const double s = ones + rest;
    const bool any = !(s == 0.0); // a row that nothing is left of: -inf, entropy 0
    const double ls = any ? log1p(ones - 1.0 + rest) : 0.0;
    const auto logp = [&](float z) { return z == -INFINITY && ls == ls ? -INFINITY : (float)((double)z - (double)m - ls); };
    if (tid == 0) {
        if (o.lse)
            o.lse[row] = any ? (float)((double)m + ls) : -INFINITY;
        if (o.entropy)
            o.entropy[row] = any ? (float)(ls - dot / s) : 0.f;
        if (o.rank)
            o.rank[row] = known ? (int)above : -1;
        if (o.logprob)
            o.logprob[row] = known ? logp(zt) : 0.f;
    }
    if (!a.k)
        return;
    uint64_t best = 0;
#pragma unroll
    for (int j = 0; j < KEYS; j++)
        best = mine[j] > best ? mine[j] : best;
    const auto reach = [&](uint32_t t) { return [&mine, t](int j) { return (uint32_t)(mine[j] >> 32) >= t; }; };
    top_keys<KEYS, WAVES>(sh, a.k, (uint32_t)(best >> 32), [](int) {}, reach, [&](int j) { return mine[j]; }, best_keys);
    __syncthreads();
    if (tid < a.k) {
        const uint64_t key = best_keys[tid];
        if (o.top_index)
            o.top_index[row * a.k + tid] = key ? index_of(key) : -1;
        if (o.top_logprob)
            o.top_logprob[row * a.k + tid] = key ? logp(value_of(key)) : -INFINITY;
    }
}

struct Plan {
    int E, waves, S;
    size_t stat, keys;
};

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// Chunks of six loads per thread (6144 fp32 or 12288 16-bit logits, a quarter
// of that for one wave), or of eight logits per thread where the long ones
// would leave compute units idle. 1021 rows of 100003 bf16 logits, with four,
// six, eight loads: 60, 58, 61 us; 300 of 131072 fp32 ones: 43 with four, 39
// with six.
Plan plan(int type, int q, int V, int k)
{
    Plan p{};
    // a row may start up to seven elements into its first 16 bytes
    const auto chunks = [&](int E, int waves) { return (int)ceil_div((int64_t)V + 7, (int64_t)E * 64 * waves); };
    const auto fits = [&](int E, int waves) { return (int64_t)chunks(E, waves) * k <= kJoinKeys * kThreads; };
    p.E = kLoads * (type == RFX_F32 ? 4 : 8);
    p.waves = k <= kWaveTop && fits(p.E, 1) ? 1 : kWaves;
    if ((int64_t)q * chunks(p.E, p.waves) * p.waves < 2048 && fits(kShort, p.waves))
        p.E = kShort;
    p.S = chunks(p.E, p.waves);
    p.stat = align256((size_t)q * p.S * p.waves * sizeof(Stat));
    p.keys = align256((size_t)q * p.S * k * sizeof(uint64_t));
    return p;
}

static_assert((kMaxVocab + 7 + 4 * kLoads * kThreads - 1) / (4 * kLoads * kThreads) * kMaxTop <= kJoinKeys * kThreads, "the join holds all keys");

bool shape_ok(int q, int V, int k) { return q >= 0 && q <= RFX_LOGPROB_MAX_Q && V >= 1 && V <= kMaxVocab && k >= 0 && k <= kMaxTop; }

template <int WAVES>
void launch(const LogpArgs &a, int type, int E, hipStream_t st)
{
    const dim3 grid((unsigned)a.q * a.S), block(64 * WAVES);
#define RFX_LOGP(TYPE, N) hipLaunchKernelGGL((logprob_chunk_kernel<TYPE, N, WAVES>), grid, block, 0, st, a)
    if (type == RFX_F32) {
        if (E == kShort)
            RFX_LOGP(RFX_F32, kShort);
        else
            RFX_LOGP(RFX_F32, 4 * kLoads);
    } else if (type == RFX_F16) {
        if (E == kShort)
            RFX_LOGP(RFX_F16, kShort);
        else
            RFX_LOGP(RFX_F16, 8 * kLoads);
    } else {
        if (E == kShort)
            RFX_LOGP(RFX_BF16, kShort);
        else
            RFX_LOGP(RFX_BF16, 8 * kLoads);
    }
#undef RFX_LOGP
}

// Whether one wave joins a row: no barriers, and more rows on a compute unit
// (one row of 32000 and five alternatives 7.0 us, with four waves 8.8; one of
// 128000 in 250 chunks 6.4 and 5.3).
bool few_keys(const LogpArgs &a) { return a.k <= 32 && a.S * a.k <= 64 * kFewKeys && a.S * a.waves <= 128; }

} // namespace

extern "C" {

size_t rfx_token_logprobs_workspace_bytes(int q, int n_vocab, int top_k)
{
    if (!shape_ok(q, n_vocab, top_k))
        return 0;
    // for logits of any type: fp32's chunks are the most
    const Plan a = plan(RFX_F32, q, n_vocab, top_k), b = plan(RFX_BF16, q, n_vocab, top_k);
    return std::max(a.stat, b.stat) + std::max(a.keys, b.keys);
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
    const Plan p = plan(O->type, O->q, O->n_vocab, O->top_k);
    const size_t need = rfx_token_logprobs_workspace_bytes(O->q, O->n_vocab, O->top_k);
    if (!ws || ws_bytes < need) {
        if (O->q)
            return fail(RFX_E_WORKSPACE, "rfx_token_logprobs: workspace %zu < %zu bytes", ws ? ws_bytes : (size_t)0, need);
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
    a.waves = p.waves;
    a.tokens = tokens;
    a.stat = static_cast<Stat *>(ws);
    a.keys = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) + p.stat);
    a.out = *O;
    const hipStream_t hs = (hipStream_t)stream;
    if (p.waves == 1)
        launch<1>(a, O->type, p.E, hs);
    else
        launch<kWaves>(a, O->type, p.E, hs);
    if ((st = hip_status("token_logprobs chunk launch")))
        return st;
    if (few_keys(a))
        hipLaunchKernelGGL((logprob_join_kernel<1, kFewKeys>), dim3(a.q), dim3(64), 0, hs, a);
    else
        hipLaunchKernelGGL((logprob_join_kernel<kWaves, kJoinKeys>), dim3(a.q), dim3(kThreads), 0, hs, a);
    return hip_status("token_logprobs join launch");
}

} // extern "C"
