// Weight and activation fragments of the matrix-core paths (prefill FFN,
// packed product): a lane's eight weights of a 32-weight block as the f16 B
// operand of v_mfma_f32_16x16x32_f16, int8 codes as f16, and direct loads
// into LDS.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "rfx_decode.h"

namespace rfx {
namespace dev {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// f16 high bytes of the codebook values (the low bytes are zero).
// FP2 {-3, -1, 1, 3}; FP3 {-7, -5, ..., 7}; FP4 magnitudes {0, 1, 2, 3, 4,
// 6, 8, 12} (2 x E2M1), the sign going to bit 7.
constexpr uint32_t kH2 = 0x423CBCC2u;
constexpr uint32_t kH3Lo = 0xBCC2C5C7u, kH3Hi = 0x4745423Cu;
constexpr uint32_t kH4Lo = 0x42403C00u, kH4Hi = 0x4A484644u;

// One lane's packed words of half a 256-column tile (4 blocks): per block,
// the word that holds its K group (FP3: the low-bit word, then the
// high-bit word), and its row's four block scales.
template <int F>
struct WHalf {
    uint32_t c[F == RFX_FP3 ? 8 : 4];
    uint32_t s[F == RFX_FP4 ? 1 : 2];
};

// Half hf of tile `tile`, row r (0..63), lane K group g.
template <int F>
__device__ __forceinline__ WHalf<F> load_whalf(const uint8_t *__restrict__ tile, int r, int g, int hf)
{
    WHalf<F> w;
    const uint8_t *rp = tile + r * 16;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int b = 4 * hf + j;
        if constexpr (F == RFX_FP4) {
            w.c[j] = *reinterpret_cast<const uint32_t *>(rp + b * 1024 + g * 4);
        } else {
            const uint32_t lo = *reinterpret_cast<const uint32_t *>(rp + (b >> 1) * 1024 + (b & 1) * 8 + (g >> 1) * 4);
            if constexpr (F == RFX_FP3) {
                w.c[2 * j] = lo;
                w.c[2 * j + 1] = *reinterpret_cast<const uint32_t *>(rp + (4 + hf) * 1024 + j * 4);
            } else {
                w.c[j] = lo;
            }
        }
    }
    if constexpr (F == RFX_FP4) {
        w.s[0] = *reinterpret_cast<const uint32_t *>(tile + 8192 + r * 8 + 4 * hf);
    } else {
        const u32x2 sc = *reinterpret_cast<const u32x2 *>(rp + (F == RFX_FP3 ? 6 : 4) * 1024 + 8 * hf);
        w.s[0] = sc.x;
        w.s[1] = sc.y;
    }
    return w;
}

// Weights 8g..8g+7 of block j of the half as eight f16 values.
template <int F>
__device__ __forceinline__ f16x8 wfrag(const WHalf<F> &w, int j, int g)
{
    uint32_t ha, hb; // f16 high bytes of weights 8g..8g+3 and 8g+4..8g+7
    if constexpr (F == RFX_FP4) {
        // word g: weight 8g + 4i + j at bits 8j + 4i
        const uint32_t na = w.c[j] & 0x0F0F0F0Fu, nb = (w.c[j] >> 4) & 0x0F0F0F0Fu;
        ha = __builtin_amdgcn_perm(kH4Hi, kH4Lo, na & 0x07070707u) | ((na << 4) & 0x80808080u);
        hb = __builtin_amdgcn_perm(kH4Hi, kH4Lo, nb & 0x07070707u) | ((nb << 4) & 0x80808080u);
    } else {
        // word g / 2: weight 16m + 4i + j at bits 8j + 2i; the K group
        // takes i = 2 (g % 2) and i + 1
        const uint32_t word = F == RFX_FP3 ? w.c[2 * j] : w.c[j];
        const uint32_t sh = 4u * (uint32_t)(g & 1);
        uint32_t sa = (word >> sh) & 0x03030303u, sb = (word >> (sh + 2u)) & 0x03030303u;
        if constexpr (F == RFX_FP3) {
            // high bit of weight 4i + j at bit 8j + i, i = 2g and 2g + 1
            const uint32_t h = w.c[2 * j + 1] >> (2u * (uint32_t)g);
            sa |= (h & 0x01010101u) << 2;
            sb |= ((h >> 1) & 0x01010101u) << 2;
            ha = __builtin_amdgcn_perm(kH3Hi, kH3Lo, sa);
            hb = __builtin_amdgcn_perm(kH3Hi, kH3Lo, sb);
        } else {
            ha = __builtin_amdgcn_perm(0u, kH2, sa);
            hb = __builtin_amdgcn_perm(0u, kH2, sb);
        }
    }
    const u32x4 v = {__builtin_amdgcn_perm(0u, ha, 0x010C000Cu), __builtin_amdgcn_perm(0u, ha, 0x030C020Cu),
                     __builtin_amdgcn_perm(0u, hb, 0x010C000Cu), __builtin_amdgcn_perm(0u, hb, 0x030C020Cu)};
    return __builtin_bit_cast(f16x8, v);
}

// Weight scale of block j of the half, for the lane's row.
template <int F>
__device__ __forceinline__ float wscale(const WHalf<F> &w, int j)
{
    if constexpr (F == RFX_FP4) {
        const uint32_t e = (w.s[0] >> (8 * j)) & 0xffu;
        return ldexpf(1.0f, (int)e - 128);
    } else {
        const uint32_t s2 = w.s[j >> 1];
        return half_bits_to_float((j & 1) ? (s2 >> 16) : (s2 & 0xffffu));
    }
}

// Four int8 codes -> two dwords of f16 (exact: f16 holds 1024 + u exactly
// for u = x + 128 in 0..255).
__device__ __forceinline__ void i8x4_to_f16(uint32_t x, uint32_t &p01, uint32_t &p23)
{
    const uint32_t u = x ^ 0x80808080u;
    const f16x2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
    p01 = __builtin_bit_cast(uint32_t,
                             __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - off);
    p23 = __builtin_bit_cast(uint32_t,
                             __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - off);
}

// Direct loads into LDS: each lane's 16 (4) bytes land at lds_dst + 16 (4) *
// lane.
__device__ __forceinline__ void lds_dma16(const void *src, void *lds_dst)
{
    typedef const __attribute__((address_space(1))) void *gptr;
    typedef __attribute__((address_space(3))) void *lptr;
    __builtin_amdgcn_global_load_lds((gptr)(uintptr_t)src, (lptr)(uint32_t)(uintptr_t)lds_dst, 16, 0, 0);
}

__device__ __forceinline__ void lds_dma4(const void *src, void *lds_dst)
{
    typedef const __attribute__((address_space(1))) void *gptr;
    typedef __attribute__((address_space(3))) void *lptr;
    __builtin_amdgcn_global_load_lds((gptr)(uintptr_t)src, (lptr)(uint32_t)(uintptr_t)lds_dst, 4, 0, 0);
}

} // namespace dev
} // namespace rfx
