// Epilogue of the packed products: y = resid + act(acc + bias), fp32.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "rfx.h"

namespace rfx {

// The split-K exchange slots that a single GEMV needs at most: row groups x
// (splits - 1) x 4 columns x 256 bytes, which is 329 KiB (47 groups, eight
// splits); rfx_gemv.hip checks it against the split rule.
constexpr size_t kGemvSlotBytes = 384u << 10;

struct EpiArgs {
    const float *bias;  // [N] or null
    const float *resid; // [q][N] or null
    int act;
};

namespace dev {

// SiLU and the tanh form of GELU as z / (1 + e^-u): where u is far below
// zero the exponential overflows and the quotient is zero. GELU through
// erfc, which keeps its relative accuracy at negative z.
__device__ __forceinline__ float activate(float z, int act)
{
    switch (act) {
    case RFX_ACT_RELU: return z <= 0.0f ? 0.0f : z; // NaN stays NaN
    case RFX_ACT_SILU: return z / (1.0f + expf(-z));
    case RFX_ACT_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);
    case RFX_ACT_GELU_TANH: return z / (1.0f + expf(-1.5957691216057308f * (z + 0.044715f * z * z * z)));
    }
    return z;
}

// The epilogue of output (column j, row n of N).
__device__ __forceinline__ float finish(const EpiArgs &e, float acc, size_t j, int n, int N)
{
    if (e.bias)
        acc += e.bias[n];
    acc = activate(acc, e.act);
    if (e.resid)
        acc += e.resid[j * N + n];
    return acc;
}

} // namespace dev

// rfx_gemv's launch with the epilogue (rfx_gemv.hip); arguments checked.
int gemv_epi(const rfx_qmat *W, const int8_t *xq, const float *xs, const int32_t *xsum, int q, const EpiArgs &e,
             float *y, void *ws, hipStream_t st);

} // namespace rfx
