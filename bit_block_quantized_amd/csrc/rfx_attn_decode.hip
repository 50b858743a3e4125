// Attention of few new tokens per sequence (rfx_attn_decode.h): the kernels and
// their launches.
#include "rfx_attn_decode.h"

using namespace rfx;
using namespace rfx::dev;

namespace {

using namespace rfx::dev::decode;

template <class T, int DP, int NR, Pages PG, class Args>
__global__ __launch_bounds__(64 * kWaves) void attn_decode_kernel(Args args)
{
    __shared__ __align__(16) char smem[lds_bytes<DP>()];
    __shared__ float s_m[kWaves][NR * 16], s_l[kWaves][NR * 16];
    attention<T, DP, NR, PG>(args, blockIdx.x, smem, s_m, s_l);
}

unsigned blocks(const AttnArgs &a) { return (unsigned)a.kv.n_seq * a.kv.Hk * a.S; }
unsigned blocks(const SharedArgs &a) { return a.group_blocks + blocks(a.own); }
const KvArgs &cache_of(const AttnArgs &a) { return a.kv; }
const KvArgs &cache_of(const SharedArgs &a) { return a.own.kv; }

template <class T, int DP, int NR, class Args>
int launch(const Args &a, hipStream_t st)
{
    const KvArgs &kv = cache_of(a);
    const dim3 grid(blocks(a)), block(64 * kWaves);
    if (kv.D != DP || kv.page_shift < 4)
        hipLaunchKernelGGL((attn_decode_kernel<T, DP, NR, kAny, Args>), grid, block, 0, st, a);
    else if (kv.page_shift == 4)
        hipLaunchKernelGGL((attn_decode_kernel<T, DP, NR, kTwo, Args>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((attn_decode_kernel<T, DP, NR, kOne, Args>), grid, block, 0, st, a);
    return hip_status("attn decode launch");
}

template <class T, class Args>
int launch_dim(const Args &a, int row_tiles, hipStream_t st)
{
    const int D = cache_of(a).D;
    if (row_tiles == 1)
        return D <= 64 ? launch<T, 64, 1>(a, st) : D <= 128 ? launch<T, 128, 1>(a, st) : launch<T, 256, 1>(a, st);
    return D <= 64 ? launch<T, 64, 2>(a, st) : launch<T, 128, 2>(a, st);
}

} // namespace

namespace rfx {

int attn_decode_launch(const AttnArgs &a, int type, int row_tiles, hipStream_t st)
{
    return type == RFX_BF16 ? launch_dim<BF16>(a, row_tiles, st) : launch_dim<F16>(a, row_tiles, st);
}

int attn_decode_launch(const SharedArgs &a, int type, int row_tiles, hipStream_t st)
{
    return type == RFX_BF16 ? launch_dim<BF16>(a, row_tiles, st) : launch_dim<F16>(a, row_tiles, st);
}

} // namespace rfx
