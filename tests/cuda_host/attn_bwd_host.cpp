// attn_bwd_host.cpp — the prompt gradients' source on the emulated device.
#include "attn_host.h"

namespace kda {
bool encode_attn_map(CUtensorMap *tm, const void *base, int H, int D, long long tokens)
{
    const tc::Map m{static_cast<const uint16_t *>(base), (uint64_t)D, (uint64_t)H, (uint64_t)tokens};
    std::memcpy(tm, &m, sizeof m);
    return true;
}
}
#include "kda_attn_bwd.cu"

// Returns the status word, or -1 for an error of the host side.
extern "C" int attn_bwd_host_run(const void *q, const void *k, const void *v, const void *o, const float *lse,
                                 const void *dO, const int *cu, int N, int B, int T, int Hq, int Hkv, int d,
                                 float scale, void *gq, void *gk, void *gv, void *ws, int ctas, unsigned seed)
{
    const kda::AttnProblem p = problem(q, k, v, cu, N, B, T, Hq, Hkv, d, scale, ctas, seed);
    if (kda::launch_attn_tc_bwd(p, o, lse, dO, gq, gk, gv, ws, nullptr) != cudaSuccess) return -1;
    return *static_cast<int *>(ws);
}
