// attn_fwd_host.cpp — the prompt forward's source on the emulated device.
#include "attn_host.h"

#include "kda_attn_fwd.cu"

// Returns the status word, or -1 for an error of the host side.
extern "C" int attn_fwd_host_run(const void *q, const void *k, const void *v, const int *cu, int N, int B, int T,
                                 int Hq, int Hkv, int d, float scale, void *o, float *lse, void *ws, int ctas,
                                 unsigned seed)
{
    const kda::AttnProblem p = problem(q, k, v, cu, N, B, T, Hq, Hkv, d, scale, ctas, seed);
    if (kda::launch_attn_tc_fwd(p, o, lse, ws, nullptr) != cudaSuccess) return -1;
    return *static_cast<int *>(ws);
}
