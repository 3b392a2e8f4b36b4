// attn_tree_host.cpp — tree attention's host side, plan and join on the emulated device; calls of
// many rows run on it as a whole (attn_tree_tc_host.cpp has their kernel).
#define FEW_ROWS
#include "attn_host.h"

#include "kda_attn_tree.cu"

// Returns the status word, -1 for an error of the host side, -2 for a call of few rows.
extern "C" int attn_tree_host_run(const void *q, const void *k, const void *v, const int *table, const int *ctx,
                                  const int *parents, int N, int R, int Hq, int Hkv, int d, int P, int M, int shift,
                                  float scale, void *o, float *lse, void *ws, unsigned long long bytes, unsigned seed)
{
    kda::TreeProblem p{};
    p.q = q; p.k_pages = k; p.v_pages = v; p.table = table; p.ctx_lens = ctx; p.parents = parents;
    p.N = N; p.R = R; p.Hq = Hq; p.Hkv = Hkv; p.d = d; p.P = P; p.M = M; p.page_shift = shift;
    p.scale = scale; p.dtype = KDA_DTYPE_BF16; p.o = o; p.lse = lse;
    emu::seed = seed;
    emu::ctas = 0;
    if (!kda::many_rows(p)) return -2;
    if (kda::tree_workspace_bytes(p) > bytes || kda::launch_attn_tree(p, ws, nullptr) != cudaSuccess) return -1;
    return *static_cast<int *>(ws);
}
