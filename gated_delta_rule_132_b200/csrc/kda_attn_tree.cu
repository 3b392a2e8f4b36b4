// kda_attn_tree.cu — attention of a tree of drafted tokens over a paged cache, one
// warp per (sequence, token, head).
#include "kda_attn_rows.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

// The drafted tokens that token i attends to, as bits: itself and its ancestors; 0
// where it, or one of them, has a parent that is neither -1 nor an earlier token.
__device__ __forceinline__ unsigned long long ancestors(const int32_t *parents, int i)
{
    if (!parents) return (2ull << i) - 1;  // a chain
    unsigned long long seen = 0;
    int j = i;
    while (j >= 0) {
        seen |= 1ull << j;
        const int up = parents[j];
        if (up < -1 || up >= j) return 0;
        j = up;
    }
    return seen;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) tree_rows_kernel(TreeProblem p)
{
    constexpr int V = D / 32;
    const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (unit >= (long long)p.N * p.R * p.Hq) return;
    const int h = (int)(unit % p.Hq), i = (int)(unit / p.Hq % p.R), n = (int)(unit / p.Hq / p.R);
    const int hk = h / (p.Hq / p.Hkv), page = 1 << p.page_shift;
    const int32_t *row = p.table + (size_t)n * p.M;
    const int limit = p.M << p.page_shift;
    const int ctx = min(max(p.ctx_lens[n], 0), limit);
    const unsigned long long seen = ancestors(p.parents ? p.parents + (size_t)n * p.R : nullptr, i);
    float q[V], x[V], y[V];
    load_row<T, D>(static_cast<const T *>(p.q) + (size_t)unit * D, q);
    RowSoftmax<V> sm;
    bool any = false;
    const int end = seen ? min(ctx + p.R, limit) : 0;
    for (int c = 0; c < end; ++c) {
        if (c >= ctx && !(seen >> (c - ctx) & 1)) continue;
        const int id = row[c >> p.page_shift];
        if (id < 0 || id >= p.P) continue;
        const size_t at = (((size_t)id * p.Hkv + hk) * page + (c & (page - 1))) * D;
        load_row<T, D>(static_cast<const T *>(p.k_pages) + at, x);
        load_row<T, D>(static_cast<const T *>(p.v_pages) + at, y);
        sm.add(row_dot(q, x) * p.scale, y);
        any = true;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = any ? sm.acc[e] / sm.l : 0.f;
    store_row<T, D>(static_cast<T *>(p.o) + (size_t)unit * D, y);
    if (p.lse && (threadIdx.x & 31) == 0) p.lse[unit] = any ? sm.m + logf(sm.l) : -INFINITY;
}

template <typename T, int D>
cudaError_t launch(const TreeProblem &p, cudaStream_t st)
{
    const long long units = (long long)p.N * p.R * p.Hq;
    tree_rows_kernel<T, D><<<(unsigned)((units + 7) / 8), kThreads, 0, st>>>(p);
    note_launch();
    return cudaGetLastError();
}

}  // namespace

size_t tree_workspace_bytes(const TreeProblem &) { return 0; }

cudaError_t launch_attn_tree(const TreeProblem &p, void *, cudaStream_t st)
{
    if (p.dtype == KDA_DTYPE_F32) {
        if (p.d == 32) return launch<float, 32>(p, st);
        if (p.d == 64) return launch<float, 64>(p, st);
        return launch<float, 128>(p, st);
    }
    if (p.d == 32) return launch<__nv_bfloat16, 32>(p, st);
    if (p.d == 64) return launch<__nv_bfloat16, 64>(p, st);
    return launch<__nv_bfloat16, 128>(p, st);
}

}  // namespace kda
