// kda_attn.cuh — declarations shared by the full-attention translation units.
#pragma once

#include "kda_internal.cuh"

namespace kda {

// A prompt-attention call after host-side validation.
struct AttnProblem {
    const void *q, *k, *v;
    const int32_t *cu_seqlens;  // device, or null (uniform sequences of length T)
    int N, B, T, Hq, Hkv, d;
    float scale;
    kda_dtype_t dtype;
    long long tokens;           // B * T
};

// One tile of consecutive tokens of one sequence: the unit of work of the prompt
// kernels, listed by falling place in the sequence (see kda_attn_plan.cu), since later
// tiles see more keys.
struct __align__(16) AttnTile {
    int first;      // packed token of the tile's first row
    int seq_start;  // packed token range of its sequence
    int seq_end;
    int unused;
};

// Most tiles of `rows` tokens that the sequences can have.
inline long long attn_tiles(const AttnProblem &p, int rows)
{
    return p.cu_seqlens ? p.tokens / rows + p.N
                        : (long long)p.B * ((p.T + rows - 1) / rows);
}

// Workspace of a prompt call: the header (status word), the plan (varlen calls:
// sanitised starts, longest-first order, tile offsets; the tile list) and, for the
// backward, per query head and token D_r = <dO_r, o_r> and then lse_r log2 e.
struct AttnWorkspace {
    size_t starts, order, tiles, delta, total;
};

inline AttnWorkspace attn_workspace_layout(const AttnProblem &p, int rows, bool bwd)
{
    AttnWorkspace w;
    size_t at = kWsHeader;
    w.starts = at; at += sizeof(int32_t) * ((size_t)p.N + 1);
    w.order = at; at += sizeof(int32_t) * 2 * ((size_t)p.N + 1);
    at = align_up(at, 16);
    w.tiles = at; at += sizeof(AttnTile) * (size_t)attn_tiles(p, rows);
    at = align_up(at, 256);
    w.delta = at; if (bwd) at += 2 * sizeof(float) * (size_t)p.tokens * p.Hq;
    w.total = align_up(at, 256);
    return w;
}

// Clears the status word and lists the tiles (the list's unused end gets empty
// sequences).
cudaError_t launch_attn_plan(const AttnProblem &p, int rows, void *workspace, cudaStream_t st);

int attn_fwd_rows(const AttnProblem &p);  // tokens per tile of the path that serves p
int attn_bwd_rows(const AttnProblem &p);
cudaError_t launch_attn_fwd(const AttnProblem &p, void *o, float *lse, void *workspace,
                            cudaStream_t st);
cudaError_t launch_attn_bwd(const AttnProblem &p, const void *o, const float *lse,
                            const void *dO, void *gq, void *gk, void *gv, void *workspace,
                            cudaStream_t st);

// The tensor-core path (bf16).
int attn_tc_fwd_rows(const AttnProblem &p);
int attn_tc_bwd_rows();
cudaError_t launch_attn_tc_fwd(const AttnProblem &p, void *o, float *lse, void *workspace,
                               cudaStream_t st);
cudaError_t launch_attn_tc_bwd(const AttnProblem &p, const void *o, const float *lse,
                               const void *dO, void *gq, void *gk, void *gv, void *workspace,
                               cudaStream_t st);
// D_r = <dO_r, o_r> and lse_r log2 e of every token and query head.
cudaError_t launch_attn_delta(const AttnProblem &p, const void *o, const float *lse,
                              const void *dO, float *delta, float *lse2, cudaStream_t st);

// dK and dV of a key tile can be shared out over a cluster of CTAs, each with some of the
// group's query heads; the partial sums are added in rank order through distributed
// shared memory. That pays where the key tiles alone make too few CTAs (below `enough`):
// one per SM on the tensor cores, whose CTAs take an SM each and some 10 us to begin and to
// be joined (nine packed documents, 272 CTAs: 110 us, split in two 130 us), four per SM
// in fp32 (B = 2, T = 777, 8/4 heads of 64, 200 CTAs: 180 us, split in two 122 us).
inline int attn_head_split(const AttnProblem &p, int rows, int enough)
{
    const long long ctas = attn_tiles(p, rows) * p.Hkv;
    int split = 1;
    while (split < 4 && split * 2 <= p.Hq / p.Hkv && ctas * split < enough) split *= 2;
    return split;
}

// A launch as clusters of `split` CTAs (1: none). `early`: its CTAs may start while those of
// the kernel before it, which allows it, still run; it waits for that kernel's end itself.
template <typename K, typename P>
cudaError_t launch_kernel(K kernel, const P &params, long long ctas, int threads, size_t smem,
                          int split, bool early, cudaStream_t st)
{
    if (ctas * split > INT32_MAX) return cudaErrorInvalidValue;
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr[2] = {};
    int attrs = 0;
    if (split > 1) {
        attr[attrs].id = cudaLaunchAttributeClusterDimension;
        attr[attrs].val.clusterDim.x = (unsigned)split;
        attr[attrs].val.clusterDim.y = attr[attrs].val.clusterDim.z = 1;
        ++attrs;
    }
    if (early) {
        attr[attrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[attrs].val.programmaticStreamSerializationAllowed = 1;
        ++attrs;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(ctas * split));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = (unsigned)attrs;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, params);
    note_launch();
    return e;
}

// The kernel launched early behind this one may start; this kernel waits for the end of
// the one before it and sees what that wrote.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ int cluster_rank()
{
    int r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// All threads of all CTAs of the cluster; orders their shared-memory accesses.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The float at this CTA's shared address `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ float peer_float(uint32_t addr, int rank)
{
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
                 "ld.shared::cluster.f32 %0, [a];\n\t}" : "=f"(v) : "r"(addr), "r"(rank) : "memory");
    return v;
}

// A tree-attention call after host-side validation.
struct TreeProblem {
    const void *q, *k_pages, *v_pages;
    const int32_t *table, *ctx_lens, *parents;
    int N, R, Hq, Hkv, d, P, M, page_shift;
    float scale;
    kda_dtype_t dtype;
    void *o;
    float *lse;
};
size_t tree_workspace_bytes(const TreeProblem &p);
cudaError_t launch_attn_tree(const TreeProblem &p, void *workspace, cudaStream_t st);

// Launches of the cache's page calls (kda_cache.cu); sizes are validated.
struct PagePool {
    void *k, *v;
    int P, Hkv, d, page_shift, elem;  // elem: bytes per element
};
cudaError_t launch_cache_fork(int32_t *refs, const int32_t *table, const int32_t *lens,
                              const int32_t *parents, int N_in, int N_out, int M, int P,
                              int32_t *new_table, int32_t *new_lens, cudaStream_t st);
cudaError_t launch_cache_reserve(int32_t *refs, int32_t *table, int32_t *lens,
                                 const int32_t *add, int N, int M, int P, int page_shift,
                                 int32_t *copies, int32_t *status, void *workspace,
                                 cudaStream_t st);
cudaError_t launch_cache_release(int32_t *refs, int32_t *table, int32_t *lens,
                                 const int32_t *new_lens, int N, int M, int P, int page_shift,
                                 cudaStream_t st);
cudaError_t launch_cache_append(const PagePool &pool, const int32_t *table, const int32_t *start,
                                const void *k_new, const void *v_new, const int32_t *cu_seqlens,
                                int N, int B, int T, int M, cudaStream_t st);
cudaError_t launch_cache_compact(const PagePool &pool, const int32_t *table,
                                 const int32_t *ctx_lens, const int32_t *path, int N, int R,
                                 int M, int32_t *new_lens, cudaStream_t st);
cudaError_t launch_cache_copy(const PagePool &pool, const int32_t *copies, int C,
                              cudaStream_t st);

}  // namespace kda
