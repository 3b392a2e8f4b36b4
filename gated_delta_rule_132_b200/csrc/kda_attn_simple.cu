// kda_attn_simple.cu — prompt attention and its gradients, one warp per row.
#include "kda_attn_rows.cuh"

namespace kda {
namespace {

constexpr int kRows = 64;
constexpr int kThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
rows_fwd_kernel(AttnProblem p, const AttnTile *tiles, T *o, float *lse)
{
    const AttnTile t = tiles[blockIdx.x / p.Hq];
    const int h = blockIdx.x % p.Hq;
    const int end = min(t.first + kRows, t.seq_end);
    for (int r = t.first + (threadIdx.x >> 5); r < end; r += kThreads / 32)
        attn_row_fwd<T, D>(p, r, t.seq_start, h, o, lse);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
rows_bwd_kernel(AttnProblem p, const AttnTile *tiles, const float *lse, const float *delta,
                const T *dO, T *gq, T *gk, T *gv)
{
    const int heads = p.Hq + p.Hkv;
    const AttnTile t = tiles[blockIdx.x / heads];
    const int h = blockIdx.x % heads;
    const int end = min(t.first + kRows, t.seq_end);
    for (int r = t.first + (threadIdx.x >> 5); r < end; r += kThreads / 32) {
        if (h < p.Hq)
            attn_row_dq<T, D>(p, r, t.seq_start, h, lse, delta, dO, gq);
        else
            attn_row_dkv<T, D>(p, r, t.seq_end, h - p.Hq, lse, delta, dO, gk, gv);
    }
}

template <typename T, int D>
cudaError_t fwd(const AttnProblem &p, void *o, float *lse, void *workspace, cudaStream_t st)
{
    const AttnWorkspace w = attn_workspace_layout(p, kRows, false);
    const AttnTile *tiles =
        reinterpret_cast<const AttnTile *>(static_cast<char *>(workspace) + w.tiles);
    cudaError_t e = launch_attn_plan(p, kRows, workspace, st);
    if (e != cudaSuccess) return e;
    rows_fwd_kernel<T, D><<<(unsigned)(attn_tiles(p, kRows) * p.Hq), kThreads, 0, st>>>(
        p, tiles, static_cast<T *>(o), lse);
    note_launch();
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t bwd(const AttnProblem &p, const void *o, const float *lse, const void *dO, void *gq,
                void *gk, void *gv, void *workspace, cudaStream_t st)
{
    const AttnWorkspace w = attn_workspace_layout(p, kRows, true);
    char *ws = static_cast<char *>(workspace);
    const AttnTile *tiles = reinterpret_cast<const AttnTile *>(ws + w.tiles);
    float *delta = reinterpret_cast<float *>(ws + w.delta);
    cudaError_t e = launch_attn_plan(p, kRows, workspace, st);
    if (e != cudaSuccess) return e;
    e = launch_attn_delta(p, o, lse, dO, delta, delta + (size_t)p.tokens * p.Hq, st);
    if (e != cudaSuccess) return e;
    rows_bwd_kernel<T, D>
        <<<(unsigned)(attn_tiles(p, kRows) * (p.Hq + p.Hkv)), kThreads, 0, st>>>(
            p, tiles, lse, delta, static_cast<const T *>(dO), static_cast<T *>(gq),
            static_cast<T *>(gk), static_cast<T *>(gv));
    note_launch();
    return cudaGetLastError();
}

}  // namespace

int attn_fwd_rows(const AttnProblem &p)
{
    return p.dtype == KDA_DTYPE_BF16 ? attn_tc_fwd_rows() : kRows;
}
int attn_bwd_rows(const AttnProblem &p)
{
    return p.dtype == KDA_DTYPE_BF16 ? attn_tc_bwd_rows() : kRows;
}

cudaError_t launch_attn_fwd(const AttnProblem &p, void *o, float *lse, void *ws, cudaStream_t st)
{
    if (p.dtype == KDA_DTYPE_BF16) return launch_attn_tc_fwd(p, o, lse, ws, st);
    if (p.d == 32) return fwd<float, 32>(p, o, lse, ws, st);
    if (p.d == 64) return fwd<float, 64>(p, o, lse, ws, st);
    return fwd<float, 128>(p, o, lse, ws, st);
}

cudaError_t launch_attn_bwd(const AttnProblem &p, const void *o, const float *lse, const void *dO,
                            void *gq, void *gk, void *gv, void *ws, cudaStream_t st)
{
    if (p.dtype == KDA_DTYPE_BF16)
        return launch_attn_tc_bwd(p, o, lse, dO, gq, gk, gv, ws, st);
    if (p.d == 32) return bwd<float, 32>(p, o, lse, dO, gq, gk, gv, ws, st);
    if (p.d == 64) return bwd<float, 64>(p, o, lse, dO, gq, gk, gv, ws, st);
    return bwd<float, 128>(p, o, lse, dO, gq, gk, gv, ws, st);
}

}  // namespace kda
