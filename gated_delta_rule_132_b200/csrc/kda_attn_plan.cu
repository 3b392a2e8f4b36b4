// kda_attn_plan.cu — the tile list of the prompt-attention kernels.
//
// cu_seqlens lives in device memory, so it is sanitised here as the prefill's plan
// does it: offsets clamped to [0, tokens] and made non-decreasing.
//
// A tile's work grows with its place in its sequence, and persistent CTAs take the list's
// entries in turn: so it is sorted by falling place. Sequences are ranked by decreasing
// length first; those that have a tile at place t are then the first ones, and an entry's
// position is the number of tiles at later places plus its sequence's rank. The ranking
// is quadratic: beyond kRankMax sequences they keep their order, last tile first in each.
#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int kThreads = 1024;
constexpr int kRankMax = 2048;

// Inclusive scan over the block; s_warp holds one value per warp.
template <bool kMax>
__device__ int block_scan(int x, int *s_warp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto op = [](int a, int b) { return kMax ? max(a, b) : a + b; };
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x = op(x, y);
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = s_warp[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) w = op(w, y);
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    if (warp > 0) x = op(x, s_warp[warp - 1]);
    __syncthreads();
    return x;
}

__global__ void __launch_bounds__(kThreads)
attn_plan_kernel(const int32_t *__restrict__ cu, int N, int T, int tokens, int rows, int max_tiles,
                 int *status, int32_t *starts, int32_t *order, int32_t *offs, AttnTile *tiles)
{
    __shared__ int s_warp[32];
    __shared__ int s_carry;
    __shared__ int s_len[kRankMax], s_tiles[kRankMax];
    const int tid = threadIdx.x;
    let_next_start();
    if (tid == 0) *status = 0;
    // sanitised starts
    if (tid == 0) s_carry = 0;
    __syncthreads();
    for (int base = 0; base <= N; base += kThreads) {
        const int n = base + tid;
        int x = 0;
        if (n <= N) x = cu ? min(max(cu[n], 0), tokens) : n * T;
        x = block_scan<true>(max(x, s_carry), s_warp);
        if (n <= N) starts[n] = x;
        if (tid == kThreads - 1) s_carry = x;
        __syncthreads();
    }
    if (N <= kRankMax) {
        // longest first, ties by index
        for (int n = tid; n < N; n += kThreads) s_len[n] = starts[n + 1] - starts[n];
        __syncthreads();
        for (int n = tid; n < N; n += kThreads) {
            const int ln = s_len[n];
            int rank = 0;
            for (int m = 0; m < N; ++m) rank += s_len[m] > ln || (s_len[m] == ln && m < n);
            order[rank] = n;
            s_tiles[rank] = (ln + rows - 1) / rows;
        }
        __syncthreads();
        const int lane = tid & 31;
        if (tid == 0) s_carry = 0;
        __syncthreads();
        for (int t = tid >> 5; t < s_tiles[0]; t += kThreads / 32) {
            int later = 0, here = 0;
            for (int r = lane; r < N && s_tiles[r] > t; r += 32) {
                later += s_tiles[r] - t - 1;
                ++here;
            }
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) {
                later += __shfl_xor_sync(0xffffffffu, later, d);
                here += __shfl_xor_sync(0xffffffffu, here, d);
            }
            for (int r = lane; r < here; r += 32) {
                const int n = order[r], a = starts[n];
                tiles[later + r] = AttnTile{a + t * rows, a, starts[n + 1], 0};
            }
            if (lane == 0) atomicAdd(&s_carry, here);
        }
        __syncthreads();
        for (int t = s_carry + tid; t < max_tiles; t += kThreads) tiles[t] = AttnTile{0, 0, 0, 0};
        return;
    }
    for (int n = tid; n < N; n += kThreads) order[n] = n;
    __syncthreads();
    // first tile of each rank
    if (tid == 0) s_carry = 0;
    __syncthreads();
    for (int base = 0; base < N; base += kThreads) {
        const int r = base + tid;
        int c = 0;
        if (r < N) c = (starts[order[r] + 1] - starts[order[r]] + rows - 1) / rows;
        const int incl = block_scan<false>(c, s_warp);
        const int carry = s_carry;
        if (r < N) offs[r] = carry + incl - c;
        __syncthreads();
        if (tid == kThreads - 1) s_carry = carry + incl;
        __syncthreads();
    }
    const int used = s_carry;
    // the list: one warp per sequence
    for (int r = tid >> 5; r < N; r += kThreads / 32) {
        const int n = order[r], a = starts[n], b = starts[n + 1];
        const int count = (b - a + rows - 1) / rows;
        for (int t = tid & 31; t < count; t += 32)
            tiles[offs[r] + t] = AttnTile{a + (count - 1 - t) * rows, a, b, 0};
    }
    for (int t = used + tid; t < max_tiles; t += kThreads) tiles[t] = AttnTile{0, 0, 0, 0};
}

}  // namespace

cudaError_t launch_attn_plan(const AttnProblem &p, int rows, void *workspace, cudaStream_t st)
{
    const AttnWorkspace w = attn_workspace_layout(p, rows, false);
    char *ws = static_cast<char *>(workspace);
    int32_t *order = reinterpret_cast<int32_t *>(ws + w.order);
    attn_plan_kernel<<<1, kThreads, 0, st>>>(
        p.cu_seqlens, p.N, p.T, (int)p.tokens, rows, (int)attn_tiles(p, rows),
        reinterpret_cast<int *>(ws), reinterpret_cast<int32_t *>(ws + w.starts), order,
        order + p.N + 1, reinterpret_cast<AttnTile *>(ws + w.tiles));
    note_launch();
    return cudaGetLastError();
}

}  // namespace kda
