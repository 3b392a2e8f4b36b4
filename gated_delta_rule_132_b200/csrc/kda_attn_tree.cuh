// kda_attn_tree.cuh — what the kernels of tree attention share: the problem, a CTA's
// share of it, which drafts a token sees, and how a row is finished.
#pragma once

#include "kda_attn_rows.cuh"
#include "kda_attn_tc.cuh"

namespace kda {

constexpr float kTreeLog2e = 1.44269504088896340736f;
constexpr float kTreeLn2 = 0.693147180559945309417f;

// The drafted tokens that token i attends to, as bits: itself and its ancestors; 0
// where it, or one of them, has a parent that is neither -1 nor an earlier token.
__device__ __forceinline__ unsigned long long ancestors(const int32_t *parents, int i)
{
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

struct TreeParams {
    TreeProblem p;
    int rows;       // R * G
    int tile_rows;  // of them per CTA
    int row_tiles;  // CTAs that share a chunk's keys
    int tile_keys;  // chunks are multiples of this
    int chunks;     // most chunks of a sequence
    float share, per_round;  // (kv heads x row tiles) / places, the CTAs that run at a time; and 1 /
                             // the rounds of them that a long call should have
    int least_keys, most_keys;  // of a chunk in more rounds than one, and of any
    float *part_o;  // [n, hk, chunk, row, D]: sums over e^(s - m) v
    float2 *part_ml;
    // bf16: the pools as rows of a head's channels, q as tokens of a kv head's G heads
    // (tensor-core path for many rows), and where the waits report
    CUtensorMap k, v, q;
    int pool_rows;
    int *status;
    uint32_t spin;
    int starve;
};

// Where key `pos` of a row of the table is, in elements; -1 where it has no page.
__device__ __forceinline__ long long key_at(const TreeProblem &p, const int32_t *row, int pos,
                                            int hk)
{
    const int id = __ldg(row + (pos >> p.page_shift));
    if ((unsigned)id >= (unsigned)p.P) return -1;
    return (((((long long)id * p.Hkv + hk) << p.page_shift) + (pos & ((1 << p.page_shift) - 1)))) * p.d;
}

__device__ __forceinline__ int ctx_of(const TreeProblem &p, int n)
{
    return min(max(p.ctx_lens[n], 0), p.M << p.page_shift);
}

__device__ __forceinline__ int end_of(const TreeProblem &p, int n)
{
    return min(ctx_of(p, n) + p.R, p.M << p.page_shift);
}

// Keys per chunk of sequence n, and its length. Lengths are known on the device only, so
// every warp adds them up (so a sequence's split, and with it its rounding, depends on the
// others of its batch): chunks are to give one CTA to every place and not more, and of long
// calls up to 1 / f.per_round to a place, as long as they keep f.least_keys; no smaller than a
// tile and no larger than f.most_keys. In fp32, whose divisions are quick: most CTAs of a
// short call find here that they have no chunk.
__device__ __forceinline__ int chunk_of(const TreeParams &f, int n, int &end)
{
    constexpr int kCounted = 1024;  // sequences whose lengths are added up
    int ctx = f.p.ctx_lens[n];
    const int lane = threadIdx.x & 31, most = f.p.M << f.p.page_shift;
    float total = 0.f;
    if (f.chunks > 1 && f.p.N <= kCounted) {
        for (int i = lane; i < f.p.N; i += 32) total += (float)end_of(f.p, i);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    }
    ctx = min(max(ctx, 0), most);
    end = min(ctx + f.p.R, most);
    if (f.chunks == 1) return INT32_MAX;
    float target = 2048.f;
    bool once = false;  // one CTA to a place
    if (f.p.N <= kCounted) {
        const float one = total * f.share, least = (float)f.least_keys;
        once = one <= least;
        target = fmaxf(one * f.per_round, fminf(one, least));
        target = fminf(fmaxf(target, (float)f.tile_keys), (float)f.most_keys);
    }
    const float parts = __fdividef((float)end, target);
    const int count = max(1, min(f.chunks, (int)(once ? parts : ceilf(parts))));
    return ((end + count - 1) / count + f.tile_keys - 1) / f.tile_keys * f.tile_keys;
}

// One row from the keys it sees alone: one warp.
template <typename T, int D>
__device__ __noinline__ void tree_row(const TreeProblem &p, int n, int i, int h)
{
    constexpr int V = D / 32;
    const int32_t *row = p.table + (size_t)n * p.M;
    const int ctx = ctx_of(p, n), end = end_of(p, n);
    const unsigned long long seen =
        p.parents ? ancestors(p.parents + (size_t)n * p.R, i) : (2ull << i) - 1;
    const size_t unit = ((size_t)n * p.R + i) * p.Hq + h;
    const int hk = h / (p.Hq / p.Hkv);
    float q[V], x[V], y[V];
    load_row<T, D>(static_cast<const T *>(p.q) + unit * D, q);
    RowSoftmax<V> sm;
    bool any = false;
    for (int c = 0; c < (seen ? end : 0); ++c) {
        if (c >= ctx && !(seen >> (c - ctx) & 1)) continue;
        const long long at = key_at(p, row, c, hk);
        if (at < 0) continue;
        load_row<T, D>(static_cast<const T *>(p.k_pages) + at, x);
        load_row<T, D>(static_cast<const T *>(p.v_pages) + at, y);
        sm.add(row_dot(q, x) * p.scale, y);
        any = true;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = any ? sm.acc[e] / sm.l : 0.f;
    store_row<T, D>(static_cast<T *>(p.o) + unit * D, y);
    if (p.lse && (threadIdx.x & 31) == 0) p.lse[unit] = any ? sm.m + logf(sm.l) : -INFINITY;
}

// What a warp does with a row's finished sums (lane l: elements from l * D / 32 on, the
// maximum m in log2 units, the sum l): the result, or the row again from its keys.
template <typename T, int D>
__device__ __forceinline__ void finish_row(const TreeProblem &p, int n, int i, int h, float m,
                                           float l, bool absent, const float (&acc)[D / 32])
{
    const size_t unit = ((size_t)n * p.R + i) * p.Hq + h;
    const bool none = absent || (m == -INFINITY && l == 0.f);
    float y[D / 32], odd = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
        y[e] = none ? 0.f : acc[e] / l;
        odd = fmaf(y[e], 0.f, odd);
    }
    if (__any_sync(0xffffffffu, !(odd == 0.f))) {
        tree_row<T, D>(p, n, i, h);
        return;
    }
    store_row<T, D>(static_cast<T *>(p.o) + unit * D, y);
    if (p.lse && (threadIdx.x & 31) == 0) p.lse[unit] = none ? -INFINITY : m * kTreeLn2 + logf(l);
}

__device__ __forceinline__ void cp_async16_or_zero(void *dst, const void *src, bool real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"(tc::smem_u32(dst)), "l"(src), "r"(real ? 16 : 0) : "memory");
}

// What both forms of the kernel know about their share.
struct Share {
    int n, hk, chunk, row0, ctx, first, last;  // keys [first, last)
    const int32_t *table;
    bool alone;  // the sequence's only chunk
};

__device__ __forceinline__ bool share_of(const TreeParams &f, Share &s)
{
    int x = blockIdx.x;  // the chunks that most sequences do not have come last
    s.row0 = x % f.row_tiles * f.tile_rows; x /= f.row_tiles;
    s.hk = x % f.p.Hkv; x /= f.p.Hkv;
    s.n = x % f.p.N;
    s.chunk = x / f.p.N;
    int end;
    const int chunk = chunk_of(f, s.n, end);
    s.ctx = ctx_of(f.p, s.n);
    s.alone = end <= chunk;
    if (s.chunk && (s.alone || (long long)s.chunk * chunk >= end)) return false;
    s.first = s.chunk ? s.chunk * chunk : 0;
    s.last = s.alone ? end : min(s.first + chunk, end);
    s.table = f.p.table + (size_t)s.n * f.p.M;
    return true;  // an empty sequence's rows are still written
}

// The drafts that every drafted token sees, by the CTA's first S::kMaskThreads threads
// (they meet in barrier 1).
template <typename S>
__device__ __forceinline__ const unsigned long long *tree_masks(const TreeParams &f, int n, char *smem)
{
    unsigned long long *seen = reinterpret_cast<unsigned long long *>(smem + S::kSeen);
    int32_t *parents = reinterpret_cast<int32_t *>(smem + S::kParents);
    const int i = threadIdx.x;
    if (i < f.p.R) {
        parents[i] = f.p.parents ? f.p.parents[(size_t)n * f.p.R + i] : -1;
        if (!f.p.parents) seen[i] = (2ull << i) - 1;  // a chain
    }
    asm volatile("bar.sync 1, %0;" ::"n"(S::kMaskThreads) : "memory");
    if (f.p.parents && i < f.p.R) seen[i] = ancestors(parents, i);
    asm volatile("bar.sync 1, %0;" ::"n"(S::kMaskThreads) : "memory");
    return seen;
}

// The pages of a tile of kKeys keys, as a loading warp sees them (pages of at least eight
// tokens): a box per page, or one where a page covers the tile; lane b < boxes has box b.
template <int kKeys> struct Boxes {
    int shift;  // log2 of a box's keys
    __device__ __forceinline__ explicit Boxes(const TreeParams &f)
        : shift(min(f.p.page_shift, kKeys == 64 ? 6 : 7)) {}
    __device__ __forceinline__ int count() const { return kKeys >> shift; }
    __device__ __forceinline__ int key() const { return (threadIdx.x & 31) << shift; }  // the box's first

    // This lane's page of the tile at pos: a table entry, read well before it is used.
    __device__ __forceinline__ int page(const TreeParams &f, const Share &s, int pos) const
    {
        const int c = pos + key();
        return key() < kKeys && c < s.last ? __ldg(s.table + (c >> f.p.page_shift)) : -1;
    }
    // Its box's first row of the pool; behind the pool (reads zero) where there is no page.
    __device__ __forceinline__ int row(const TreeParams &f, const Share &s, int pos, int page) const
    {
        if ((unsigned)page >= (unsigned)f.p.P) return f.pool_rows;
        return ((page * f.p.Hkv + s.hk) << f.p.page_shift) +
               ((pos + key()) & ((1 << f.p.page_shift) - 1));
    }
    // Bit l: key 32 e + l of the tile is the sequence's and has a page.
    __device__ __forceinline__ uint32_t there(const TreeParams &f, const Share &s, int pos, int row,
                                              int e) const
    {
        const int key = 32 * e + (threadIdx.x & 31);
        const int of = __shfl_sync(0xffffffffu, row, key >> shift);
        return __ballot_sync(0xffffffffu, of < f.pool_rows && pos + key < s.last);
    }
};

// The tensor-core kernel for many rows (kda_attn_tree_tc.cu).
int tree_tc_rows(const TreeProblem &p);  // rows per CTA; 0: it does not serve this problem
cudaError_t launch_tree_tc(const TreeParams &f, long long ctas, cudaStream_t st);

}  // namespace kda
