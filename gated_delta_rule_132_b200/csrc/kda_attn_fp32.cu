// kda_attn_fp32.cu — causal prompt attention and its gradients in fp32 (CUDA cores),
// and the choice between this path and the tensor-core path.
//
// A CTA of 128 threads (8 x 16) owns 32 tokens and walks over the 64-token tiles that
// they meet. A product of the two tiles over the channels gives each thread 4 x 4 pairs
// (own rows 4 ty + i, walked rows tx + 16 j), a product of a 32 x 64 weight tile with the
// walked rows 4 rows x D / 16 channels; both read shared memory 16 bytes at a time, from
// swizzled rows. The FMA rate bounds the kernels: per four channels a warp issues 64 FMAs
// (16 cycles of the SM) for 12 cycles of shared memory reads. 32 own tokens rather than
// 64 because calls in fp32 are short: B = 2, T = 777, 8 heads of 64 are 208 tiles of 64,
// one wave whose longest CTA takes 84 us forward, and 400 of 32, which fill the SMs: 71 us,
// forward and backward 230 us. There the busiest SM issues in 61% of its cycles and the
// average one in 42%, for CTAs' lengths differ; of what is issued 64% are FMAs. (Two CTAs to
// an SM instead of three: the forward 66 us, all 240 us.)
//
// The gradients follow the tensor-core path's split: one CTA per key tile for dK and
// dV, one per query tile for dQ, every result written once. Rows that are not finite
// are computed again from what they see (0 times a masked infinity is NaN).
#include "kda_attn_rows.cuh"
#include "tc_primitives.cuh"

namespace kda {
namespace {

constexpr int kRows = 32;  // own tokens
constexpr int kWalk = 64;  // tokens of a walked tile
constexpr int kThreads = 128;
constexpr int kW = 68;  // row length of a weight tile
constexpr float kLog2e = 1.44269504088896340736f;

// Element offset of 4-channel unit u of row r of a tile: units are exchanged within a
// row so that eight consecutive rows' equal units lie in different banks.
template <int D> __device__ __forceinline__ int unit_at(int r, int u)
{
    return r * D + (u ^ (r & 7)) * 4;
}

// Start the copies of kCount tokens of one head from `first` on; tokens from `end` on are
// filled with zeros.
template <int D, int kCount>
__device__ __forceinline__ void load_tile(float *dst, const float *src, int heads, int h,
                                          int first, int end)
{
    constexpr int kUnits = D / 4;
    const int u = threadIdx.x % kUnits;
#pragma unroll
    for (int r = threadIdx.x / kUnits; r < kCount; r += kThreads / kUnits) {
        const bool real = first + r < end;
        const float *from = src + ((size_t)(real ? first + r : first) * heads + h) * D + u * 4;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     ::"r"(tc::smem_u32(dst + unit_at<D>(r, u))), "l"(from), "r"(real ? 16 : 0)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// All but the last N groups of copies have landed, for every thread of the CTA.
template <int N> __device__ __forceinline__ void landed()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
    __syncthreads();
}

// x[i][j] = <row 4 ty + i of a, row tx + 16 j of b>.
template <int D>
__device__ __forceinline__ void dot_tiles(const float *a, const float *b, float (&x)[4][4])
{
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = 0.f;
    }
#pragma unroll 4
    for (int u = 0; u < D / 4; ++u) {
        float4 p[4], q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4 *>(a + unit_at<D>(4 * ty + i, u));
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = *reinterpret_cast<const float4 *>(b + unit_at<D>(tx + 16 * j, u));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[i][j] = fmaf(p[i].x, q[j].x, fmaf(p[i].y, q[j].y, fmaf(p[i].z, q[j].z, fmaf(p[i].w, q[j].w, x[i][j]))));
        }
    }
}

// A thread's channels of a row: groups of kVec from tx * kVec + 16 kVec e on.
template <int D> struct Cols {
    static constexpr int kVec = D >= 64 ? 4 : 2, kGroups = D / 16 / kVec;
    static __device__ __forceinline__ int at(int r, int e)
    {
        const int c = ((threadIdx.x & 15) + 16 * e) * kVec;
        return unit_at<D>(r, c >> 2) + (c & 3);
    }
    static __device__ __forceinline__ int channel(int e) { return ((threadIdx.x & 15) + 16 * e) * kVec; }
};

// acc[i] += sum over 64 tokens r of w(4 ty + i, r) * row r of y.
template <int D>
__device__ __forceinline__ void add_weighted(const float *w, const float *y, float (&acc)[4][D / 16])
{
    using C = Cols<D>;
    const int ty = threadIdx.x >> 4;
#pragma unroll 2
    for (int r = 0; r < kWalk; r += 4) {
        float p[4][4];  // [i][token]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(w + (4 * ty + i) * kW + r);
            p[i][0] = x.x; p[i][1] = x.y; p[i][2] = x.z; p[i][3] = x.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int e = 0; e < C::kGroups; ++e) {
                float v[C::kVec];
                if (C::kVec == 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(y + C::at(r + j, e));
                    v[0] = x.x; v[1] = x.y; v[C::kVec - 2] = x.z; v[C::kVec - 1] = x.w;
                } else {
                    const float2 x = *reinterpret_cast<const float2 *>(y + C::at(r + j, e));
                    v[0] = x.x; v[1] = x.y;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int a = 0; a < C::kVec; ++a)
                        acc[i][e * C::kVec + a] = fmaf(p[i][j], v[a], acc[i][e * C::kVec + a]);
                }
            }
        }
    }
}

__device__ __forceinline__ void store_weights(float *w, const float (&x)[4][4])
{
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[(4 * ty + i) * kW + tx + 16 * j] = x[i][j];
    }
}

// A thread's rows times `by[i]` to out (row 0 of the tile, rows `stride` apart), below
// `rows`; flags rows that are not finite.
template <int D>
__device__ __forceinline__ void store_rows(const float (&acc)[4][D / 16], const float (&by)[4],
                                           float *out, size_t stride, int rows, unsigned *bad)
{
    using C = Cols<D>;
    const int ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * ty + i;
        if (r >= rows) continue;
        float odd = 0.f;
#pragma unroll
        for (int e = 0; e < C::kGroups; ++e) {
            float *to = out + r * stride + C::channel(e);
#pragma unroll
            for (int a = 0; a < C::kVec; ++a) {
                const float v = acc[i][e * C::kVec + a] * by[i];
                odd = fmaf(v, 0.f, odd);
                to[a] = v;
            }
        }
        if (!(odd == 0.f)) atomicOr(bad, 1u << r);
    }
}

// After all stores: the flagged rows again, one warp each.
template <typename F> __device__ __forceinline__ void redo_rows(const unsigned *bad, F redo)
{
    __syncthreads();
    for (int r = threadIdx.x >> 5; r < kRows; r += kThreads / 32)
        if (*bad >> r & 1) redo(r);
}

struct F32Params {
    AttnProblem p;
    const AttnTile *tiles;  // null: uniform sequences
    const float *lse, *lse2, *delta, *dO;
    float *o, *lse_out, *gq, *gk, *gv;
    int *status;  // of the workspace: nothing here can fail, the first CTA clears it
    int split;    // dK and dV: CTAs per key tile, see attn_head_split
};

__device__ __forceinline__ AttnTile tile_of(const F32Params &f, int idx)
{
    if (f.tiles) return f.tiles[idx];
    const int count = (f.p.T + kRows - 1) / kRows, b = idx % f.p.B, t = count - 1 - idx / f.p.B;
    return AttnTile{b * f.p.T + t * kRows, b * f.p.T, (b + 1) * f.p.T, 0};
}

template <int D> __device__ __noinline__ void redo_fwd(const F32Params &f, int row, int start, int h)
{
    attn_row_fwd<float, D>(f.p, row, start, h, f.o, f.lse_out);
}
template <int D> __device__ __noinline__ void redo_dq(const F32Params &f, int row, int start, int h)
{
    attn_row_dq<float, D>(f.p, row, start, h, f.lse, f.delta, f.dO, f.gq);
}
template <int D> __device__ __noinline__ void redo_dkv(const F32Params &f, int col, int end, int hk)
{
    attn_row_dkv<float, D>(f.p, col, end, hk, f.lse, f.delta, f.dO, f.gk, f.gv);
}

// The walked tiles of an own query tile: from the one with its last token down.
__device__ __forceinline__ int last_walked(const AttnTile &t)
{
    return t.seq_start + (t.first - t.seq_start) / kWalk * kWalk;
}

// ---------------------------------------------------------------- forward
template <int D>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const __grid_constant__ F32Params f)
{
    extern __shared__ __align__(16) float smem[];
    __shared__ unsigned bad;
    float *q = smem, *k = q + kRows * D, *v = k + kWalk * D, *w = v + kWalk * D;
    const AttnTile t = tile_of(f, blockIdx.x / f.p.Hq);
    if (t.first >= t.seq_end) return;
    const int h = blockIdx.x % f.p.Hq, hk = h / (f.p.Hq / f.p.Hkv);
    if (!f.tiles && blockIdx.x == 0 && threadIdx.x == 0) *f.status = 0;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const float *gk = static_cast<const float *>(f.p.k), *gv = static_cast<const float *>(f.p.v);
    if (threadIdx.x == 0) bad = 0;
    const int last = last_walked(t);
    load_tile<D, kRows>(q, static_cast<const float *>(f.p.q), f.p.Hq, h, t.first, t.seq_end);
    load_tile<D, kWalk>(k, gk, f.p.Hkv, hk, last, t.seq_end);
    const float c = f.p.scale * kLog2e;
    float m[4], l[4] = {}, acc[4][D / 16] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = -INFINITY;
    for (int at = last; at >= t.seq_start; at -= kWalk) {
        load_tile<D, kWalk>(v, gv, f.p.Hkv, hk, at, t.seq_end);
        landed<1>();
        float x[4][4];
        dot_tiles<D>(q, k, x);
        const int diag = t.first - at;  // keys up to row + diag are seen
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = tx + 16 * j <= 4 * ty + i + diag ? x[i][j] * c : -INFINITY;
                top = fmaxf(top, x[i][j]);
            }
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float ref = top == -INFINITY ? 0.f : top, keep = exp2f(m[i] - ref);
            m[i] = top;
            l[i] *= keep;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = exp2f(x[i][j] - ref);
                l[i] += x[i][j];
            }
#pragma unroll
            for (int e = 0; e < D / 16; ++e) acc[i][e] *= keep;
        }
        store_weights(w, x);
        landed<0>();  // the values, the weights, and k is free
        if (at > t.seq_start) load_tile<D, kWalk>(k, gk, f.p.Hkv, hk, at - kWalk, t.seq_end);
        add_weighted<D>(w, v, acc);
        __syncthreads();
    }
    float by[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
        by[i] = 1.f / l[i];
        const int row = t.first + 4 * ty + i;
        if (f.lse_out && tx == 0 && row < t.seq_end)
            f.lse_out[(size_t)row * f.p.Hq + h] = m[i] * 0.693147180559945309417f + logf(l[i]);
    }
    store_rows<D>(acc, by, f.o + ((size_t)t.first * f.p.Hq + h) * D, (size_t)f.p.Hq * D,
                  t.seq_end - t.first, &bad);
    redo_rows(&bad, [&](int r) { redo_fwd<D>(f, t.first + r, t.seq_start, h); });
}

// lse2 and D of kCount query rows; rows behind the sequence get weights of zero.
template <int kCount>
__device__ __forceinline__ void load_stats(const F32Params &f, float *lse2, float *del, int h,
                                           int first, int end)
{
    if (threadIdx.x < kCount) {
        const int r = first + threadIdx.x;
        const size_t at = (size_t)h * f.p.tokens + r;
        lse2[threadIdx.x] = r < end ? f.lse2[at] : INFINITY;
        del[threadIdx.x] = r < end ? f.delta[at] : 0.f;
    }
}

// ---------------------------------------------------------------- dQ
// Launched early behind dK and dV, of which it needs nothing: it fills the SMs that have
// run out of them, and only must not end before they do.
template <int D>
__global__ void __launch_bounds__(kThreads) dq_kernel(const __grid_constant__ F32Params f)
{
    extern __shared__ __align__(16) float smem[];
    __shared__ float lse2[kRows], del[kRows];
    __shared__ unsigned bad;
    float *q = smem, *g = q + kRows * D, *k = g + kRows * D, *v = k + kWalk * D, *w = v + kWalk * D;
    const AttnTile t = tile_of(f, blockIdx.x / f.p.Hq);
    if (t.first >= t.seq_end) {  // where all sequences are empty no other CTA waits
        wait_for_previous();
        return;
    }
    const int h = blockIdx.x % f.p.Hq, hk = h / (f.p.Hq / f.p.Hkv);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    if (threadIdx.x == 0) bad = 0;
    load_stats<kRows>(f, lse2, del, h, t.first, t.seq_end);
    load_tile<D, kRows>(q, static_cast<const float *>(f.p.q), f.p.Hq, h, t.first, t.seq_end);
    load_tile<D, kRows>(g, f.dO, f.p.Hq, h, t.first, t.seq_end);
    const float c = f.p.scale * kLog2e;
    float acc[4][D / 16] = {};
    for (int at = last_walked(t); at >= t.seq_start; at -= kWalk) {
        load_tile<D, kWalk>(k, static_cast<const float *>(f.p.k), f.p.Hkv, hk, at, t.seq_end);
        load_tile<D, kWalk>(v, static_cast<const float *>(f.p.v), f.p.Hkv, hk, at, t.seq_end);
        landed<1>();
        float x[4][4], y[4][4];
        dot_tiles<D>(q, k, x);
        landed<0>();
        dot_tiles<D>(g, v, y);
        const int diag = t.first - at;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float z = lse2[4 * ty + i], dl = del[4 * ty + i];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[i][j] = tx + 16 * j <= 4 * ty + i + diag
                              ? exp2f(fmaf(x[i][j], c, -z)) * (y[i][j] - dl) : 0.f;
        }
        store_weights(w, x);
        __syncthreads();
        add_weighted<D>(w, k, acc);
        __syncthreads();
    }
    const float by[4] = {f.p.scale, f.p.scale, f.p.scale, f.p.scale};
    store_rows<D>(acc, by, f.gq + ((size_t)t.first * f.p.Hq + h) * D, (size_t)f.p.Hq * D,
                  t.seq_end - t.first, &bad);
    redo_rows(&bad, [&](int r) { redo_dq<D>(f, t.first + r, t.seq_start, h); });
    wait_for_previous();
}

// ---------------------------------------------------------------- dK and dV
// Own rows are keys, walked rows queries.
template <int D>
__global__ void __launch_bounds__(kThreads) dkv_kernel(const __grid_constant__ F32Params f)
{
    extern __shared__ __align__(16) float smem[];
    __shared__ float lse2[kWalk], del[kWalk];
    __shared__ unsigned bad;
    float *k = smem, *v = k + kRows * D, *q = v + kRows * D, *g = q + kWalk * D, *w = g + kWalk * D;
    const int rank = f.split > 1 ? cluster_rank() : 0, unit = blockIdx.x / f.split;
    let_next_start();
    AttnTile t = tile_of(f, unit / f.p.Hkv);
    if (t.first >= t.seq_end) return;  // all of a cluster
    if (!f.tiles && blockIdx.x == 0 && threadIdx.x == 0) *f.status = 0;
    // the list begins with a sequence's last tile; here the first one has most work
    const int count = (t.seq_end - t.seq_start + kRows - 1) / kRows;
    t.first = t.seq_start + (count - 1 - (t.first - t.seq_start) / kRows) * kRows;
    const int hk = unit % f.p.Hkv, G = f.p.Hq / f.p.Hkv;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    if (threadIdx.x == 0) bad = 0;
    load_tile<D, kRows>(k, static_cast<const float *>(f.p.k), f.p.Hkv, hk, t.first, t.seq_end);
    load_tile<D, kRows>(v, static_cast<const float *>(f.p.v), f.p.Hkv, hk, t.first, t.seq_end);
    const float c = f.p.scale * kLog2e;
    float ak[4][D / 16] = {}, av[4][D / 16] = {};
    for (int h = hk * G + rank; h < (hk + 1) * G; h += f.split)
        for (int at = t.first; at < t.seq_end; at += kWalk) {
            load_stats<kWalk>(f, lse2, del, h, at, t.seq_end);
            load_tile<D, kWalk>(q, static_cast<const float *>(f.p.q), f.p.Hq, h, at, t.seq_end);
            load_tile<D, kWalk>(g, f.dO, f.p.Hq, h, at, t.seq_end);
            landed<1>();
            float x[4][4], y[4][4];
            dot_tiles<D>(k, q, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float z = lse2[tx + 16 * j];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[i][j] = at > t.first || 4 * ty + i <= tx + 16 * j ? exp2f(fmaf(x[i][j], c, -z)) : 0.f;
            }
            store_weights(w, x);
            landed<0>();
            add_weighted<D>(w, g, av);
            dot_tiles<D>(v, g, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float dl = del[tx + 16 * j];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i][j] *= y[i][j] - dl;
            }
            __syncthreads();
            store_weights(w, x);
            __syncthreads();
            add_weighted<D>(w, q, ak);
            __syncthreads();
        }
    if (f.split > 1) {  // the first CTA adds up the others' sums, kept thread by thread
        if (rank) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int e = 0; e < D / 16; ++e) {
                    smem[(i * (D / 16) + e) * kThreads + threadIdx.x] = ak[i][e];
                    smem[((4 + i) * (D / 16) + e) * kThreads + threadIdx.x] = av[i][e];
                }
            }
        }
        cluster_sync();
        for (int r = 1; r < f.split && !rank; ++r) {
            const uint32_t from = tc::smem_u32(smem + threadIdx.x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int e = 0; e < D / 16; ++e) {
                    ak[i][e] += peer_float(from + (i * (D / 16) + e) * kThreads * 4, r);
                    av[i][e] += peer_float(from + ((4 + i) * (D / 16) + e) * kThreads * 4, r);
                }
            }
        }
        cluster_sync();
        if (rank) return;
    }
    const size_t out = ((size_t)t.first * f.p.Hkv + hk) * D, stride = (size_t)f.p.Hkv * D;
    const float one[4] = {1.f, 1.f, 1.f, 1.f};
    const float by[4] = {f.p.scale, f.p.scale, f.p.scale, f.p.scale};
    store_rows<D>(av, one, f.gv + out, stride, t.seq_end - t.first, &bad);
    store_rows<D>(ak, by, f.gk + out, stride, t.seq_end - t.first, &bad);
    redo_rows(&bad, [&](int r) { redo_dkv<D>(f, t.first + r, t.seq_end, hk); });
}

// The tile list, or none for uniform sequences.
cudaError_t prepare(const AttnProblem &p, bool bwd, void *workspace, F32Params &f, cudaStream_t st)
{
    f.status = static_cast<int *>(workspace);
    if (!p.cu_seqlens) return cudaSuccess;
    f.tiles = reinterpret_cast<const AttnTile *>(
        static_cast<char *>(workspace) + attn_workspace_layout(p, kRows, bwd).tiles);
    return launch_attn_plan(p, kRows, workspace, st);
}

template <int D>
cudaError_t fwd(const AttnProblem &p, void *o, float *lse, void *workspace, cudaStream_t st)
{
    F32Params f{};
    f.p = p;
    f.o = static_cast<float *>(o);
    f.lse_out = lse;
    const cudaError_t e = prepare(p, false, workspace, f, st);
    if (e != cudaSuccess) return e;
    return launch_kernel(fwd_kernel<D>, f, attn_tiles(p, kRows) * p.Hq, kThreads,
                         ((kRows + 2 * kWalk) * D + kRows * kW) * 4, 1, false, st);
}

template <int D>
cudaError_t bwd(const AttnProblem &p, const void *o, const float *lse, const void *dO, void *gq,
                void *gk, void *gv, void *workspace, cudaStream_t st)
{
    F32Params f{};
    f.p = p;
    float *delta = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                             attn_workspace_layout(p, kRows, true).delta);
    float *lse2 = delta + (size_t)p.tokens * p.Hq;
    f.lse = lse; f.lse2 = lse2; f.delta = delta;
    f.dO = static_cast<const float *>(dO);
    f.gq = static_cast<float *>(gq);
    f.gk = static_cast<float *>(gk);
    f.gv = static_cast<float *>(gv);
    cudaError_t e = prepare(p, true, workspace, f, st);
    if (e == cudaSuccess) e = launch_attn_delta(p, o, lse, dO, delta, lse2, st);
    const long long tiles = attn_tiles(p, kRows);
    const size_t smem = (2 * (kRows + kWalk) * D + kRows * kW) * 4;
    f.split = attn_head_split(p, kRows, 148 * 4);
    if (e == cudaSuccess) e = launch_kernel(dkv_kernel<D>, f, tiles * p.Hkv, kThreads, smem, f.split, false, st);
    if (e == cudaSuccess) e = launch_kernel(dq_kernel<D>, f, tiles * p.Hq, kThreads, smem, 1, true, st);
    return e;
}

}  // namespace

int attn_fwd_rows(const AttnProblem &p)
{
    return p.dtype == KDA_DTYPE_BF16 ? attn_tc_fwd_rows(p) : kRows;
}

int attn_bwd_rows(const AttnProblem &p)
{
    return p.dtype == KDA_DTYPE_BF16 ? attn_tc_bwd_rows() : kRows;
}

cudaError_t launch_attn_fwd(const AttnProblem &p, void *o, float *lse, void *ws, cudaStream_t st)
{
    if (p.dtype == KDA_DTYPE_BF16) return launch_attn_tc_fwd(p, o, lse, ws, st);
    if (p.d == 32) return fwd<32>(p, o, lse, ws, st);
    if (p.d == 64) return fwd<64>(p, o, lse, ws, st);
    return fwd<128>(p, o, lse, ws, st);
}

cudaError_t launch_attn_bwd(const AttnProblem &p, const void *o, const float *lse, const void *dO,
                            void *gq, void *gk, void *gv, void *ws, cudaStream_t st)
{
    if (p.dtype == KDA_DTYPE_BF16)
        return launch_attn_tc_bwd(p, o, lse, dO, gq, gk, gv, ws, st);
    if (p.d == 32) return bwd<32>(p, o, lse, dO, gq, gk, gv, ws, st);
    if (p.d == 64) return bwd<64>(p, o, lse, dO, gq, gk, gv, ws, st);
    return bwd<128>(p, o, lse, dO, gq, gk, gv, ws, st);
}

}  // namespace kda
