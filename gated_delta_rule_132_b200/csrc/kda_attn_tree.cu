// kda_attn_tree.cu — attention of a tree of drafted tokens (or one token) over a
// paged cache.
//
// The R tokens of a sequence times the G query heads that share a key/value head are
// the rows of one problem over that head's keys, so the cache is read once for all of
// them. One token of G heads reads 4 D bytes per key for 4 D G flops: HBM bounds the
// call until the rows number about a hundred.
//
// A CTA owns a tile of rows and a chunk of consecutive keys of one (sequence, kv
// head); chunks are what keeps all SMs busy when there are few sequences or their
// lengths differ. Softmax statistics run in fp32 over the chunk; a second kernel joins
// the chunks of rows that have several, in order.
//
// bf16: one warp brings tiles of 64 keys in by TMA, a box per page and 64 channels in
// the 128-byte swizzle (by 16-byte copies to the same places where a page has fewer
// than eight tokens), three stages deep; the other warps multiply with mma.sync, whose
// rate such few rows do not need all of. One warp that loads and knows the table takes
// a tile's cost from 716 instructions a warp (each thread copying, with a table lookup
// per key: 4.8 TB/s for one token of 256 sequences) to about 200: that case takes 691 us,
// 6.69 TB/s, all of the measured rate.
// fp32: 32 keys by 16-byte copies, CUDA cores.
// A key without a page, or behind the sequence, is filled with zeros and masked.
//
// Only drafted tokens are masked for some rows and not for others, so only their
// values can reach a row through 0 * inf: rows whose result is not finite are computed
// again from the keys they see.
#include <algorithm>

#include "kda_attn_tree.cuh"

namespace kda {
namespace {

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// ---------------------------------------------------------------- shapes
constexpr int kStages = 3;
enum : int { kErrTreeFull = 121, kErrTreeFree, kErrTreeDrain };

// bf16: kWm x kWk warps that multiply (kWm groups of 16 rows, the tile's keys shared out
// over kWk warps, whose sums are joined at the end) and one that loads. Row r of the
// problem is token r / G, head r % G.
template <int D, int kWm, int kWk>
struct MmaShape {
    static constexpr int kWarps = kWm * kWk, kThreads = 32 * (kWarps + 1), kMaskThreads = 32 * kWarps;
    static constexpr int kGroups = kWk, kRows = 16 * kWm, kKeys = 64;
    static constexpr int kBlocks = (D + 63) / 64, kBlock = kKeys * 128;
    static constexpr int kTile = kBlocks * kBlock;  // of K, and of V
    static constexpr int kRing = kStages * 2 * kTile, kJoin = kWk * kRows * D * 4;
    static constexpr int kMl = kRing > kJoin ? kRing : kJoin;  // float2 [kWk][kRows]
    static constexpr int kSeen = kMl + kWk * kRows * 8;        // 64 x 8 bytes
    static constexpr int kParents = kSeen + 512;               // 64 x 4
    static constexpr int kBars = kParents + 256;
    static constexpr int kBytes = kBars + 128 + 1024;          // and the base's alignment
};

// fp32: 128 threads, 16 rows.
template <int D>
struct F32Shape {
    static constexpr int kThreads = 128, kMaskThreads = 128, kGroups = 1, kRows = 16, kKeys = 32;
    static constexpr int kTile = kKeys * D * 4, kRing = kStages * 2 * kTile;
    static constexpr int kMl = kRing, kSeen = kMl + kRows * 8, kParents = kSeen + 512;
    static constexpr int kQ = kParents + 256, kP = kQ + kRows * D * 4;  // P [16][36]
    static constexpr int kBytes = kP + kRows * 36 * 4;
};

// fp32: byte offset of 16-byte unit u of row r in a tile; units are exchanged within a
// row so that eight consecutive rows' equal units lie in different banks.
template <int D> __device__ __forceinline__ uint32_t unit_at(int r, int u)
{
    return (uint32_t)(r * (D / 4) + (u ^ (r & 7))) * 16;
}

// fp32: start the copies of the tile of keys from pos on.
template <int D, int kKeys, int kThreads>
__device__ __forceinline__ void load_keys(const TreeParams &f, const Share &s, int pos, char *k,
                                          char *v)
{
    constexpr int kUnits = D / 4, kStep = kThreads / kUnits;
    const int u = threadIdx.x % kUnits;
#pragma unroll
    for (int r = threadIdx.x / kUnits; r < kKeys; r += kStep) {
        const int c = pos + r;
        const long long at = c < s.last ? key_at(f.p, s.table, c, s.hk) : -1;
        const size_t off = (at < 0 ? 0 : (size_t)at * 4) + u * 16;
        const uint32_t to = unit_at<D>(r, u);
        cp_async16_or_zero(k + to, static_cast<const char *>(f.p.k_pages) + off, at >= 0);
        cp_async16_or_zero(v + to, static_cast<const char *>(f.p.v_pages) + off, at >= 0);
    }
}

// Bit j: key pos + j is one of the sequence's and has a page (32 keys from pos on).
__device__ __forceinline__ uint32_t real_keys(const TreeParams &f, const Share &s, int pos)
{
    const int c = pos + (threadIdx.x & 31);
    return __ballot_sync(0xffffffffu, c < s.last && key_at(f.p, s.table, c, s.hk) >= 0);
}

// Join the key groups' sums of each row (in shared memory) and write the row, or its
// share of it.
template <typename T, int D, typename S>
__device__ __forceinline__ void join_rows(const TreeParams &f, const Share &s, const char *smem)
{
    constexpr int V = D / 32;
    const float *sums = reinterpret_cast<const float *>(smem);
    const float2 *ml = reinterpret_cast<const float2 *>(smem + S::kMl);
    const unsigned long long *seen = reinterpret_cast<const unsigned long long *>(smem + S::kSeen);
    const int lane = threadIdx.x & 31, G = f.p.Hq / f.p.Hkv;
    for (int r = threadIdx.x >> 5; r < S::kRows && s.row0 + r < f.rows; r += S::kThreads / 32) {
        float m = -INFINITY, l = 0.f, acc[V] = {};
#pragma unroll
        for (int w = 0; w < S::kGroups; ++w) m = fmaxf(m, ml[w * S::kRows + r].x);
#pragma unroll
        for (int w = 0; w < S::kGroups; ++w) {
            const float2 x = ml[w * S::kRows + r];
            if (x.x == -INFINITY && x.y == 0.f) continue;  // this group had no key
            const float by = tc::exp2_fast(x.x - m);
            l = fmaf(x.y, by, l);
#pragma unroll
            for (int e = 0; e < V; ++e)
                acc[e] = fmaf(sums[(w * S::kRows + r) * D + lane * V + e], by, acc[e]);
        }
        const int row = s.row0 + r, i = row / G, h = s.hk * G + row % G;
        if (s.alone) {
            finish_row<T, D>(f.p, s.n, i, h, m, l, seen[i] == 0, acc);
        } else {
            const size_t at = (((size_t)s.n * f.p.Hkv + s.hk) * f.chunks + s.chunk) * f.rows + row;
#pragma unroll
            for (int e = 0; e < V; ++e) f.part_o[at * D + lane * V + e] = acc[e];
            if (lane == 0) f.part_ml[at] = make_float2(m, l);
        }
    }
}

// ---------------------------------------------------------------- bf16
// The loading warp: 64 keys from pos on into a stage, and which of them are there. By a
// box per page (`page`: this lane's), or by 16-byte copies where pages have fewer than
// eight tokens.
template <int D, typename S>
__device__ __forceinline__ void load_boxes(const TreeParams &f, const Share &s, int pos, int page,
                                           char *k, uint64_t *full, unsigned long long *there)
{
    const Boxes<64> boxes(f);
    const int lane = threadIdx.x & 31, row = boxes.row(f, s, pos, page);
    const uint32_t lo = boxes.there(f, s, pos, row, 0), hi = boxes.there(f, s, pos, row, 1);
    if (lane == 0) {
        *there = (unsigned long long)hi << 32 | lo;
        tc::mbar_arrive_expect_tx(full, 2 * S::kTile);
    }
    __syncwarp();
    if (lane < boxes.count()) {
#pragma unroll
        for (int b = 0; b < S::kBlocks; ++b) {
            char *to = k + b * S::kBlock + boxes.key() * 128;
            tc::tma_load_2d(to, &f.k, b * 64, row, full);
            tc::tma_load_2d(to + S::kTile, &f.v, b * 64, row, full);
        }
    }
}

template <int D, typename S>
__device__ __forceinline__ void load_units(const TreeParams &f, const Share &s, int pos, char *k,
                                           uint64_t *full, unsigned long long *there)
{
    constexpr int kUnits = D / 8;
    const int lane = threadIdx.x & 31;
    unsigned long long real = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int c = pos + 32 * e + lane;
        real |= (unsigned long long)__ballot_sync(0xffffffffu, c < s.last && key_at(f.p, s.table, c, s.hk) >= 0)
                << 32 * e;
    }
    if (lane == 0) *there = real;
    for (int i = lane; i < 64 * kUnits; i += 32) {
        const int r = i / kUnits, u = i % kUnits;
        const bool is = real >> r & 1;
        const size_t from = (is ? (size_t)key_at(f.p, s.table, pos + r, s.hk) * 2 : 0) + u * 16;
        char *to = k + (u >> 3) * S::kBlock + tc::sw128(r, (u & 7) * 16);
        cp_async16_or_zero(to, static_cast<const char *>(f.p.k_pages) + from, is);
        cp_async16_or_zero(to + S::kTile, static_cast<const char *>(f.p.v_pages) + from, is);
    }
    tc::cp_async_arrive(full);
    if (lane == 0) tc::mbar_arrive(full);
    __syncwarp();
}

template <int D, int kWm, int kWk>
__global__ void __launch_bounds__(MmaShape<D, kWm, kWk>::kThreads)
tree_mma_kernel(const __grid_constant__ TreeParams f)
{
    typedef __nv_bfloat16 T;
    using S = MmaShape<D, kWm, kWk>;
    extern __shared__ char smem_raw[];
    char *smem = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr int kMine = S::kKeys / kWk;  // keys of a tile that are this warp's
    constexpr int kNt = kMine / 8, kDt = D / 8;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + S::kBars), *free = full + kStages;
    unsigned long long *there_of = reinterpret_cast<unsigned long long *>(free + kStages);
    volatile int *abort = reinterpret_cast<volatile int *>(there_of + kStages);
    if (blockIdx.x == 0 && threadIdx.x == 0) *f.status = 0;
    asm volatile("griddepcontrol.launch_dependents;");
    Share s;
    if (!share_of(f, s)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = s.last > s.first ? (s.last - s.first + S::kKeys - 1) / S::kKeys : 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(full + i, f.p.page_shift >= 3 ? 1 : 33);
            tc::mbar_init(free + i, S::kWarps);
        }
        *abort = 0;
        tc::fence_mbar_init();
    }
    __syncthreads();

    if (warp == S::kWarps) {
        if (!f.starve) {
            const bool by_page = f.p.page_shift >= 3;
            int tile = 0, page = by_page && tiles ? Boxes<64>(f).page(f, s, s.first) : 0;
            for (; tile < tiles; ++tile) {
                const int st = tile % kStages, use = tile / kStages, pos = s.first + tile * S::kKeys;
                char *to = smem + st * 2 * S::kTile;
                const int next = by_page ? Boxes<64>(f).page(f, s, pos + S::kKeys) : 0;
                const bool go = !use || tc::mbar_wait(free + st, (use - 1) & 1, abort, f.status, kErrTreeFree, f.spin);
                if (!__all_sync(0xffffffffu, go)) break;
                if (by_page) load_boxes<D, S>(f, s, pos, page, to, full + st, there_of + st);
                else load_units<D, S>(f, s, pos, to, full + st, there_of + st);
                page = next;
            }
            // whatever the other warps do, the copies land before the memory is used again
            for (int i = max(0, tile - kStages); i < tile; ++i)
                tc::mbar_drain(full + i % kStages, (i / kStages) & 1, f.status, kErrTreeDrain);
        }
        __syncthreads();
    } else {
        const int wm = warp / kWk, wk = warp % kWk, g = lane >> 2, t = lane & 3;
        const int G = f.p.Hq / f.p.Hkv;
        const unsigned long long *seen = tree_masks<S>(f, s.n, smem);
        // this warp's 16 rows of q as operands, and the drafts that its two rows see
        uint32_t q[D / 16][4];
        unsigned long long mine[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = min(s.row0 + wm * 16 + g + 8 * e, f.rows - 1), i = r / G, h = s.hk * G + r % G;
            const uint32_t *from = reinterpret_cast<const uint32_t *>(
                static_cast<const T *>(f.p.q) + (((size_t)s.n * f.p.R + i) * f.p.Hq + h) * D);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                q[kk][e] = __ldg(from + kk * 8 + t);
                q[kk][2 + e] = __ldg(from + kk * 8 + 4 + t);
            }
            mine[e] = seen[i];
        }
        // A row of a block is 128 bytes, its 16-byte units exchanged by the row's low three
        // bits, which are the lane's in every access here; so an operand's place is a
        // lane's constant exclusive-or its unit, plus constants.
        const uint32_t base = tc::smem_u32(smem);
        const uint32_t k_lane = (wk * kMine + (lane >> 4) * 8 + (lane & 7)) * 128;
        const uint32_t k_unit = (((lane >> 3) & 1) ^ (lane & 7)) * 16;
        const uint32_t v_lane = (wk * kMine + (lane & 15)) * 128;
        const uint32_t v_unit = ((lane >> 4) ^ (lane & 7)) * 16;

        const float c = f.p.scale * kTreeLog2e;
        float o[kDt][4] = {};
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        for (int tile = 0; tile < tiles; ++tile) {
            const int st = tile % kStages;
            if (!__all_sync(0xffffffffu, tc::mbar_wait(full + st, (tile / kStages) & 1, abort, f.status,
                                                       kErrTreeFull, f.spin)))
                break;
            const uint32_t k = base + st * 2 * S::kTile + k_lane, v = base + (st * 2 + 1) * S::kTile + v_lane;
            const int pos = s.first + tile * S::kKeys + wk * kMine;  // of this warp's first key
            float x[kNt][4] = {};
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t at = k + (kk >> 2) * S::kBlock + (k_unit ^ ((kk & 3) * 32));
#pragma unroll
                for (int nt = 0; nt < kNt; nt += 2) {
                    uint32_t b[4];  // two groups of 8 keys x 16 channels
                    ldmatrix4(at + nt * 8 * 128, b);
                    mma16816(x[nt], q[kk], b[0], b[1]);
                    mma16816(x[nt + 1], q[kk], b[2], b[3]);
                }
            }
            // keys that are there and seen; whole tiles of cached keys need no look
            const unsigned long long there = there_of[st];
            if (there != ~0ull || pos + kMine > s.ctx) {
                // what is behind the sequence in its last page is not to meet a weight of 0;
                // a warp clears what it will read itself
                for (int r = lane; r < kMine; r += 32)
                    if (!(there >> (wk * kMine + r) & 1)) {
#pragma unroll
                        for (int b = 0; b < S::kBlocks; ++b) {
                            uint4 *row = reinterpret_cast<uint4 *>(
                                smem + (st * 2 + 1) * S::kTile + b * S::kBlock + (wk * kMine + r) * 128);
#pragma unroll
                            for (int u = 0; u < 8; ++u) row[u] = make_uint4(0, 0, 0, 0);
                        }
                    }
                tc::fence_proxy_async_smem();  // before a later copy into the stage
                __syncwarp();
#pragma unroll
                for (int nt = 0; nt < kNt; ++nt) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = nt * 8 + t * 2 + (e & 1), draft = pos + j - s.ctx;
                        const bool see = (there >> (wk * kMine + j) & 1) &&
                                         (draft < 0 || (mine[e >> 1] >> (draft & 63) & 1));
                        if (!see) x[nt][e] = -INFINITY;
                    }
                }
            }
            uint32_t p[kNt][2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = -INFINITY;
#pragma unroll
                for (int nt = 0; nt < kNt; ++nt) top = fmaxf(top, fmaxf(x[nt][2 * e], x[nt][2 * e + 1]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                top = fmaxf(m[e], top * c);
                const float ref = top == -INFINITY ? 0.f : top;
                if (__any_sync(0xffffffffu, top != m[e])) {
                    const float keep = tc::exp2_fast(m[e] - ref);
                    l[e] *= keep;
#pragma unroll
                    for (int dt = 0; dt < kDt; ++dt) {
                        o[dt][2 * e] *= keep;
                        o[dt][2 * e + 1] *= keep;
                    }
                    m[e] = top;
                }
#pragma unroll
                for (int nt = 0; nt < kNt; ++nt) {
                    const float a = tc::exp2_fast(fmaf(x[nt][2 * e], c, -ref));
                    const float b = tc::exp2_fast(fmaf(x[nt][2 * e + 1], c, -ref));
                    l[e] += a + b;
                    p[nt][e] = tc::bf16x2(a, b);
                }
            }
#pragma unroll
            for (int kk = 0; kk < kNt / 2; ++kk) {
                const uint32_t a[4] = {p[2 * kk][0], p[2 * kk][1], p[2 * kk + 1][0], p[2 * kk + 1][1]};
#pragma unroll
                for (int dt = 0; dt < kDt; dt += 2) {
                    uint32_t b[4];  // 16 keys x 16 channels, transposed
                    ldmatrix4_t(v + kk * 16 * 128 + (dt >> 3) * S::kBlock + (v_unit ^ ((dt & 7) * 16)), b);
                    mma16816(o[dt], a, b[0], b[1]);
                    mma16816(o[dt + 1], a, b[2], b[3]);
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(free + st);
        }
        __syncthreads();  // the ring is done with
        float *sums = reinterpret_cast<float *>(smem);
        float2 *ml = reinterpret_cast<float2 *>(smem + S::kMl);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            const int r = wk * S::kRows + wm * 16 + g + 8 * e;
            if (t == 0) ml[r] = make_float2(m[e], l[e]);
#pragma unroll
            for (int dt = 0; dt < kDt; ++dt)
                *reinterpret_cast<float2 *>(sums + r * D + dt * 8 + t * 2) =
                    make_float2(o[dt][2 * e], o[dt][2 * e + 1]);
        }
    }
    __syncthreads();
    if (*abort) return;
    join_rows<T, D, S>(f, s, smem);
}

// ---------------------------------------------------------------- fp32, CUDA cores
// 128 threads, 16 rows: 8 threads per row, each 4 of the 32 keys, then D / 8 channels.
template <int D>
__global__ void __launch_bounds__(128) tree_fp32_kernel(const __grid_constant__ TreeParams f)
{
    typedef float T;
    using S = F32Shape<D>;
    constexpr int kPer = D / 8, kQ = D / 4;
    extern __shared__ __align__(128) char smem[];
    if (blockIdx.x == 0 && threadIdx.x == 0) *f.status = 0;
    asm volatile("griddepcontrol.launch_dependents;");
    Share s;
    if (!share_of(f, s)) return;
    const int r = threadIdx.x >> 3, j8 = threadIdx.x & 7, G = f.p.Hq / f.p.Hkv;
    const int row = s.row0 + r;
    float *q = reinterpret_cast<float *>(smem + S::kQ), *w = reinterpret_cast<float *>(smem + S::kP);

    const int tiles = s.last > s.first ? (s.last - s.first + S::kKeys - 1) / S::kKeys : 0;
    auto load = [&](int tile) {
        if (tile < tiles) {
            char *k = smem + tile % kStages * 2 * S::kTile;
            load_keys<D, S::kKeys, S::kThreads>(f, s, s.first + tile * S::kKeys, k, k + S::kTile);
        }
        cp_async_commit();
    };
    for (int i = 0; i < kStages - 1; ++i) load(i);
    for (int i = threadIdx.x; i < 16 * D; i += S::kThreads) {
        const int x = min(s.row0 + i / D, f.rows - 1);
        q[i] = static_cast<const T *>(
            f.p.q)[(((size_t)s.n * f.p.R + x / G) * f.p.Hq + s.hk * G + x % G) * D + i % D];
    }
    const unsigned long long *seen = tree_masks<S>(f, s.n, smem);
    const unsigned long long mine = row < f.rows ? seen[row / G] : 0;
    const float4 *qr = reinterpret_cast<const float4 *>(q + r * D);

    float m = -INFINITY, l = 0.f, o[kPer] = {};
    for (int tile = 0; tile < tiles; ++tile) {
        cp_async_wait<kStages - 2>();
        __syncthreads();
        load(tile + kStages - 1);
        const char *k = smem + tile % kStages * 2 * S::kTile, *v = k + S::kTile;
        const int pos = s.first + tile * S::kKeys;
        float x[4] = {};
        for (int e = 0; e < kQ; ++e) {
            const float4 a = qr[e];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 b = *reinterpret_cast<const float4 *>(k + unit_at<D>(j8 + 8 * j, e));
                x[j] = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, x[j]))));
            }
        }
        const uint32_t there = real_keys(f, s, pos);
        float top = m;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int key = j8 + 8 * j, draft = pos + key - s.ctx;
            const bool see = (there >> key & 1) && (draft < 0 || (mine >> (draft & 63) & 1));
            x[j] = see ? x[j] * f.p.scale * kTreeLog2e : -INFINITY;
            top = fmaxf(top, x[j]);
        }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float ref = top == -INFINITY ? 0.f : top;
        const float keep = exp2f(m - ref);
        m = top;
        l *= keep;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float p = exp2f(x[j] - ref);
            l += p;
            w[r * 36 + j8 + 8 * j] = p;
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] *= keep;
        // thread j8 has the channels of units j8, j8 + 8, ...
        for (int key = 0; key < S::kKeys; ++key) {
            const float p = w[r * 36 + key];
#pragma unroll
            for (int e = 0; e < kPer / 4; ++e) {
                const float4 b = *reinterpret_cast<const float4 *>(v + unit_at<D>(key, j8 + 8 * e));
                o[4 * e] = fmaf(p, b.x, o[4 * e]);
                o[4 * e + 1] = fmaf(p, b.y, o[4 * e + 1]);
                o[4 * e + 2] = fmaf(p, b.z, o[4 * e + 2]);
                o[4 * e + 3] = fmaf(p, b.w, o[4 * e + 3]);
            }
        }
        __syncwarp();
    }
    cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    float *sums = reinterpret_cast<float *>(smem);
    if (j8 == 0) reinterpret_cast<float2 *>(smem + S::kMl)[r] = make_float2(m, l);
#pragma unroll
    for (int e = 0; e < kPer / 4; ++e)
        *reinterpret_cast<float4 *>(sums + r * D + (j8 + 8 * e) * 4) =
            make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
    __syncthreads();
    join_rows<T, D, S>(f, s, smem);
}

// ---------------------------------------------------------------- joining chunks
// kWarps warps per row of a sequence that has several chunks: each adds up every
// kWarps-th chunk, the first one adds up the warps. One warp per row where there are
// rows enough to fill the SMs; eight shorten the chain of dependent reads (32 rows of 15
// chunks: 8.8 us with one).
template <typename T, int D, int kWarps>
__global__ void __launch_bounds__(256) tree_join_kernel(const __grid_constant__ TreeParams f)
{
    constexpr int V = D / 32;
    __shared__ float s_acc[8][D], s_l[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % kWarps;
    // rows fit in 31 bits (with 64-bit divisions 12288 rows take 4 us longer)
    const unsigned unit = blockIdx.x * (8 / kWarps) + warp / kWarps;
    if (unit >= (unsigned)(f.p.N * f.p.R * f.p.Hq)) return;  // whole blocks where kWarps is 8
    const int G = f.p.Hq / f.p.Hkv;
    const int h = unit % (unsigned)f.p.Hq, t = unit / (unsigned)f.p.Hq, i = t % f.p.R, n = t / f.p.R;
    int end;
    const int chunk = chunk_of(f, n, end);
    // an absent token's sums mean nothing
    const bool absent = f.p.parents && ancestors(f.p.parents + (size_t)n * f.p.R, i) == 0;
    wait_for_previous();
    if (end <= chunk) return;
    const int count = (end + chunk - 1) / chunk;
    const size_t base = ((size_t)n * f.p.Hkv + h / G) * f.chunks * f.rows + i * G + h % G;
    float m = -INFINITY;
    for (int c = lane; c < count; c += 32) m = fmaxf(m, f.part_ml[base + (size_t)c * f.rows].x);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float l = 0.f, acc[V] = {};
#pragma unroll 8
    for (int c = part; c < count; c += kWarps) {
        const size_t at = base + (size_t)c * f.rows;
        const float2 x = f.part_ml[at];
        const bool none = x.x == -INFINITY && x.y == 0.f;  // the chunk had no key for this row
        const float by = tc::exp2_fast(x.x - m);
        l = none ? l : fmaf(x.y, by, l);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float y = f.part_o[at * D + lane * V + e];
            acc[e] = none ? acc[e] : fmaf(y, by, acc[e]);
        }
    }
    if (kWarps > 1) {
#pragma unroll
        for (int e = 0; e < V; ++e) s_acc[warp][lane * V + e] = acc[e];
        if (lane == 0) s_l[warp] = l;
        __syncthreads();
        if (part) return;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            l += s_l[w];
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] += s_acc[w][lane * V + e];
        }
    }
    finish_row<T, D>(f.p, n, i, h, m, l, absent, acc);
}

// ---------------------------------------------------------------- host
// More than 32 rows go to the tcgen05 kernel (64 rows of 16 sequences of 8000 tokens: 153 us,
// by mma.sync, whose rate bounds it, 198; 48 rows of 64 of 4000: 247, 380; 64 rows of one of
// 900: 21.5, 19.5). 32 rows and fewer are as quick either way where there is much to read.
bool many_rows(const TreeProblem &p)
{
    return p.dtype == KDA_DTYPE_BF16 && p.R * (p.Hq / p.Hkv) > 32 && tree_tc_rows(p) > 0;
}

int rows_per_cta(const TreeProblem &p)
{
    const int rows = p.R * (p.Hq / p.Hkv);
    if (rows <= 16 || p.dtype == KDA_DTYPE_F32) return 16;
    return many_rows(p) ? tree_tc_rows(p) : 32;
}

TreeParams plan(const TreeProblem &p)
{
    TreeParams f{};
    f.p = p;
    f.rows = p.R * (p.Hq / p.Hkv);
    f.tile_rows = rows_per_cta(p);
    f.row_tiles = (f.rows + f.tile_rows - 1) / f.tile_rows;
    f.tile_keys = many_rows(p) ? 128 : 64;
    // mma.sync: two CTAs to an SM, many rows: one. A chunk's beginning and end cost as much as
    // four tiles or so. So short calls get one CTA to a place, longer ones chunks of 1024
    // keys until these make six rounds (three) of CTAs, which balance the SMs (in us, against
    // six rounds for all: one token of 8 sequences of 2000 tokens 34, 42; of 16 of 8168: 112,
    // 134; 4 of 32 of 1000..2147: 62, 101; 8 of 4 of 16000: 77, 122. 24 drafts over 16
    // contexts of 1024..65536, three rounds: 590; chunks of 2048 keys 731; chunks that fill
    // whole rounds 623). A sequence can have as many chunks as make 2048 CTAs of equal ones,
    // or up to four that make 8192: half of that costs batches of unequal lengths more (64000
    // tokens and 15 times 1000: 89 and 124) than CTAs without a chunk cost others (8 of 2000:
    // 34 and 30).
    const long long longest = (long long)p.M << p.page_shift;
    const long long units = (long long)p.N * p.Hkv * f.row_tiles;
    const bool many = many_rows(p);
    const long long most = many ? 148 * 8 / units : std::max(2048 / units, std::min(8192 / units, 4ll));
    f.share = (float)(p.Hkv * f.row_tiles) / (many ? 148 : 148 * 2);
    f.per_round = 1.f / (many ? 3 : 6);
    f.least_keys = 1024;
    f.most_keys = many ? 1 << 20 : 2048;
    f.chunks = (int)std::min({(longest + f.tile_keys - 1) / f.tile_keys, std::max(most, 1ll), 256ll});
    return f;
}

// A launch that may begin while its predecessor ends (it waits for it itself).
template <typename K>
cudaError_t start(K kernel, const TreeParams &f, long long ctas, int threads, int smem,
                  bool follows, cudaStream_t st)
{
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    if (smem > 48 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = follows ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, f);
    note_launch();
    return e;
}

template <int D, int kWm, int kWk>
cudaError_t start_mma(const TreeParams &f, long long ctas, cudaStream_t st)
{
    using S = MmaShape<D, kWm, kWk>;
    return start(tree_mma_kernel<D, kWm, kWk>, f, ctas, S::kThreads, S::kBytes, false, st);
}

// A pool as rows of a head's D channels, boxes of 64 channels x the rows that a tile has
// of a page; what lies outside reads zero.
bool encode_pool_map(CUtensorMap *tm, const void *base, int D, long long rows, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)D * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    cuuint32_t estride[2] = {1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides,
               box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t launch(const TreeProblem &p, void *workspace, cudaStream_t st)
{
    TreeParams f = plan(p);
    char *ws = static_cast<char *>(workspace);
    const size_t parts = (size_t)p.N * p.Hkv * f.chunks * f.rows;
    f.status = reinterpret_cast<int *>(ws);
    f.part_ml = reinterpret_cast<float2 *>(ws + kWsHeader);
    f.part_o = reinterpret_cast<float *>(ws + kWsHeader + align_up(parts * sizeof(float2), 256));
    const DebugKnobs dbg = debug_knobs();
    f.spin = dbg.wait_limit ? dbg.wait_limit : tc::kSpinLimit;
    f.starve = dbg.starve_carry;
    const long long ctas = (long long)p.N * p.Hkv * f.row_tiles * f.chunks;
    cudaError_t e;
    if constexpr (sizeof(T) == 4) {
        using S = F32Shape<D>;
        e = start(tree_fp32_kernel<D>, f, ctas, S::kThreads, S::kBytes, false, st);
    } else {
        const int page = 1 << p.page_shift;
        f.pool_rows = p.P * p.Hkv * page;
        const int box = page < f.tile_keys ? page : f.tile_keys;
        if (page >= 8 && (!encode_pool_map(&f.k, p.k_pages, D, f.pool_rows, box) ||
                          !encode_pool_map(&f.v, p.v_pages, D, f.pool_rows, box)))
            return cudaErrorInvalidValue;
        e = f.tile_rows == 16   ? start_mma<D, 1, 4>(f, ctas, st)
            : f.tile_rows == 32 ? start_mma<D, 2, 2>(f, ctas, st)
                                : launch_tree_tc(f, ctas, st);
    }
    if (e != cudaSuccess || f.chunks == 1) return e;
    const long long rows = (long long)p.N * p.R * p.Hq;
    return rows < 148 * 8
               ? start(tree_join_kernel<T, D, 8>, f, rows, 256, 0, true, st)
               : start(tree_join_kernel<T, D, 1>, f, (rows + 7) / 8, 256, 0, true, st);
}

}  // namespace

size_t tree_workspace_bytes(const TreeProblem &p)
{
    if (p.R == 0) return 0;
    const TreeParams f = plan(p);
    const size_t parts = f.chunks == 1 ? 0 : (size_t)p.N * p.Hkv * f.chunks * f.rows;
    return kWsHeader + align_up(parts * sizeof(float2), 256) + parts * p.d * sizeof(float);
}

cudaError_t launch_attn_tree(const TreeProblem &p, void *workspace, cudaStream_t st)
{
    if (p.dtype == KDA_DTYPE_F32) {
        if (p.d == 32) return launch<float, 32>(p, workspace, st);
        if (p.d == 64) return launch<float, 64>(p, workspace, st);
        return launch<float, 128>(p, workspace, st);
    }
    if (p.d == 32) return launch<__nv_bfloat16, 32>(p, workspace, st);
    if (p.d == 64) return launch<__nv_bfloat16, 64>(p, workspace, st);
    return launch<__nv_bfloat16, 128>(p, workspace, st);
}

}  // namespace kda
