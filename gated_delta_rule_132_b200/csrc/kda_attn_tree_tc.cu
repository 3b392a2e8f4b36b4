// kda_attn_tree_tc.cu — tree attention of more than 32 rows per key/value head on the
// tcgen05 tensor cores (bf16).
//
// The prompt forward's pipeline over a chunk of a paged cache: S = Q K^T in TMEM, one
// thread per row for the softmax, P in bf16 over S, O += P V. A query tile is as many
// whole tokens as fit in 128 rows, fetched by one box of a four-dimensional map (token,
// kv head, head of its group, channel). Two softmax warpgroups work in turn:
//  * two query tiles, each over all keys of the chunk (kPair), or
//  * one query tile, the first warpgroup over the even key tiles, the second over the
//    odd ones, with sums of their own in TMEM that both join at the end.
// Either way one half's products run while the other half is in its softmax. 24 drafts of
// 32 heads over 16 contexts of 1024..65536 tokens, 618,000 in all: 583 us, 4.35 TB/s, 0.66
// of the measured rate. While all SMs have keys to read the cache's bytes bound it; the
// difference is chunks that begin (four tiles' time) and end at different times, and the
// partial sums' join (15 us).
#include "kda_attn_tree.cuh"

namespace kda {
namespace {

constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * 168, "register split");
constexpr float kRescale = 8.f;  // log2 of the growth that moves the reference

enum : int { kErrQ = 131, kErrV, kErrFree, kErrS, kErrP, kErrO, kErrDrain };

template <int D, bool kPair>
struct TcShape {
    static constexpr int kMaskThreads = 256;
    // Without kPair a stage is to serve the same half always: even numbers of them.
    static constexpr int kStagesK = D < 128 || !kPair ? 4 : 2, kStagesV = D < 128 ? 4 : 2;
    static constexpr uint32_t kTile = TileShape<D>::kBytes;
    static constexpr uint32_t kQ = 0, kK = (kPair ? 2 : 1) * kTile, kV = kK + kStagesK * kTile;
    static constexpr uint32_t kSeen = kV + kStagesV * kTile;  // 64 x 8 bytes
    static constexpr uint32_t kParents = kSeen + 512;         // 64 x 4
    static constexpr uint32_t kMl = kParents;                 // then float2 [128] of the odd tiles
    static constexpr uint32_t kBad = kMl + 1024;              // rows to compute again, 8 words
    // [step % 8] 16 bytes: which keys are there. Written with the keys' load, read when their
    // scores are; by then the loads are at most six steps on.
    static constexpr uint32_t kThere = kBad + 32;
    static constexpr uint32_t kBars = kThere + 128;
    static constexpr uint32_t kBytes = kBars + (6 + 2 * kStagesK + 2 * kStagesV) * 8 + 8 + 1024;
    static_assert(kThere % 16 == 0, "alignment");
    static constexpr uint32_t kTmemS = 0, kTmemO = 256;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

// A loading warp: 128 keys from pos on of one pool into a stage, by a box per page.
template <int D>
__device__ __forceinline__ void load_boxes(const Boxes<kTileRows> &boxes, int row, const CUtensorMap *map,
                                           uint8_t *to, uint64_t *full)
{
    const int lane = threadIdx.x & 31;
    if (lane == 0) tc::mbar_arrive_expect_tx(full, TileShape<D>::kBytes);
    __syncwarp();
    if (lane < boxes.count()) {
#pragma unroll
        for (int b = 0; b < TileShape<D>::kBlocks; ++b)
            tc::tma_load_2d(to + b * kBlockBytes + boxes.key() * 128, map, b * 64, row, full);
    }
}

// The same by 16-byte copies, where pages have fewer than eight tokens.
template <int D>
__device__ __forceinline__ void load_units(const TreeParams &f, const Share &s, int pos, const void *pool,
                                           uint8_t *to, uint64_t *full)
{
    constexpr int kUnits = D / 8;
    const int lane = threadIdx.x & 31;
    for (int i = lane; i < kTileRows * kUnits; i += 32) {
        const int r = i / kUnits, u = i % kUnits;
        const long long at = pos + r < s.last ? key_at(f.p, s.table, pos + r, s.hk) : -1;
        cp_async16_or_zero(to + (u >> 3) * kBlockBytes + tc::sw128(r, (u & 7) * 16),
                           static_cast<const char *>(pool) + (at < 0 ? 0 : (size_t)at * 2) + u * 16, at >= 0);
    }
    tc::cp_async_wait_all();
    tc::fence_proxy_async_smem();  // the tensor cores read what these copies wrote
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(full);
}

template <int D>
__device__ __noinline__ void redo_row(const TreeParams &f, int n, int i, int h)
{
    tree_row<__nv_bfloat16, D>(f.p, n, i, h);
}

template <int D, bool kPair>
__global__ void __launch_bounds__(kThreads, 1) tree_tc_kernel(const __grid_constant__ TreeParams f)
{
    typedef __nv_bfloat16 T;
    using S = TcShape<D, kPair>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *q_full = reinterpret_cast<uint64_t *>(sm + S::kBars);
    uint64_t *k_full = q_full + 1, *k_free = k_full + S::kStagesK;
    uint64_t *v_full = k_free + S::kStagesK, *v_free = v_full + S::kStagesV;
    uint64_t *s_full = v_free + S::kStagesV, *p_full = s_full + 2, *o_full = p_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(o_full + 1);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
    uint32_t *there_of = reinterpret_cast<uint32_t *>(sm + S::kThere);
    uint32_t *bad = reinterpret_cast<uint32_t *>(sm + S::kBad);

    if (blockIdx.x == 0 && threadIdx.x == 0) *f.status = 0;
    asm volatile("griddepcontrol.launch_dependents;");
    Share s;
    if (!share_of(f, s)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = f.p.Hq / f.p.Hkv, tokens = kTileRows / G, rows = tokens * G;  // of a query tile
    const int i0 = s.row0 / G;                                                  // this CTA's first token
    const bool two = kPair && i0 + tokens < f.p.R;
    const int steps = s.last > s.first ? (s.last - s.first + kTileRows - 1) / kTileRows : 0;

    if (warp == 8) tc::tmem_alloc(tmem_slot, 512);
    if (threadIdx.x == 0) {
        tc::mbar_init(q_full, 1);
        for (int i = 0; i < S::kStagesK; ++i) {
            tc::mbar_init(k_full + i, 1);
            tc::mbar_init(k_free + i, 1 + two);  // kPair: by both halves
        }
        for (int i = 0; i < S::kStagesV; ++i) {
            tc::mbar_init(v_full + i, 1);
            tc::mbar_init(v_free + i, 1 + two);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(s_full + i, 1);
            tc::mbar_init(p_full + i, 4);
        }
        tc::mbar_init(o_full, kPair ? 1 + two : 2);
        *abort = 0;
        for (int i = 0; i < 8; ++i) bad[i] = 0;
        tc::fence_mbar_init();
    }
    tc::tc_fence_before_sync();
    __syncthreads();
    tc::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    // step it: key tile it, by both halves (kPair) or by half it & 1
    auto works = [&](int w, int it) { return kPair ? w == 0 || two : (it & 1) == w; };

    if (warp >= 8) {
        tc::fewer_registers<kRegsOther>();
        // one warp loads the keys, with which of them are there, and q; one the values
        if ((warp == 9 || warp == 10) && !f.starve) {
            const bool keys = warp == 9, by_page = f.p.page_shift >= 3;
            if (keys && lane == 0) {
                tc::mbar_arrive_expect_tx(q_full, (two ? 2 : 1) * TileShape<D>::kBlocks * rows * 128);
                for (int w = 0; w <= two; ++w)
                    for (int b = 0; b < TileShape<D>::kBlocks; ++b)
                        tc::tma_load_4d(sm + S::kQ + w * S::kTile + b * kBlockBytes, &f.q, b * 64, 0, s.hk,
                                        s.n * f.p.R + i0 + w * tokens, q_full);
            }
            __syncwarp();
            const Boxes<kTileRows> boxes(f);
            uint64_t *full = keys ? k_full : v_full, *free = keys ? k_free : v_free;
            uint8_t *ring = sm + (keys ? S::kK : S::kV);
            const CUtensorMap *map = keys ? &f.k : &f.v;
            const int stages = keys ? S::kStagesK : S::kStagesV;
            int it = 0, page = by_page && steps ? boxes.page(f, s, s.first) : 0;
            for (; it < steps; ++it) {
                const int st = it % stages, use = it / stages, pos = s.first + it * kTileRows;
                const int next = by_page ? boxes.page(f, s, pos + kTileRows) : 0;
                const bool go = !use || tc::mbar_wait(free + st, (use - 1) & 1, abort, f.status, kErrFree, f.spin);
                if (!__all_sync(0xffffffffu, go)) break;
                const int row = by_page ? boxes.row(f, s, pos, page) : 0;
                if (keys) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t there =
                            by_page ? boxes.there(f, s, pos, row, e)
                                    : __ballot_sync(0xffffffffu, pos + 32 * e + lane < s.last &&
                                                                     key_at(f.p, s.table, pos + 32 * e + lane, s.hk) >= 0);
                        if (lane == 0) there_of[it % 8 * 4 + e] = there;
                    }
                }
                if (by_page) load_boxes<D>(boxes, row, map, ring + st * S::kTile, full + st);
                else load_units<D>(f, s, pos, keys ? f.p.k_pages : f.p.v_pages, ring + st * S::kTile, full + st);
                page = next;
            }
            // whatever the other warps do, the copies land before the memory is let go
            if (lane == 0) {
                if (keys) tc::mbar_drain(q_full, 0, f.status, kErrDrain);
                for (int i = max(0, it - stages); i < it; ++i)
                    tc::mbar_drain(full + i % stages, (i / stages) & 1, f.status, kErrDrain);
            }
        }
        // one warp issues for each half
        const int w = warp == 8 ? 0 : warp == 11 && (two || !kPair) ? 1 : -1;
        if (w >= 0) {
            const uint32_t lead = lane == 0;
            const uint32_t q = tc::smem_u32(sm + S::kQ + (kPair ? w : 0) * S::kTile),
                           k = tc::smem_u32(sm + S::kK), v = tc::smem_u32(sm + S::kV);
            const uint32_t s_acc = tmem + S::kTmemS + w * 128, o_acc = tmem + S::kTmemO + w * D;
            constexpr int kEvery = kPair ? 1 : 2;  // steps between two of a half
            auto wait = [&](uint64_t *bar, int n, int code) {
                return __all_sync(0xffffffffu, tc::mbar_wait(bar, n & 1, abort, f.status, code, f.spin));
            };
            bool go = wait(q_full, 0, kErrQ);
            int nth = 0;
            for (int it = kPair ? 0 : w; go; it += kEvery, ++nth) {
                const int st = it % S::kStagesK, last = it - kEvery;
                const int before = (last + S::kStagesV) % S::kStagesV;
                const bool qk = it < steps, pv = nth > 0;  // S of this step, O += P V of the half's last
                go = tc::wait_three(qk ? k_full + st : q_full, qk ? it / S::kStagesK : 0,
                                    pv ? v_full + before : q_full, pv ? last / S::kStagesV : 0,
                                    pv ? p_full + w : q_full, pv ? nth - 1 : 0, abort, f.status, kErrP, f.spin);
                if (!go) break;
                tc::tc_fence_after_sync();
                if (pv) tc::mma_weights_rows<D, 32>(o_acc, s_acc, v + before * S::kTile, nth > 1, lead);
                if (!qk) break;
                tc::mma_rows_rows<D>(s_acc, q, k + st * S::kTile, lead);
                tc::commit(s_full + w, lead);
                tc::commit(k_free + st, lead);
                if (pv) tc::commit(v_free + before, lead);
            }
            tc::commit(o_full, lead);
            tc::mbar_drain(o_full, 0, f.status, kErrDrain);
        }
    } else {
        tc::more_registers<kRegsSoftmax>();
        const unsigned long long *seen = tree_masks<S>(f, s.n, reinterpret_cast<char *>(sm));
        const int w = warp >> 2, in_tile = threadIdx.x & 127;
        // this thread's row: token i (of the sequence's R), head h
        const int i = i0 + (kPair ? w * tokens : 0) + in_tile / G, h = s.hk * G + in_tile % G;
        const bool mine = in_tile < rows && i < f.p.R;
        const unsigned long long see = mine ? seen[i] : 0;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t ts = tmem + lanes + S::kTmemS + w * 128;
        const uint32_t to = tmem + lanes + S::kTmemO + w * D;
        const float c = f.p.scale * kTreeLog2e;
        float m = -INFINITY, l = 0.f;  // reference (unscaled score) and sum
        bool go = true;
        int nth = 0;
        for (int it = 0; it < steps; ++it) {
            if (!works(w, it)) continue;
            go = __all_sync(0xffffffffu, tc::mbar_wait(s_full + w, nth & 1, abort, f.status, kErrS, f.spin));
            if (!go) break;
            tc::tc_fence_after_sync();
            const int pos = s.first + it * kTileRows;
            float x[128];
#pragma unroll
            for (int j = 0; j < 4; ++j) tc::tmem_start(ts + 32 * j, x + 32 * j);
#pragma unroll
            for (int j = 0; j < 4; ++j) tc::tmem_ready(x + 32 * j);
            const uint4 there = *reinterpret_cast<const uint4 *>(there_of + it % 8 * 4);
            const uint32_t real[4] = {there.x, there.y, there.z, there.w};
            if ((real[0] & real[1] & real[2] & real[3]) != ~0u || pos + kTileRows > s.ctx) {
                // what is behind the sequence in its last page is not to meet a weight of 0
                const int st = it % S::kStagesV;
                go = __all_sync(0xffffffffu, tc::mbar_wait(v_full + st, (it / S::kStagesV) & 1, abort, f.status,
                                                           kErrV, f.spin));
                if (!go) break;
                if (!(real[in_tile >> 5] >> (in_tile & 31) & 1)) {
#pragma unroll
                    for (int b = 0; b < TileShape<D>::kBlocks; ++b) {
                        uint4 *row = reinterpret_cast<uint4 *>(sm + S::kV + st * S::kTile + b * kBlockBytes + in_tile * 128);
#pragma unroll
                        for (int u = 0; u < 8; ++u) row[u] = make_uint4(0, 0, 0, 0);
                    }
                }
                tc::fence_proxy_async_smem();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // of 32 keys, the cached ones and the drafts that the row sees
                    const int draft = pos + 32 * e - s.ctx;
                    uint32_t ok;
                    if (draft >= 0) ok = draft < 64 ? (uint32_t)(see >> draft) : 0;
                    else ok = draft <= -32 ? ~0u : ((1u << -draft) - 1) | (uint32_t)(see << -draft);
                    ok &= real[e];
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[32 * e + j] = ok >> j & 1 ? x[32 * e + j] : -INFINITY;
                }
            }
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int j = 4; j < 124; j += 8) {
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = tc::max3(mx[e], x[j + e], x[j + e + 4]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[124 + e]);
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            const bool grown = (top - m) * c > kRescale || m == -INFINITY;
            if (nth == 0) {
                m = top;
            } else if (__any_sync(0xffffffffu, grown)) {
                // this half's products so far were complete before these scores were
                const float m_new = fmaxf(m, top);
                const float keep = m_new == -INFINITY ? 1.f : tc::exp2_fast((m - m_new) * c);
                m = m_new;
                l *= keep;
#pragma unroll
                for (int j = 0; j < D; j += 16) {
                    float y[16];
                    tc::tmem_ld16_sync(to + j, y);
                    uint32_t z[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) z[e] = __float_as_uint(y[e] * keep);
                    tc::tmem_st16(to + j, z);
                }
            }
            const float ref = m == -INFINITY ? 0.f : m * c;
            const tc::f32x2 c2 = tc::pack2(c, c), r2 = tc::pack2(-ref, -ref);
            tc::f32x2 sum = 0;
#pragma unroll
            for (int j = 0; j < 128; j += 32) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float a, b;
                    tc::unpack2(tc::fma2(tc::pack2(x[j + e], x[j + e + 1]), c2, r2), a, b);
                    a = tc::exp2_fast(a);
                    b = tc::exp2_fast(b);
                    sum = tc::add2(sum, tc::pack2(a, b));
                    pk[e / 2] = tc::bf16x2(a, b);
                }
                tc::tmem_st16(ts + j / 2, pk);
            }
            float sa, sb;
            tc::unpack2(sum, sa, sb);
            l += sa + sb;
            tc::tmem_st_wait();
            tc::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(p_full + w);
            ++nth;
        }
        go = __all_sync(0xffffffffu, go && tc::mbar_wait(o_full, 0, abort, f.status, kErrO, f.spin));
        // the sums of the row's halves, in log2 units of the reference
        float2 *odd = reinterpret_cast<float2 *>(sm + S::kMl);
        const bool any = l != 0.f || m != -INFINITY;  // keys it has seen (or NaN among them)
        float by[2] = {1.f, 0.f}, ref = m * c, sum = l;
        bool none = !any;
        if (!kPair) {
            // both warpgroups join the halves and write half of the channels each
            if (w) odd[in_tile] = make_float2(ref, l);
            asm volatile("bar.sync 1, 256;" ::: "memory");
            const float2 b = odd[in_tile];
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (!w) odd[in_tile] = make_float2(ref, l);
            asm volatile("bar.sync 1, 256;" ::: "memory");
            const float2 a = odd[in_tile];
            const bool has_a = a.y != 0.f || a.x != -INFINITY, has_b = b.y != 0.f || b.x != -INFINITY;
            ref = fmaxf(has_a ? a.x : -INFINITY, has_b ? b.x : -INFINITY);
            by[0] = has_a ? tc::exp2_fast(a.x - ref) : 0.f;
            by[1] = has_b ? tc::exp2_fast(b.x - ref) : 0.f;
            sum = (has_a ? a.y * by[0] : 0.f) + (has_b ? b.y * by[1] : 0.f);
            none = !has_a && !has_b;
        }
        const bool absent = see == 0;
        bool redo = false;
        if (go && !*abort) {
            tc::tc_fence_after_sync();
            constexpr int kCols = kPair ? D : D / 2;
            const int col0 = kPair ? 0 : w * kCols;
            const int row = i * G + in_tile % G;
            const size_t part = (((size_t)s.n * f.p.Hkv + s.hk) * f.chunks + s.chunk) * f.rows + row;
            const size_t unit = ((size_t)s.n * f.p.R + i) * f.p.Hq + h;
            const float inv = 1.f / sum;
            float nan = 0.f;
            // what a half without keys left in TMEM is not to meet a weight of 0
            const bool use0 = kPair ? !none : by[0] != 0.f || !(by[0] == by[0]);
            const bool use1 = !kPair && (by[1] != 0.f || !(by[1] == by[1]));
#pragma unroll
            for (int j = 0; j < kCols; j += 16) {
                float y[16];
                tc::tmem_ld16_sync((kPair ? to : tmem + lanes + S::kTmemO) + col0 + j, y);
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = use0 ? y[e] * by[0] : 0.f;
                if (!kPair) {
                    float z[16];
                    tc::tmem_ld16_sync(tmem + lanes + S::kTmemO + D + col0 + j, z);
#pragma unroll
                    for (int e = 0; e < 16; ++e) y[e] = use1 ? fmaf(z[e], by[1], y[e]) : y[e];
                }
                if (!mine) continue;
                if (s.alone) {
                    uint32_t pk[8];
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float a = none || absent ? 0.f : y[e] * inv, b = none || absent ? 0.f : y[e + 1] * inv;
                        nan = fmaf(a, 0.f, fmaf(b, 0.f, nan));
                        pk[e / 2] = tc::bf16x2(a, b);
                    }
                    uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(f.p.o) + unit * D + col0 + j);
                    out[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    out[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                } else {
                    float4 *out = reinterpret_cast<float4 *>(f.part_o + part * D + col0 + j);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        out[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                }
            }
            if (mine && (kPair || w == 0)) {
                if (!s.alone)
                    f.part_ml[part] = none ? make_float2(-INFINITY, 0.f) : make_float2(ref, sum);
                else if (f.p.lse)
                    f.p.lse[unit] = none || absent ? -INFINITY : ref * kTreeLn2 + logf(sum);
            }
            redo = mine && s.alone && !(nan == 0.f);
        }
        const unsigned todo_mine = __ballot_sync(0xffffffffu, redo);
        if (lane == 0 && todo_mine) atomicOr(bad + (kPair ? warp : warp & 3), todo_mine);
        asm volatile("bar.sync 1, 256;" ::: "memory");  // all stores are made
        for (unsigned todo = bad[kPair ? warp : warp & 3]; todo; todo &= todo - 1) {
            const int r = (warp & 3) * 32 + __ffs(todo) - 1;
            if (!kPair && (r & 1) != w) continue;
            redo_row<D>(f, s.n, i0 + (kPair ? w * tokens : 0) + r / G, s.hk * G + r % G);
        }
        tc::tc_fence_before_sync();
    }
    __syncthreads();
    if (warp == 8) {
        tc::tc_fence_after_sync();
        tc::tmem_relinquish();
        tc::tmem_dealloc(tmem, 512);
    }
}

// q [N * R tokens, Hkv, G, D] as a {D, G, Hkv, tokens} tensor, boxes of 64 channels x all
// heads of a group x the tokens of a query tile.
bool encode_query_map(CUtensorMap *tm, const TreeProblem &p, int G, int tokens)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t row = (cuuint64_t)p.d * 2;
    cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)G, (cuuint64_t)p.Hkv, (cuuint64_t)p.N * p.R};
    cuuint64_t strides[3] = {row, row * G, row * p.Hq};
    cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)tokens};
    cuuint32_t estride[4] = {1, 1, 1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p.q), dims, strides, box,
               estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <int D, bool kPair>
cudaError_t start(const TreeParams &f, long long ctas, cudaStream_t st)
{
    using S = TcShape<D, kPair>;
    const cudaError_t e = cudaFuncSetAttribute(
        tree_tc_kernel<D, kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    if (e != cudaSuccess) return e;
    tree_tc_kernel<D, kPair><<<(unsigned)ctas, kThreads, S::kBytes, st>>>(f);
    note_launch();
    return cudaGetLastError();
}

}  // namespace

int tree_tc_rows(const TreeProblem &p)
{
    const int G = p.Hq / p.Hkv;
    if (G > kTileRows) return 0;
    const int tile = kTileRows / G * G;
    return p.R * G > tile ? 2 * tile : tile;
}

cudaError_t launch_tree_tc(const TreeParams &fp, long long ctas, cudaStream_t st)
{
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    TreeParams f = fp;
    const int G = f.p.Hq / f.p.Hkv;
    if (!encode_query_map(&f.q, f.p, G, kTileRows / G)) return cudaErrorInvalidValue;
    const bool pair = f.tile_rows > kTileRows / G * G;
    if (f.p.d == 32) return pair ? start<32, true>(f, ctas, st) : start<32, false>(f, ctas, st);
    if (f.p.d == 64) return pair ? start<64, true>(f, ctas, st) : start<64, false>(f, ctas, st);
    return pair ? start<128, true>(f, ctas, st) : start<128, false>(f, ctas, st);
}

}  // namespace kda
