// kda_attn_bwd.cu — gradients of causal prompt attention on the tensor cores (bf16).
//
// Two kernels recompute P from q, k and lse: one CTA per (128 keys, kv head) sums
// dK and dV over the query tiles behind it and the group's query heads, one CTA per
// (128 queries, head) sums dQ over the key tiles before it. Each output is written by
// one CTA in a fixed order, so results do not depend on timing and no fp32 gradient
// is accumulated in memory; the price is that S and dO V^T are formed twice (7
// products per tile pair instead of 5).
//
// In both, two products give S and dP in TMEM (transposed in the first kernel: a row
// is a key); eight warps turn them into P and dS = P (dP - D) in registers, two
// threads per row with 64 columns each, and write them in bf16 over dP, from where the
// gradient products read them as their TMEM operand; S is free for a later step as soon
// as it has been read. scale is applied to the finished sums.
//
// Roundings: P and dS are operands of bf16 products, each off by at most 2^-8 relative
// to itself and independently of one another, so a sum over them is off by about as much
// as its own rounding to bf16 at the end; D comes from the o that is given, itself
// rounded. Sums, P, dP and D are fp32.
//
// Bound: 16384 tokens, 32 query heads over 8 of 128 channels, forward and backward: 9.4 ms,
// at the power limit. A step of the first kernel takes 3600 cycles, its four products
// 2250; of the second 2700, its three 1710. The rest is the eight warps' arithmetic (P: some
// 1000 cycles of issue per warp, two warps to a scheduler), which the products overlap but
// for the way from dS to the next dP.
//
// 0 times what a masked place holds may be NaN. What lies behind a sequence's end (padding may
// hold anything; o and lse there need not have been written) is cleared in shared memory before
// a product reads it, where it would meet a weight of 0: one warp's stores per tile with an end
// (nine packed documents, forward and gradients: 276 us, without it 272). Rows that tokens of
// the sequence itself make not finite are computed again from the visible pairs alone, at the
// CTA's end, as in the forward.
#include <algorithm>

#include "kda_attn_rows.cuh"
#include "kda_attn_tc.cuh"

namespace kda {
namespace {

constexpr int kThreads = 384;
constexpr int kRegsCompute = 216, kRegsOther = 72;
static_assert(256 * kRegsCompute + 128 * kRegsOther <= kThreads * 168, "register split");
constexpr float kLog2e = 1.44269504088896340736f;

struct BwdParams {
    CUtensorMap q, k, v, dO;
    AttnProblem p;
    const AttnTile *tiles;  // null: uniform sequences
    const float *lse, *lse2, *delta;
    const __nv_bfloat16 *dO_raw;
    __nv_bfloat16 *gq, *gk, *gv;
    int *status;
    uint32_t spin;
    int starve;
    int split;  // dK and dV: CTAs per key tile, see attn_head_split
    int dkv_items, dq_items;
};

// Shared memory: two tiles that stay (k, v or q, dO), and a ring of stages of the two
// tiles that pass (q, dO with their rows' lse2 and D, or k, v).
template <int D, bool kKeys>
struct BwdShape {
    // The first ring's tile is held to the end of its step and read at the next one's
    // beginning: dQ has room for a third.
    static constexpr int kStages = D == 128 ? 2 : 4, kStages0 = D == 128 && !kKeys ? 3 : kStages;
    static constexpr uint32_t kTile = TileShape<D>::kBytes;
    static constexpr uint32_t kStay = 0, kRing0 = 2 * kTile, kRing1 = kRing0 + kStages0 * kTile;
    static constexpr uint32_t kStats = kRing1 + kStages * kTile;  // [stage][lse2, D][128]
    static constexpr uint32_t kBars = kStats + (kKeys ? kStages * 1024 : 0);
    static constexpr uint32_t kBytes = kBars + 320 + 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

enum : int { kErrStay = 111, kErrA, kErrB, kErrFree, kErrS, kErrDp, kErrDs, kErrAcc,
             kErrBwdDrain };

struct Bars {
    uint64_t *stay, *stay_free, *done, *part, *full0, *free0, *full1, *free1, *s_full, *s_free, *dp_full, *ds_full, *acc;
    uint32_t *tmem_slot;
    volatile int *abort;
    volatile uint32_t *odd_rows;  // whether a row is not finite
    __device__ Bars(uint8_t *at)
    {
        constexpr int kMost = 4;  // stages
        stay = reinterpret_cast<uint64_t *>(at);
        stay_free = stay + 1; done = stay + 2; part = stay + 3;
        full0 = stay + 4; free0 = full0 + kMost;
        full1 = free0 + kMost; free1 = full1 + kMost;
        s_full = free1 + kMost; s_free = s_full + 2; dp_full = s_free + 2;
        ds_full = dp_full + 1; acc = ds_full + 1;
        tmem_slot = reinterpret_cast<uint32_t *>(acc + 1);
        abort = reinterpret_cast<volatile int *>(tmem_slot + 1);
        odd_rows = tmem_slot + 2;
    }
};

// full0_count: arrivals that fill a stage of the first ring; warps: that issue products
// (the first ring's stages are freed by all of them).
__device__ __forceinline__ uint32_t start_cta(const Bars &b, int full0_count, int warps)
{
    const int warp = threadIdx.x >> 5;
    if (warp == 8) tc::tmem_alloc(b.tmem_slot, 512);
    if (threadIdx.x == 0) {
        tc::mbar_init(b.stay, 1);
        tc::mbar_init(b.stay_free, warps);
        tc::mbar_init(b.done, warps);
        tc::mbar_init(b.part, 1);
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(b.full0 + i, full0_count);
            tc::mbar_init(b.free0 + i, warps);
            tc::mbar_init(b.full1 + i, 1);
            tc::mbar_init(b.free1 + i, 1);
        }
        tc::mbar_init(b.s_full, 1);
        tc::mbar_init(b.s_full + 1, 1);
        tc::mbar_init(b.s_free, 8);
        tc::mbar_init(b.s_free + 1, 8);
        tc::mbar_init(b.dp_full, 1);
        tc::mbar_init(b.ds_full, 8);
        tc::mbar_init(b.acc, 1);
        *b.abort = 0;
        *b.odd_rows = 0;
        tc::fence_mbar_init();
    }
    tc::tc_fence_before_sync();
    __syncthreads();
    tc::tc_fence_after_sync();
    return *b.tmem_slot;
}

__device__ __forceinline__ void end_cta(uint32_t tmem)
{
    tc::tc_fence_before_sync();
    __syncthreads();
    if (threadIdx.x >> 5 == 8) {
        tc::tc_fence_after_sync();
        tc::tmem_relinquish();
        tc::tmem_dealloc(tmem, 512);
    }
}

// 64 fp32 values of a row as bf16 over 32 columns.
__device__ __forceinline__ void store_weights(uint32_t taddr, const float *x)
{
#pragma unroll
    for (int i = 0; i < 64; i += 32) {
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) pk[j] = tc::bf16x2(x[i + 2 * j], x[i + 2 * j + 1]);
        tc::tmem_st16(taddr + i / 2, pk);
    }
}

// A warp's share of a weights tile is in TMEM.
__device__ __forceinline__ void weights_done(uint64_t *bar)
{
    tc::tmem_st_wait();
    tc::tc_fence_before_sync();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
}

// Row `mine` of an accumulator [128 x D] times `by`, in bf16 to `out` (null: nowhere).
// Returns whether all of it is finite.
template <int D>
__device__ __forceinline__ bool store_sums(uint32_t taddr, float by, __nv_bfloat16 *out)
{
    float odd = 0.f;
#pragma unroll
    for (int i = 0; i < D; i += 32) {
        float x[32];
        tc::tmem_start(taddr + i, x);
        tc::tmem_ready(x);
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            x[j] *= by;
            x[j + 1] *= by;
            odd = fmaf(x[j], 0.f, fmaf(x[j + 1], 0.f, odd));
            pk[j / 2] = tc::bf16x2(x[j], x[j + 1]);
        }
        if (out) {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                *reinterpret_cast<uint4 *>(out + i + 2 * j) =
                    make_uint4(pk[j], pk[j + 1], pk[j + 2], pk[j + 3]);
        }
    }
    return odd == 0.f;
}

// Behind all items: whether any of the CTA's eight warps had a row that is not finite, and
// none has given up.
__device__ __forceinline__ bool any_odd_rows(const Bars &b, bool odd)
{
    if (odd) *b.odd_rows = 1;
    asm volatile("bar.sync 1, 256;" ::: "memory");
    return *b.odd_rows && !*b.abort;
}

template <int D>
__device__ __noinline__ void redo_dkv(const BwdParams &f, int col, int end, int hk)
{
    attn_row_dkv<__nv_bfloat16, D>(f.p, col, end, hk, f.lse, f.delta, f.dO_raw, f.gk, f.gv);
}

template <int D>
__device__ __noinline__ void redo_dq(const BwdParams &f, int row, int start, int h)
{
    attn_row_dq<__nv_bfloat16, D>(f.p, row, start, h, f.lse, f.delta, f.dO_raw, f.gq);
}

// ---------------------------------------------------------------- dK and dV
// An item: a key tile and its kv head; its steps are (query head, query tile). Persistent
// CTAs take items in order of falling work, a cluster that shares one out takes one.
struct KeyItem {
    int hk, first, seq_end, per_head, steps;
    __device__ __forceinline__ bool get(const BwdParams &f, int n, int rank)
    {
        const int idx = f.split == 1 ? nth_item(n, f.dkv_items) : n ? -1 : blockIdx.x / f.split;
        if (idx < 0) return false;
        const AttnTile t = attn_tile(f.tiles, idx / f.p.Hkv, kTileRows, f.p.B, f.p.T);
        if (t.first >= t.seq_end) return false;  // the list's unused end
        hk = idx % f.p.Hkv;
        seq_end = t.seq_end;
        // the list begins with a sequence's last tile; here the first one has most work
        const int count = (t.seq_end - t.seq_start + kTileRows - 1) / kTileRows;
        const int tile = count - 1 - (t.first - t.seq_start) / kTileRows;
        first = t.seq_start + tile * kTileRows;
        const int G = f.p.Hq / f.p.Hkv, heads = (G - rank + f.split - 1) / f.split;
        per_head = count - tile;
        steps = per_head * heads;
        return true;
    }
    // query head and first token of a step; the heads of a cluster's CTAs: rank, rank + split, ...
    __device__ __forceinline__ int head(const BwdParams &f, int it, int rank) const
    {
        return hk * (f.p.Hq / f.p.Hkv) + rank + it / per_head * f.split;
    }
    __device__ __forceinline__ int token(int it) const { return first + it % per_head * kTileRows; }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_dkv_kernel(const __grid_constant__ BwdParams f)
{
    using S = BwdShape<D, true>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const Bars b(sm + S::kBars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = f.split > 1 ? cluster_rank() : 0;
    if (!f.tiles && blockIdx.x == 0 && threadIdx.x == 0) *f.status = 0;
    let_next_start();
    KeyItem t;
    if (f.split > 1 && !t.get(f, 0, rank)) return;  // all of a cluster

    const uint32_t tmem = start_cta(b, 1 + 32, 2);
    constexpr uint32_t kS = 0, kDp = 128, kDv = 256, kDk = 256 + D;
    const float *stats = reinterpret_cast<const float *>(sm + S::kStats);

    if (warp >= 8) {
        tc::fewer_registers<kRegsOther>();
        if (warp == 9 && !f.starve) {
            int g0 = 0, g = 0, n = 0, parts = 0;  // stages filled in either ring, items begun, tiles cleared
            bool go = true;
            for (; go && t.get(f, n, rank); ++n) {
                if (n && !__all_sync(0xffffffffu, tc::mbar_wait(b.stay_free, (n - 1) & 1, b.abort, f.status, kErrFree, f.spin)))
                    break;
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(b.stay, 2 * S::kTile);
                    tc::load_tile<D>(sm + S::kStay, &f.k, t.hk, t.first, b.stay);
                    tc::load_tile<D>(sm + S::kStay + S::kTile, &f.v, t.hk, t.first, b.stay);
                }
                auto wait_free = [&](uint64_t *bar, int use) {
                    return !use || __all_sync(0xffffffffu, tc::mbar_wait(bar, (use - 1) & 1, b.abort, f.status, kErrFree, f.spin));
                };
                for (int it = 0; it < t.steps; ++it) {
                    const int st = g0 % S::kStages, use = g0 / S::kStages;
                    const int h = t.head(f, it, rank), token = t.token(it);
                    if (!(go = wait_free(b.free0 + st, use))) break;
                    float *to = reinterpret_cast<float *>(sm + S::kStats) + st * 256;
                    const size_t base = (size_t)h * f.p.tokens;
#pragma unroll
                    for (int i = lane; i < kTileRows; i += 32) {
                        // behind the sequence nobody may have written lse and o: 0 there
                        const bool real = token + i < t.seq_end;
                        const size_t at = base + (real ? token + i : token);
                        tc::cp_async4(to + i, f.lse2 + at, real);
                        tc::cp_async4(to + 128 + i, f.delta + at, real);
                    }
                    tc::cp_async_arrive(b.full0 + st);
                    if (t.seq_end - token < kTileRows) {
                        // A tile with the sequence's end is passed on without what lies behind it.
                        if (!(go = wait_free(b.free1 + st, use))) break;
                        uint8_t *q = sm + S::kRing0 + st * S::kTile, *dO = sm + S::kRing1 + st * S::kTile;
                        if (lane == 0) {
                            tc::mbar_arrive_expect_tx(b.part, 2 * S::kTile);
                            tc::load_tile<D>(q, &f.q, h, token, b.part);
                            tc::load_tile<D>(dO, &f.dO, h, token, b.part);
                        }
                        __syncwarp();
                        ++parts;
                        go = __all_sync(0xffffffffu, tc::mbar_wait(b.part, (parts - 1) & 1, b.abort, f.status, kErrB, f.spin));
                        if (!go) break;
                        clear_rows<D>(q, t.seq_end - token, kTileRows);
                        clear_rows<D>(dO, t.seq_end - token, kTileRows);
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tc::mbar_arrive(b.full0 + st);
                            tc::mbar_arrive(b.full1 + st);
                        }
                        ++g0;
                        ++g;
                        continue;
                    }
                    if (lane == 0) {
                        tc::mbar_arrive_expect_tx(b.full0 + st, S::kTile);
                        tc::load_tile<D>(sm + S::kRing0 + st * S::kTile, &f.q, h, token, b.full0 + st);
                    }
                    __syncwarp();
                    ++g0;
                    if (!(go = wait_free(b.free1 + st, use))) break;
                    if (lane == 0) {
                        tc::mbar_arrive_expect_tx(b.full1 + st, S::kTile);
                        tc::load_tile<D>(sm + S::kRing1 + st * S::kTile, &f.dO, h, token, b.full1 + st);
                    }
                    __syncwarp();
                    ++g;
                }
            }
            tc::cp_async_wait_all();
            if (lane == 0) {  // whatever the other warps do, the copies land before the memory is let go
                if (n) tc::mbar_drain(b.stay, (n - 1) & 1, f.status, kErrBwdDrain);
                if (parts) tc::mbar_drain(b.part, (parts - 1) & 1, f.status, kErrBwdDrain);
                for (int i = max(0, g0 - S::kStages); i < g0; ++i)
                    tc::mbar_drain(b.full0 + i % S::kStages, (i / S::kStages) & 1, f.status, kErrBwdDrain);
                for (int i = max(0, g - S::kStages); i < g; ++i)
                    tc::mbar_drain(b.full1 + i % S::kStages, (i / S::kStages) & 1, f.status, kErrBwdDrain);
            }
        }
        // Warp 8 issues dK, dV and the next dP when P and dS are there, warp 10 S as soon as
        // the step before has read its place. What a product reads in TMEM a later one
        // overwrites, in the order of issue. (One warp for all: its polls and commits, 1100
        // cycles of a step, add to the products' 2250.)
        if (warp == 8 || warp == 10) {
            const uint32_t lead = lane == 0;
            const uint32_t k = tc::smem_u32(sm + S::kStay), v = k + S::kTile;
            const uint32_t q = tc::smem_u32(sm + S::kRing0), dO = tc::smem_u32(sm + S::kRing1);
            auto wait = [&](uint64_t *x, int nx, uint64_t *y, int ny, int code) {
                return tc::wait_both(x, nx, y, ny, b.abort, f.status, code, f.spin);
            };
            int g = 0;  // steps of all items
            bool go = true;
            for (int n = 0; go && t.get(f, n, rank); ++n) {
                const int begin = g, end = g + t.steps;
                go = wait(b.stay, n, b.stay, n, kErrStay);
                if (warp == 10) {
                    for (; g < end && go; ++g) {
                        const int st = g % S::kStages, use = g / S::kStages;
                        go = wait(b.full0 + st, use, g ? b.s_free : b.full0 + st, g ? g - 1 : use, kErrA);
                        if (!go) break;
                        tc::tc_fence_after_sync();
                        tc::mma_rows_rows<D>(tmem + kS, k, q + st * S::kTile, lead);
                        tc::commit(b.s_full, lead);
                        tc::commit(b.free0 + st, lead);
                        if (g + 1 == end) tc::commit(b.stay_free, lead);
                    }
                    continue;
                }
                for (; g <= end && go; ++g) {  // dK and dV of step g - 1 and dP of step g
                    const int st = g % S::kStages, use = g / S::kStages, before = (g + S::kStages - 1) % S::kStages;
                    const bool dp = g < end, sums = g > begin;
                    // dS says that the step's S was formed, so that its queries are there
                    go = !sums ? wait(b.full1 + st, use, b.full1 + st, use, kErrB)
                         : !dp ? wait(b.ds_full, g - 1, b.ds_full, g - 1, kErrDs)
                               : wait(b.full1 + st, use, b.ds_full, g - 1, kErrDs);
                    if (!go) break;
                    tc::tc_fence_after_sync();
                    if (sums) {
                        tc::mma_weights_rows<D, 64>(tmem + kDk, tmem + kDp + 32, q + before * S::kTile, g - 1 > begin, lead);
                        tc::commit(b.free0 + before, lead);
                        tc::mma_weights_rows<D, 64>(tmem + kDv, tmem + kDp, dO + before * S::kTile, g - 1 > begin, lead);
                    }
                    if (dp) {
                        tc::mma_rows_rows<D>(tmem + kDp, v, dO + st * S::kTile, lead);
                        tc::commit(b.dp_full, lead);
                        if (g + 1 == end) tc::commit(b.stay_free, lead);
                    }
                    if (sums) tc::commit(b.free1 + before, lead);
                }
                g = end;  // the next item's first dP comes with no sums
                if (go) tc::commit(b.acc, lead);
            }
            tc::commit(b.done, lead);
            tc::mbar_drain(b.done, 0, f.status, kErrBwdDrain);
        }
    } else {
        tc::more_registers<kRegsCompute>();
        const int half = warp >> 2, in_tile = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t ts = tmem + lanes + kS + half * 64, td = tmem + lanes + kDp + half * 64;
        const float c = f.p.scale * kLog2e;
        const tc::f32x2 c2 = tc::pack2(c, c);
        bool go = true, odd_rows = false;
        int g = 0;  // steps of all items
        for (int n = 0; t.get(f, n, rank); ++n) {
            for (int it = 0; it < t.steps && go; ++it, ++g) {
                const int st = g % S::kStages, i0 = it % t.per_head;
                const float *lse2 = stats + st * 256 + half * 64, *del = lse2 + 128;
                go = __all_sync(0xffffffffu,
                                tc::mbar_wait(b.s_full, g & 1, b.abort, f.status, kErrS, f.spin) &&
                                tc::mbar_wait(b.full0 + st, (g / S::kStages) & 1, b.abort, f.status, kErrA, f.spin));
                if (!go) break;
                tc::tc_fence_after_sync();
                float x[64];
                tc::tmem_start(ts, x);
                tc::tmem_start(ts + 32, x + 32);
                tc::tmem_ready(x);
                tc::tmem_ready(x + 32);
                tc::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(b.s_free);
#pragma unroll
                for (int j = 0; j < 64; j += 4) {
                    const float4 z = *reinterpret_cast<const float4 *>(lse2 + j);
                    tc::unpack2(tc::fma2(tc::pack2(x[j], x[j + 1]), c2, tc::pack2(-z.x, -z.y)), x[j], x[j + 1]);
                    tc::unpack2(tc::fma2(tc::pack2(x[j + 2], x[j + 3]), c2, tc::pack2(-z.z, -z.w)), x[j + 2], x[j + 3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[j + e] = tc::exp2_fast(x[j + e]);
                }
                // queries before the key, or behind the sequence
                const int behind = t.seq_end - (t.first + i0 * kTileRows) - half * 64;
                const int before = i0 == 0 ? in_tile - half * 64 : 0;
                if (i0 == 0 || behind < 64) {
#pragma unroll
                    for (int j = 0; j < 64; ++j) x[j] = j >= before && j < behind ? x[j] : 0.f;
                }
                go = __all_sync(0xffffffffu, tc::mbar_wait(b.dp_full, g & 1, b.abort, f.status, kErrDp, f.spin));
                if (!go) break;
                tc::tc_fence_after_sync();
                float y[64];
                tc::tmem_start(td, y);
                tc::tmem_start(td + 32, y + 32);
                tc::tmem_ready(y);
                tc::tmem_ready(y + 32);
                store_weights(td, x);  // P and dS take the place of the half's dP
#pragma unroll
                for (int j = 0; j < 64; j += 4) {
                    const float4 z = *reinterpret_cast<const float4 *>(del + j);
                    tc::unpack2(tc::mul2(tc::pack2(x[j], x[j + 1]),
                                         tc::add2(tc::pack2(y[j], y[j + 1]), tc::pack2(-z.x, -z.y))), x[j], x[j + 1]);
                    tc::unpack2(tc::mul2(tc::pack2(x[j + 2], x[j + 3]),
                                         tc::add2(tc::pack2(y[j + 2], y[j + 3]), tc::pack2(-z.z, -z.w))),
                                x[j + 2], x[j + 3]);
                }
                store_weights(td + 32, x);
                weights_done(b.ds_full);
            }
            go = __all_sync(0xffffffffu, go && tc::mbar_wait(b.acc, n & 1, b.abort, f.status, kErrAcc, f.spin));
            const int col = t.first + in_tile;
            const bool mine = col < t.seq_end;
            const bool fine = __all_sync(0xffffffffu, go && !*b.abort);
            bool bad = false;
            // the first four warps write dV, the others dK
            const uint32_t sums = tmem + lanes + (half ? kDk : kDv);
            const float by = half ? f.p.scale : 1.f;
            __nv_bfloat16 *out = (half ? f.gk : f.gv) + ((size_t)col * f.p.Hkv + t.hk) * D;
            if (fine) tc::tc_fence_after_sync();
            if (f.split == 1) {
                if (fine) bad = !store_sums<D>(sums, by, mine ? out : nullptr) && mine;
            } else {
                // every CTA lays its sums out over its ring (all copies and products are done)
                // and finishes its share of the channels, adding in rank order
                float *own = reinterpret_cast<float *>(sm) + half * 128 * D + in_tile;
                if (fine) {
#pragma unroll
                    for (int i = 0; i < D; i += 32) {
                        float x[32];
                        tc::tmem_start(sums + i, x);
                        tc::tmem_ready(x);
#pragma unroll
                        for (int j = 0; j < 32; ++j) own[(i + j) * 128] = x[j];
                    }
                }
                cluster_sync();
                const int share = D / f.split;
                const uint32_t from = tc::smem_u32(own);
                float odd = 0.f;
                for (int i = rank * share; i < (rank + 1) * share; i += 8) {
                    float x[8] = {};
                    for (int r = 0; r < f.split; ++r) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] += peer_float(from + (i + j) * 512, r);
                    }
                    uint32_t pk[4];
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        odd = fmaf(x[j], 0.f, fmaf(x[j + 1], 0.f, odd));
                        pk[j / 2] = tc::bf16x2(x[j] * by, x[j + 1] * by);
                    }
                    if (mine && fine) *reinterpret_cast<uint4 *>(out + i) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
                bad = mine && fine && !(odd == 0.f);
                cluster_sync();  // all reads and stores are made
            }
            odd_rows |= bad;
            if (!fine) break;
        }
        if (any_odd_rows(b, odd_rows))
            for (int n = 0; t.get(f, n, rank); ++n)
                for (int col = t.first + warp; col < min(t.first + kTileRows, t.seq_end); col += 8) {
                    const size_t at = ((size_t)col * f.p.Hkv + t.hk) * D;
                    if (!row_finite<__nv_bfloat16, D>(f.gk + at) || !row_finite<__nv_bfloat16, D>(f.gv + at))
                        redo_dkv<D>(f, col, t.seq_end, t.hk);
                }
    }
    if (warp >= 8 && f.split > 1) {
        __syncwarp();
        cluster_sync();
        cluster_sync();
    }
    end_cta(tmem);
}

// ---------------------------------------------------------------- dQ
// An item: a query tile and its head; its steps are the key tiles, the diagonal's first.
// Launched early behind dK and dV, of which it needs nothing: its CTAs, two for each SM
// to fill in where there is room, start as the SMs run out of key tiles, and only must
// not end before those do.
struct QueryItem {
    int h, first, seq_start, seq_end, last, steps;
    __device__ __forceinline__ bool get(const BwdParams &f, int n)
    {
        const int idx = nth_item(n, f.dq_items);
        if (idx < 0) return false;
        const AttnTile t = attn_tile(f.tiles, idx / f.p.Hq, kTileRows, f.p.B, f.p.T);
        if (t.first >= t.seq_end) return false;  // the list's unused end
        h = idx % f.p.Hq;
        first = t.first; seq_start = t.seq_start; seq_end = t.seq_end;
        last = (first - seq_start) / kTileRows;
        steps = last + 1;
        return true;
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_dq_kernel(const __grid_constant__ BwdParams f)
{
    using S = BwdShape<D, false>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const Bars b(sm + S::kBars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    QueryItem t;

    const uint32_t tmem = start_cta(b, 1, 2);
    constexpr uint32_t kS = 0, kDp = 256, kDq = 384;  // two score tiles in turn

    if (warp >= 8) {
        tc::fewer_registers<kRegsOther>();
        if (warp == 9 && lane == 0 && !f.starve) {
            int g0 = 0, g = 0, n = 0;  // stages filled in either ring, items begun
            bool go = true;
            for (; go && t.get(f, n); ++n) {
                const int hk = t.h / (f.p.Hq / f.p.Hkv);
                if (n && !tc::mbar_wait(b.stay_free, (n - 1) & 1, b.abort, f.status, kErrFree, f.spin)) break;
                tc::mbar_arrive_expect_tx(b.stay, 2 * S::kTile);
                tc::load_tile<D>(sm + S::kStay, &f.q, t.h, t.first, b.stay);
                tc::load_tile<D>(sm + S::kStay + S::kTile, &f.dO, t.h, t.first, b.stay);
                for (int it = 0; it < t.steps; ++it) {
                    const int st0 = g0 % S::kStages0, use0 = g0 / S::kStages0;
                    const int st = g % S::kStages, use = g / S::kStages;
                    const int token = t.seq_start + (t.last - it) * kTileRows;
                    go = !use0 || tc::mbar_wait(b.free0 + st0, (use0 - 1) & 1, b.abort, f.status, kErrFree, f.spin);
                    if (!go) break;
                    tc::mbar_arrive_expect_tx(b.full0 + st0, S::kTile);
                    tc::load_tile<D>(sm + S::kRing0 + st0 * S::kTile, &f.k, hk, token, b.full0 + st0);
                    ++g0;
                    go = !use || tc::mbar_wait(b.free1 + st, (use - 1) & 1, b.abort, f.status, kErrFree, f.spin);
                    if (!go) break;
                    tc::mbar_arrive_expect_tx(b.full1 + st, S::kTile);
                    tc::load_tile<D>(sm + S::kRing1 + st * S::kTile, &f.v, hk, token, b.full1 + st);
                    ++g;
                }
            }
            // whatever the other warps do, the copies land before the memory is let go
            if (n) tc::mbar_drain(b.stay, (n - 1) & 1, f.status, kErrBwdDrain);
            for (int i = max(0, g0 - S::kStages0); i < g0; ++i)
                tc::mbar_drain(b.full0 + i % S::kStages0, (i / S::kStages0) & 1, f.status, kErrBwdDrain);
            for (int i = max(0, g - S::kStages); i < g; ++i)
                tc::mbar_drain(b.full1 + i % S::kStages, (i / S::kStages) & 1, f.status, kErrBwdDrain);
        }
        // warp 8 issues S, two steps ahead, warp 10 dP and dQ
        if (warp == 8 || warp == 10) {
            const uint32_t lead = lane == 0;
            const uint32_t q = tc::smem_u32(sm + S::kStay), dO = q + S::kTile;
            const uint32_t k = tc::smem_u32(sm + S::kRing0), v = tc::smem_u32(sm + S::kRing1);
            auto wait = [&](uint64_t *x, int nx, uint64_t *y, int ny, int code) {
                return tc::wait_both(x, nx, y, ny, b.abort, f.status, code, f.spin);
            };
            int g = 0;  // steps of all items
            bool go = true;
            for (int n = 0; go && t.get(f, n); ++n) {
                const int begin = g, end = g + t.steps;
                go = wait(b.stay, n, b.stay, n, kErrStay);
                if (warp == 8) {
                    for (; g < end && go; ++g) {
                        uint64_t *keys = b.full0 + g % S::kStages0;
                        const int use = g / S::kStages0;
                        // its buffer was read (the first two steps have none to wait for)
                        go = g < 2 ? wait(keys, use, keys, use, kErrA)
                                   : wait(keys, use, b.s_free + (g & 1), (g >> 1) - 1, kErrA);
                        if (!go) break;
                        tc::tc_fence_after_sync();
                        tc::mma_rows_rows<D>(tmem + kS + (g & 1) * 128, q, k + g % S::kStages0 * S::kTile, lead);
                        tc::commit(b.s_full + (g & 1), lead);
                        tc::commit(b.free0 + g % S::kStages0, lead);
                        if (g + 1 == end) tc::commit(b.stay_free, lead);
                    }
                } else {
                    for (; g <= end && go; ++g) {  // dQ of step g - 1 and dP of step g
                        uint64_t *values = b.full1 + g % S::kStages;
                        const int use = g / S::kStages;
                        const bool dp = g < end, dq = g > begin;
                        // dS says that the step's S was formed, so that its keys are there
                        go = !dq   ? wait(values, use, values, use, kErrB)
                             : !dp ? wait(b.ds_full, g - 1, b.ds_full, g - 1, kErrDs)
                                   : wait(values, use, b.ds_full, g - 1, kErrDs);
                        if (!go) break;
                        tc::tc_fence_after_sync();
                        const int st0 = (g + S::kStages0 - 1) % S::kStages0;
                        if (dq) tc::mma_weights_rows<D, 64>(tmem + kDq, tmem + kDp, k + st0 * S::kTile, g - 1 > begin, lead);
                        if (dp) {
                            tc::mma_rows_rows<D>(tmem + kDp, dO, v + g % S::kStages * S::kTile, lead);
                            tc::commit(b.dp_full, lead);
                            tc::commit(b.free1 + g % S::kStages, lead);
                            if (g + 1 == end) tc::commit(b.stay_free, lead);
                        }
                        if (dq) tc::commit(b.free0 + st0, lead);
                    }
                    g = end;  // the next item's first dP comes with no dQ
                    if (go) tc::commit(b.acc, lead);
                }
            }
            tc::commit(b.done, lead);
            tc::mbar_drain(b.done, 0, f.status, kErrBwdDrain);
        }
    } else {
        tc::more_registers<kRegsCompute>();
        const int half = warp >> 2, in_tile = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t ts = tmem + lanes + kS + half * 64, td = tmem + lanes + kDp + half * 64;
        const float c = f.p.scale * kLog2e;
        const tc::f32x2 c2 = tc::pack2(c, c);
        bool go = true, odd_rows = false;
        int g = 0;  // steps of all items
        for (int n = 0; t.get(f, n); ++n) {
            const int row = t.first + in_tile;
            const bool mine = row < t.seq_end;
            const size_t at = (size_t)t.h * f.p.tokens + min(row, (int)f.p.tokens - 1);
            const float z = f.lse2[at], del = f.delta[at];
            const tc::f32x2 z2 = tc::pack2(-z, -z), d2 = tc::pack2(-del, -del);
            for (int it = 0; it < t.steps && go; ++it, ++g) {
                go = __all_sync(0xffffffffu, tc::mbar_wait(b.s_full + (g & 1), (g >> 1) & 1, b.abort, f.status,
                                                           kErrS, f.spin));
                if (!go) break;
                tc::tc_fence_after_sync();
                float x[64];
                tc::tmem_start(ts + (g & 1) * 128, x);
                tc::tmem_start(ts + (g & 1) * 128 + 32, x + 32);
                tc::tmem_ready(x);
                tc::tmem_ready(x + 32);
                tc::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(b.s_free + (g & 1));
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    tc::unpack2(tc::fma2(tc::pack2(x[j], x[j + 1]), c2, z2), x[j], x[j + 1]);
                    x[j] = tc::exp2_fast(x[j]);
                    x[j + 1] = tc::exp2_fast(x[j + 1]);
                }
                if (it == 0 && t.seq_end - t.first < kTileRows) {  // S is there, so k can be written
                    clear_rows<D>(sm + S::kRing0 + g % S::kStages0 * S::kTile, max(t.seq_end - t.first, warp * 16),
                                  warp * 16 + 16);
                    tc::fence_proxy_async_smem();
                }
                go = __all_sync(0xffffffffu, tc::mbar_wait(b.dp_full, g & 1, b.abort, f.status, kErrDp, f.spin));
                if (!go) break;
                tc::tc_fence_after_sync();
                float y[64];
                tc::tmem_start(td, y);
                tc::tmem_start(td + 32, y + 32);
                tc::tmem_ready(y);
                tc::tmem_ready(y + 32);
#pragma unroll
                for (int j = 0; j < 64; j += 2)
                    tc::unpack2(tc::mul2(tc::pack2(x[j], x[j + 1]), tc::add2(tc::pack2(y[j], y[j + 1]), d2)),
                                x[j], x[j + 1]);
                if (it == 0) {  // the diagonal tile: P, and dP where it is not finite
#pragma unroll
                    for (int j = 0; j < 64; ++j) x[j] = j + half * 64 <= in_tile ? x[j] : 0.f;
                }
                store_weights(td, x);
                weights_done(b.ds_full);
            }
            go = __all_sync(0xffffffffu, go && tc::mbar_wait(b.acc, n & 1, b.abort, f.status, kErrAcc, f.spin));
            const bool fine = __all_sync(0xffffffffu, go && !*b.abort);
            bool bad = false;
            if (fine) {
                tc::tc_fence_after_sync();
                // each half of the warps writes half of the row's channels
                __nv_bfloat16 *out = f.gq + ((size_t)row * f.p.Hq + t.h) * D;
                constexpr int kPart = D == 32 ? 32 : D / 2;
                if (D > 32 || half == 0)
                    bad = !store_sums<kPart>(tmem + lanes + kDq + half * kPart, f.p.scale,
                                             mine ? out + half * kPart : nullptr) && mine;
            }
            odd_rows |= bad;
            if (!fine) break;
        }
        if (any_odd_rows(b, odd_rows))
            for (int n = 0; t.get(f, n); ++n)
                for (int row = t.first + warp; row < min(t.first + kTileRows, t.seq_end); row += 8)
                    if (!row_finite<__nv_bfloat16, D>(f.gq + ((size_t)row * f.p.Hq + t.h) * D))
                        redo_dq<D>(f, row, t.seq_start, t.h);
    }
    wait_for_previous();
    end_cta(tmem);
}

// ---------------------------------------------------------------- D and lse log2 e
// D / 8 threads (or D / 4, fp32) per row, 16 bytes each.
template <typename T, int D>
__global__ void __launch_bounds__(256)
attn_delta_kernel(const T *o, const float *lse, const T *dO, long long tokens, int Hq,
                  float *delta, float *lse2)
{
    constexpr int kPer = 16 / sizeof(T), kLanes = D / kPer;
    const long long row = ((long long)blockIdx.x * 256 + threadIdx.x) / kLanes;
    const int part = threadIdx.x % kLanes;
    const bool in = row < tokens * Hq;
    float s = 0.f;
    if (in) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(o) + row * kLanes + part);
        const uint4 g = __ldg(reinterpret_cast<const uint4 *>(dO) + row * kLanes + part);
        const T *x = reinterpret_cast<const T *>(&a), *y = reinterpret_cast<const T *>(&g);
#pragma unroll
        for (int i = 0; i < kPer; ++i) s = fmaf(to_f32(x[i]), to_f32(y[i]), s);
    }
#pragma unroll
    for (int m = kLanes / 2; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (in && part == 0) {
        const long long at = row % Hq * tokens + row / Hq;
        delta[at] = s;
        lse2[at] = lse[row] * kLog2e;
    }
}

template <typename T, int D>
cudaError_t launch_delta(const AttnProblem &p, const void *o, const float *lse, const void *dO,
                         float *delta, float *lse2, cudaStream_t st)
{
    constexpr int kLanes = D * sizeof(T) / 16;
    const long long threads = p.tokens * p.Hq * kLanes;
    attn_delta_kernel<T, D><<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(
        static_cast<const T *>(o), lse, static_cast<const T *>(dO), p.tokens, p.Hq, delta, lse2);
    note_launch();
    return cudaGetLastError();
}

template <int D>
cudaError_t launch(const AttnProblem &p, const void *o, const float *lse, const void *dO,
                   void *gq, void *gk, void *gv, void *workspace, cudaStream_t st)
{
    char *ws = static_cast<char *>(workspace);
    const AttnWorkspace w = attn_workspace_layout(p, kTileRows, true);
    BwdParams f{};
    f.p = p;
    float *delta = reinterpret_cast<float *>(ws + w.delta);
    f.delta = delta;
    f.lse2 = delta + (size_t)p.tokens * p.Hq;
    f.lse = lse;
    f.dO_raw = static_cast<const __nv_bfloat16 *>(dO);
    f.gq = static_cast<__nv_bfloat16 *>(gq);
    f.gk = static_cast<__nv_bfloat16 *>(gk);
    f.gv = static_cast<__nv_bfloat16 *>(gv);
    f.status = reinterpret_cast<int *>(ws);
    const DebugKnobs dbg = debug_knobs();
    f.spin = dbg.wait_limit ? dbg.wait_limit : tc::kSpinLimit;
    f.starve = dbg.starve_carry;
    if (!encode_attn_map(&f.q, p.q, p.Hq, D, p.tokens) ||
        !encode_attn_map(&f.k, p.k, p.Hkv, D, p.tokens) ||
        !encode_attn_map(&f.v, p.v, p.Hkv, D, p.tokens) ||
        !encode_attn_map(&f.dO, dO, p.Hq, D, p.tokens))
        return cudaErrorInvalidValue;
    cudaError_t e;
    if (p.cu_seqlens) {
        f.tiles = reinterpret_cast<const AttnTile *>(ws + w.tiles);
        if ((e = launch_attn_plan(p, kTileRows, workspace, st)) != cudaSuccess) return e;
    }
    e = launch_attn_delta(p, o, lse, dO, delta, delta + (size_t)p.tokens * p.Hq, st);
    if (e != cudaSuccess) return e;
    const long long tiles = attn_tiles(p, kTileRows);
    constexpr uint32_t dkv_smem = BwdShape<D, true>::kBytes, dq_smem = BwdShape<D, false>::kBytes;
    f.split = attn_head_split(p, kTileRows, 148);
    f.dkv_items = (int)(tiles * p.Hkv);
    f.dq_items = (int)(tiles * p.Hq);
    e = launch_kernel(attn_dkv_kernel<D>, f, f.split > 1 ? f.dkv_items : std::min(f.dkv_items, 148), kThreads,
                      dkv_smem, f.split, false, st);
    if (e != cudaSuccess) return e;
    return launch_kernel(attn_dq_kernel<D>, f, std::min(f.dq_items, 148 * 2), kThreads, dq_smem, 1, true, st);
}

}  // namespace

int attn_tc_bwd_rows() { return kTileRows; }

cudaError_t launch_attn_delta(const AttnProblem &p, const void *o, const float *lse,
                              const void *dO, float *delta, float *lse2, cudaStream_t st)
{
    if (p.dtype == KDA_DTYPE_F32) {
        if (p.d == 32) return launch_delta<float, 32>(p, o, lse, dO, delta, lse2, st);
        if (p.d == 64) return launch_delta<float, 64>(p, o, lse, dO, delta, lse2, st);
        return launch_delta<float, 128>(p, o, lse, dO, delta, lse2, st);
    }
    if (p.d == 32) return launch_delta<__nv_bfloat16, 32>(p, o, lse, dO, delta, lse2, st);
    if (p.d == 64) return launch_delta<__nv_bfloat16, 64>(p, o, lse, dO, delta, lse2, st);
    return launch_delta<__nv_bfloat16, 128>(p, o, lse, dO, delta, lse2, st);
}

cudaError_t launch_attn_tc_bwd(const AttnProblem &p, const void *o, const float *lse,
                               const void *dO, void *gq, void *gk, void *gv, void *workspace,
                               cudaStream_t st)
{
    if (p.d == 32) return launch<32>(p, o, lse, dO, gq, gk, gv, workspace, st);
    if (p.d == 64) return launch<64>(p, o, lse, dO, gq, gk, gv, workspace, st);
    return launch<128>(p, o, lse, dO, gq, gk, gv, workspace, st);
}

}  // namespace kda
