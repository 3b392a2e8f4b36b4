// kda_attn_fwd.cu — causal prompt attention on the tensor cores (bf16, d = 32, 64, 128).
//
// A work item is two query tiles of 128 rows that share the key/value tiles, walked from
// the diagonal down to the sequence's first tile: 128 tokens of two heads of one key/value
// head where those come in pairs, else 256 tokens of one head, whose first tile sits out
// a step and whose second is absent from every other sequence's end (24 packed prompts
// of up to 700 tokens, 16 heads: 44 us, 47 without the pairs). One persistent CTA per SM
// takes items in order of falling work; its loads and products run on into the next item
// while the rows of the last one are written. (With a CTA per item, beginning and end cost
// 8 us of an SM, as much as five steps.)
//
// Per tile pair S = Q K^T goes to TMEM, one thread per row turns it into
// P = 2^(c s - c m) (c = scale log2 e, m the row's running reference) in registers,
// writes P in bf16 over S, and O += P V reads it from there. Warps 0-3 own the rows of
// query tile 0, warps 4-7 those of tile 1; warps 8 and 10 issue the MMAs of a tile each;
// warp 9 loads, warp 11 clears values behind a sequence's end. A step goes in halves of 64
// keys: the first half's P V and next S run while the second half is in the softmax.
//
// Bound: 32768 tokens, 32 query heads over 8 of 128 channels: 8.5 ms, 1.03 PFLOP/s, 0.63 of
// the measured burst rate and, at the power limit where such a call runs, 0.75 of the
// sustained one. A step of both tiles takes about 3900 cycles: 64-wide products of S cost
// as much as 128-wide ones (645 cycles a half, as all of Q is read either way), 3650 in
// all, and the softmax issues for some 1000 cycles per 64 keys and warp, two warps to a
// scheduler, half of that in 2^x. One 128-wide product of S costs less but waits for both
// halves of P: 10.0 ms.
//
// The reference m moves only when the row maximum has grown by more than 2^8 in
// weight: P stays below 2^8, its bf16 relative error and the fp32 sums do not depend
// on the reference, and O is hardly ever rescaled. Sums use P before its rounding.
//
// A masked probability is 0, but 0 times an infinity or NaN in a value row is NaN. Values
// behind the sequence's end (padding may hold anything, and nobody need have written it) do
// not get that far: the products leave out whole sixteens of tokens, and of the sixteen with
// the end warp 11 clears the rest. Rows that a later token of the sequence itself makes not
// finite are computed again from the visible keys alone, once the CTA is through with its
// items: until then other warps wait for the ones that would do it.
#include "kda_attn_rows.cuh"
#include "kda_attn_tc.cuh"

namespace kda {
namespace {

constexpr int kThreads = 384;  // two softmax warpgroups; MMA, load, MMA, and the values' ends
// 384 threads start with 168 registers; the softmax keeps 64 scores and their weights.
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * 168, "register split");
constexpr float kRescale = 8.f;  // log2 of the growth that moves the reference

struct FwdParams {
    CUtensorMap q, k, v;
    AttnProblem p;
    const AttnTile *tiles;  // null: uniform sequences
    __nv_bfloat16 *o;
    float *lse;
    int *status;
    int items, heads;  // heads: of an item, 1 or 2
    uint32_t spin;
    int starve;
};

template <int D>
struct FwdShape {
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr uint32_t kTile = TileShape<D>::kBytes;
    // a stage: the keys of step p and the values of step p - 1, which are read together
    static constexpr uint32_t kQ = 0, kRing = 2 * kTile;
    static constexpr uint32_t kBars = kRing + kStages * 2 * kTile;
    static constexpr uint32_t kBytes = kBars + 256 + 1024;  // and the base's alignment
    static constexpr uint32_t kTmemS = 0, kTmemO = 256;     // columns
};

enum : int { kErrQ = 101, kErrKv, kErrFree, kErrS, kErrP, kErrO, kErrDrain, kErrClean };

template <int D>
__device__ __noinline__ void recompute_row(const FwdParams &f, int row, int start, int h)
{
    attn_row_fwd<__nv_bfloat16, D>(f.p, row, start, h, f.o, f.lse);
}

__host__ __device__ constexpr int fwd_rows(int heads) { return 2 * kTileRows / heads; }

// An item: its query tiles, and the key tiles from the last one down: step it reads key
// tile last - it; query tile w takes part from step begin(w) on.
struct FwdItem {
    int h, first, seq_start, seq_end, last, steps;
    int next_h, next_row;  // from the first tile to the second
    bool two, late;        // there is a second tile; the first one sits out a step
    __device__ __forceinline__ bool get(const FwdParams &f, int n)
    {
        const int idx = nth_item(n, f.items);
        if (idx < 0) return false;
        const int per_tile = f.p.Hq / f.heads;
        const AttnTile t = attn_tile(f.tiles, idx / per_tile, fwd_rows(f.heads), f.p.B, f.p.T);
        if (t.first >= t.seq_end) return false;  // the list's unused end
        h = idx % per_tile * f.heads;
        first = t.first; seq_start = t.seq_start; seq_end = t.seq_end;
        next_h = f.heads - 1;
        next_row = f.heads == 1 ? kTileRows : 0;
        two = first + next_row < seq_end;
        late = two && next_row;
        last = (first - seq_start) / kTileRows + late;
        steps = last + 1;
        return true;
    }
    // an absent second tile never begins
    __device__ __forceinline__ int begin(int w) const { return w ? (two ? 0 : steps + 1) : late; }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_fwd_kernel(const __grid_constant__ FwdParams f)
{
    using S = FwdShape<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + S::kBars);
    uint64_t *q_full = bars, *q_free = bars + 1, *done = bars + 2;
    uint64_t *kv_full = bars + 3, *kv_free = kv_full + S::kStages;
    uint64_t *s_full = kv_free + S::kStages;  // [tile][half] scores are in TMEM
    uint64_t *p_full = s_full + 4;            // [tile][half] probabilities are (one arrival per warp)
    // [tile][half] an item's products of that half are done. Not one more phase of s_full: the
    // next item's first scores follow without an arrival by the softmax, which may then see
    // neither; the next phase here takes that item's probabilities.
    uint64_t *o_full = p_full + 4;
    uint64_t *clean = o_full + 4;             // a stage's values are without what lies behind the sequence
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(clean + S::kStages);
    volatile int *abort = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (!f.tiles && blockIdx.x == 0 && threadIdx.x == 0) *f.status = 0;
    if (warp == 8) tc::tmem_alloc(tmem_slot, 512);
    if (threadIdx.x == 0) {
        tc::mbar_init(q_full, 1);
        tc::mbar_init(q_free, 2);
        tc::mbar_init(done, 2);
        for (int i = 0; i < S::kStages; ++i) {
            tc::mbar_init(kv_full + i, 1);
            tc::mbar_init(kv_free + i, 3);
            tc::mbar_init(clean + i, 1);
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(s_full + i, 1);
            tc::mbar_init(p_full + i, 4);
            tc::mbar_init(o_full + i, 1);
        }
        *abort = 0;
        tc::fence_mbar_init();
    }
    tc::tc_fence_before_sync();
    __syncthreads();
    tc::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    FwdItem t;
    if (f.tiles) wait_for_previous();  // the list

    if (warp >= 8) {
        tc::fewer_registers<kRegsOther>();
        if (warp == 11) {
            // The values that come with a sequence's end. It lets go of every stage too, so that
            // it is never behind on one that is filled again.
            int g = 0;
            bool go = true;
            for (int n = 0; go && t.get(f, n); ++n) {
                const int rows = t.seq_end - t.seq_start - t.last * kTileRows;
                for (int p = 0; p <= t.steps; ++p, ++g) {
                    const int st = g % S::kStages;
                    go = __all_sync(0xffffffffu, tc::mbar_wait(kv_full + st, (g / S::kStages) & 1, abort, f.status,
                                                               kErrKv, f.spin));
                    if (!go) break;
                    if (p == 1 && rows < kTileRows)
                        clear_rows<D>(sm + S::kRing + (st * 2 + 1) * S::kTile, rows, (rows + 15) & ~15);
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tc::mbar_arrive(clean + st);
                        tc::mbar_arrive(kv_free + st);
                    }
                }
            }
        } else if (warp == 9 && lane == 0 && !f.starve) {
            int g = 0, n = 0;  // stages filled, items begun
            bool go = true;
            for (; go && t.get(f, n); ++n) {
                const int hk = t.h / (f.p.Hq / f.p.Hkv);
                if (n && !tc::mbar_wait(q_free, (n - 1) & 1, abort, f.status, kErrFree, f.spin)) break;
                tc::mbar_arrive_expect_tx(q_full, (t.two ? 2 : 1) * S::kTile);
                for (int w = 0; w <= t.two; ++w)
                    tc::load_tile<D>(sm + S::kQ + w * S::kTile, &f.q, t.h + w * t.next_h,
                                     t.first + w * t.next_row, q_full);
                for (int p = 0; p <= t.steps; ++p, ++g) {
                    const int st = g % S::kStages, use = g / S::kStages;
                    uint8_t *to = sm + S::kRing + st * 2 * S::kTile;
                    const int token = t.seq_start + (t.last - p) * kTileRows;
                    go = !use || tc::mbar_wait(kv_free + st, (use - 1) & 1, abort, f.status, kErrFree, f.spin);
                    if (!go) break;
                    tc::mbar_arrive_expect_tx(kv_full + st, ((p < t.steps) + (p > 0)) * S::kTile);
                    if (p < t.steps) tc::load_tile<D>(to, &f.k, hk, token, kv_full + st);
                    if (p > 0) tc::load_tile<D>(to + S::kTile, &f.v, hk, token + kTileRows, kv_full + st);
                }
            }
            // whatever the other warps do, the copies land before the memory is let go
            if (n) tc::mbar_drain(q_full, (n - 1) & 1, f.status, kErrDrain);
            for (int i = max(0, g - S::kStages); i < g; ++i)
                tc::mbar_drain(kv_full + i % S::kStages, (i / S::kStages) & 1, f.status, kErrDrain);
        }
        // one warp issues for each query tile
        if (warp == 8 || warp == 10) {
            const int w = warp == 10;
            const uint32_t lead = lane == 0;
            const uint32_t q = tc::smem_u32(sm + S::kQ + w * S::kTile), ring = tc::smem_u32(sm + S::kRing);
            const uint32_t s_acc = tmem + S::kTmemS + w * 128, o_acc = tmem + S::kTmemO + w * D;
            auto wait = [&](uint64_t *bar, int n, int code) {
                return __all_sync(0xffffffffu, tc::mbar_wait(bar, n & 1, abort, f.status, code, f.spin));
            };
            int g = 0, weights = 0;  // stages read; phases of p_full waited for (either half)
            bool go = true;
            for (int n = 0; go && t.get(f, n); ++n) {
                const int begin = t.begin(w), steps = t.steps;
                // sixteens of step 0's keys that are the sequence's
                const int groups = (t.seq_end - t.seq_start - t.last * kTileRows + 15) >> 4;
                go = wait(q_full, n, kErrQ);
                for (int it = 0; it <= steps && go; ++it, ++g) {
                    const uint32_t k = ring + g % S::kStages * 2 * S::kTile, v = k + S::kTile;
                    const bool both = it > begin;  // and the first half's probabilities
                    const int st = g % S::kStages, use = g / S::kStages;
                    uint64_t *kv = kv_full + st;
                    go = tc::wait_both(kv, use, both ? p_full + 2 * w : kv, both ? weights : use, abort, f.status,
                                       kErrKv, f.spin);
                    // not before the stage is full: until then its last use may not be clean yet
                    if (both && it == 1 && groups < kTileRows / 16) go = go && wait(clean + st, use, kErrClean);
#pragma unroll
                    for (int h2 = 0; h2 < 2; ++h2) {
                        if (go && both) {  // O += P V of the same half of the step before
                            if (h2) go = wait(p_full + 2 * w + 1, weights, kErrP);
                            if (!go) break;
                            tc::tc_fence_after_sync();
                            tc::mma_weights_half<D>(o_acc, s_acc + h2 * 64, v, h2, it == 1 ? groups - 4 * h2 : 4,
                                                    it - 1 > begin || h2 > 0, lead);
                        }
                        if (!go || it < begin) continue;
                        if (it < steps) {
                            tc::mma_rows_half<D>(s_acc + h2 * 64, q, k, h2, lead);
                            tc::commit(s_full + 2 * w + h2, lead);
                        } else {
                            tc::commit(o_full + 2 * w + h2, lead);
                        }
                    }
                    weights += both;
                    if (!go) break;
                    if (it == steps - 1) tc::commit(q_free, lead);
                    tc::commit(kv_free + g % S::kStages, lead);
                }
            }
            tc::commit(done, lead);
            tc::mbar_drain(done, 0, f.status, kErrDrain);
        }
    } else {
        tc::more_registers<kRegsSoftmax>();
        const int w = warp >> 2, in_tile = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's TMEM lanes (32 each, bits 16 up)
        const uint32_t ts = tmem + lanes + S::kTmemS + w * 128;
        const uint32_t to = tmem + lanes + S::kTmemO + w * D;
        const float c = f.p.scale * 1.44269504088896340736f;
        int base = 0, items = 0;  // phases of s_full and of o_full before this item (of either half)
        bool go = true, odd_rows = false;
        for (int n = 0; go && t.get(f, n); ++n) {
            if (w && !t.two) continue;
            const int row = t.first + w * t.next_row + in_tile, h = t.h + w * t.next_h;
            float m = -INFINITY, l = 0.f;  // reference (unscaled score) and sum
            const int units = 2 * (t.steps - t.begin(w));  // halves of key tiles, the diagonal's first
            for (int u = 0; u < units; ++u) {
                const int half = u & 1;
                const uint32_t here = ts + half * 64;
                go = __all_sync(0xffffffffu, tc::mbar_wait(s_full + 2 * w + half, (base + (u >> 1)) & 1, abort,
                                                           f.status, kErrS, f.spin));
                if (!go) break;
                tc::tc_fence_after_sync();
                float s[64];
                tc::tmem_start(here, s);
                tc::tmem_start(here + 32, s + 32);
                tc::tmem_ready(s);
                tc::tmem_ready(s + 32);
                if (u < 2) {  // the diagonal tile
#pragma unroll
                    for (int i = 0; i < 64; ++i) s[i] = i + half * 64 <= in_tile ? s[i] : -INFINITY;
                }
                float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int i = 4; i < 60; i += 8) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) mx[j] = tc::max3(mx[j], s[i + j], s[i + j + 4]);
                }
                const float top = tc::max3(tc::max3(mx[0], s[60], s[61]), tc::max3(mx[1], s[62], s[63]),
                                           fmaxf(mx[2], mx[3]));
                if (u == 0) m = top;
                // Formed with the reference that is there, next to the search for the
                // maximum; once in a while done again.
                for (;;) {
                    const float ref = m == -INFINITY ? 0.f : m * c;
                    const tc::f32x2 c2 = tc::pack2(c, c), r2 = tc::pack2(-ref, -ref);
                    tc::f32x2 sum = 0;
#pragma unroll
                    for (int i = 0; i < 64; i += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float a, b;
                            tc::unpack2(tc::fma2(tc::pack2(s[i + j], s[i + j + 1]), c2, r2), a, b);
                            a = tc::exp2_fast(a);
                            b = tc::exp2_fast(b);
                            sum = tc::add2(sum, tc::pack2(a, b));
                            pk[j / 2] = tc::bf16x2(a, b);
                        }
                        tc::tmem_st16(here + i / 2, pk);
                    }
                    if (!__any_sync(0xffffffffu, (top - m) * c > kRescale || (m == -INFINITY && top > m))) {
                        float sa, sb;
                        tc::unpack2(sum, sa, sb);
                        l += sa + sb;
                        break;
                    }
                    // the next arrival says that the products so far are complete
                    const bool end = u + 1 == units;
                    go = __all_sync(0xffffffffu, tc::mbar_wait((end ? o_full : s_full) + 2 * w + (half ^ 1),
                                                               (end ? items : base + ((u + 1) >> 1)) & 1, abort,
                                                               f.status, kErrS, f.spin));
                    if (!go) break;
                    tc::tc_fence_after_sync();
                    const float m_new = fmaxf(m, top);
                    const float keep = m_new == -INFINITY ? 1.f : tc::exp2_fast((m - m_new) * c);
                    m = m_new;
                    l *= keep;
#pragma unroll
                    for (int i = 0; i < D; i += 16) {
                        float x[16];
                        tc::tmem_ld16_sync(to + i, x);
                        uint32_t y[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) y[j] = __float_as_uint(x[j] * keep);
                        tc::tmem_st16(to + i, y);
                    }
                }
                if (!go) break;
                tc::tmem_st_wait();
                tc::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(p_full + 2 * w + half);
            }
            base += units / 2;
            go = go && tc::wait_both(o_full + 2 * w, items, o_full + 2 * w + 1, items, abort, f.status, kErrO, f.spin);
            ++items;
            if (!go || *abort) break;
            tc::tc_fence_after_sync();
            const bool mine = row < t.seq_end;
            const float inv = 1.f / l;
            __nv_bfloat16 *out = f.o + ((size_t)row * f.p.Hq + h) * D;
            float odd = 0.f;  // NaN if any value is not finite
#pragma unroll
            for (int i = 0; i < D; i += 32) {
                float x[32];
                tc::tmem_start(to + i, x);
                tc::tmem_ready(x);
                uint32_t pk[16];
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    x[j] *= inv;
                    x[j + 1] *= inv;
                    odd = fmaf(x[j], 0.f, fmaf(x[j + 1], 0.f, odd));
                    pk[j / 2] = tc::bf16x2(x[j], x[j + 1]);
                }
                if (mine) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<uint4 *>(out + i + 2 * j) =
                            make_uint4(pk[j], pk[j + 1], pk[j + 2], pk[j + 3]);
                }
            }
            if (mine && f.lse) f.lse[(size_t)row * f.p.Hq + h] = m * f.p.scale + logf(l);
            odd_rows |= __any_sync(0xffffffffu, mine && !(odd == 0.f));
            tc::tc_fence_before_sync();
        }
        tc::tc_fence_before_sync();
        __syncwarp();
        for (int n = 0; odd_rows && go && t.get(f, n); ++n) {
            const int h = t.h + w * t.next_h;
            const int begin = t.first + w * t.next_row + (warp & 3) * 32, end = min(begin + 32, t.seq_end);
            for (int row = begin; row < end; ++row)
                if (!row_finite<__nv_bfloat16, D>(f.o + ((size_t)row * f.p.Hq + h) * D))
                    recompute_row<D>(f, row, t.seq_start, h);
        }
    }
    __syncthreads();
    if (warp == 8) {
        tc::tc_fence_after_sync();
        tc::tmem_relinquish();
        tc::tmem_dealloc(tmem, 512);
    }
}

int fwd_heads(const AttnProblem &p) { return p.Hq / p.Hkv % 2 ? 1 : 2; }

template <int D>
cudaError_t launch(const AttnProblem &p, void *o, float *lse, void *workspace, cudaStream_t st)
{
    char *ws = static_cast<char *>(workspace);
    FwdParams f{};
    f.p = p;
    f.o = static_cast<__nv_bfloat16 *>(o);
    f.lse = lse;
    f.status = reinterpret_cast<int *>(ws);
    f.heads = fwd_heads(p);
    f.items = (int)(attn_tiles(p, fwd_rows(f.heads)) * (p.Hq / f.heads));
    const DebugKnobs dbg = debug_knobs();
    f.spin = dbg.wait_limit ? dbg.wait_limit : tc::kSpinLimit;
    f.starve = dbg.starve_carry;
    if (!encode_attn_map(&f.q, p.q, p.Hq, D, p.tokens) ||
        !encode_attn_map(&f.k, p.k, p.Hkv, D, p.tokens) ||
        !encode_attn_map(&f.v, p.v, p.Hkv, D, p.tokens))
        return cudaErrorInvalidValue;
    if (p.cu_seqlens) {
        f.tiles = reinterpret_cast<const AttnTile *>(
            ws + attn_workspace_layout(p, fwd_rows(f.heads), false).tiles);
        const cudaError_t e = launch_attn_plan(p, fwd_rows(f.heads), workspace, st);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(attn_fwd_kernel<D>, f, f.items < 148 ? f.items : 148, kThreads, FwdShape<D>::kBytes,
                         1, p.cu_seqlens != nullptr, st);
}

}  // namespace

bool encode_attn_map(CUtensorMap *tm, const void *base, int H, int D, long long tokens)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)kTileRows};
    cuuint32_t estride[3] = {1, 1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides,
               box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

int attn_tc_fwd_rows(const AttnProblem &p) { return fwd_rows(fwd_heads(p)); }

cudaError_t launch_attn_tc_fwd(const AttnProblem &p, void *o, float *lse, void *workspace,
                               cudaStream_t st)
{
    if (p.d == 32) return launch<32>(p, o, lse, workspace, st);
    if (p.d == 64) return launch<64>(p, o, lse, workspace, st);
    return launch<128>(p, o, lse, workspace, st);
}

}  // namespace kda
