// kda_attn_tc.cuh — what the tensor-core attention kernels share: tile loads, MMA
// issue over tiles of 128 rows, TMEM rows in registers, packed fp32 arithmetic.
//
// A tile is 128 tokens of one head as TMA leaves it: blocks of 64 channels, each 128
// rows of 128 bytes in the 128-byte swizzle (16 KB). The same bytes are a K-major
// operand over the channels and an MN-major operand over the tokens. Heads of 32
// channels are loaded as 64 of which TMA fills the upper half with zeros.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kda_attn.cuh"
#include "tc_primitives.cuh"

namespace kda {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // kda_tc.cu

constexpr int kTileRows = 128;
constexpr uint32_t kBlockBytes = kTileRows * 128;

template <int D>
struct TileShape {
    static constexpr int kBlocks = (D + 63) / 64;
    static constexpr uint32_t kBytes = kBlocks * kBlockBytes;
};

// [tokens, H, D] bf16 as a {D, H, tokens} tensor, boxes of 64 channels x 1 head x 128
// tokens; what lies outside the tensor reads zero.
bool encode_attn_map(CUtensorMap *tm, const void *base, int H, int D, long long tokens);

// Tile `idx` of a call: from the list, or for uniform sequences (no list) by
// arithmetic in the same order, last tiles first.
__device__ __forceinline__ AttnTile attn_tile(const AttnTile *list, int idx, int rows, int B,
                                              int T)
{
    if (list) return list[idx];
    const int count = (T + rows - 1) / rows;
    const int b = idx % B, t = count - 1 - idx / B;
    return AttnTile{b * T + t * rows, b * T, (b + 1) * T, 0};
}

// The n-th work item of a persistent CTA, -1 behind the last: every other round goes
// through the CTAs backwards, so that with items in order of falling work the CTA with
// the most work of one round gets the least of the next.
__device__ __forceinline__ int nth_item(int n, int items)
{
    const long long at = (long long)n * gridDim.x + (n & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    return at < items ? (int)at : -1;
}

// Rows [first, end) of a tile become zero, by one warp: what a token behind the sequence holds
// is not to meet a weight of 0. The tile's copies have landed; the caller's fence
// (fence_proxy_async_smem) comes before the arrival that lets a product or a later copy have it.
template <int D> __device__ __forceinline__ void clear_rows(uint8_t *tile, int first, int end)
{
#pragma unroll 1  // the callers are short of registers
    for (int u = first * 8 + (threadIdx.x & 31); u < end * 8; u += 32) {  // 16 bytes in each block
#pragma unroll
        for (int b = 0; b < TileShape<D>::kBlocks; ++b)
            reinterpret_cast<uint4 *>(tile + b * kBlockBytes)[u] = make_uint4(0, 0, 0, 0);
    }
}

#ifdef __CUDACC__
namespace tc {

// Move registers between the warps of a CTA (all four warps of a warpgroup call it).
// The sum over the warpgroups must not exceed what the CTA was launched with.
template <int N> __device__ __forceinline__ void more_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void fewer_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// One tile's blocks; the barrier expects TileShape<D>::kBytes.
template <int D>
__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *tm, int head, int token,
                                          uint64_t *bar)
{
#pragma unroll
    for (int b = 0; b < TileShape<D>::kBlocks; ++b)
        tma_load_3d(dst + b * kBlockBytes, tm, b * 64, head, token, bar);
}

// 2-D tiled copy, as tma_load_3d.
__device__ __forceinline__ void tma_load_2d(void *dst_smem, const void *tmap, int x, int y,
                                            uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(smem_u32(dst_smem)), "l"(tmap), "r"(x), "r"(y), "r"(smem_u32(bar))
                 : "memory");
}

// 4-D tiled copy, as tma_load_3d.
__device__ __forceinline__ void tma_load_4d(void *dst_smem, const void *tmap, int x, int y, int z,
                                            int w, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4, %5}], [%6];"
                 ::"r"(smem_u32(dst_smem)), "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w),
                   "r"(smem_u32(bar)) : "memory");
}

// The warp that issues the MMAs runs its loop with all lanes and lets one of them
// (`lead`) issue by predicate: control flow and descriptors stay uniform, so they are kept
// in uniform registers. Issued from a single-lane branch, each instruction cost the
// moves of its operands there.

// A barrier's phase is told by its parity only: whoever waits on a barrier has to see every
// phase of it, or be sure that it is at most one ahead. (With rings whose stages alternate
// between two consumers, the number of stages is even for that; an arrival that nobody's next
// step depends on has a barrier of its own.) Polled beside another barrier it has to be sure of
// the phase before by itself, not only once the other one is through.
//
// Wait for two phases at once, by the whole warp: every other lane polls the other
// barrier, since a poll costs some 150 cycles even of a phase that is complete.
__device__ __forceinline__ bool wait_both(uint64_t *a, int na, uint64_t *b, int nb, volatile int *abort,
                                          int *err, int code, uint32_t limit)
{
    const bool odd = threadIdx.x & 1;
    return __all_sync(0xffffffffu, mbar_wait(odd ? b : a, (odd ? nb : na) & 1, abort, err, code, limit));
}

// The same for three.
__device__ __forceinline__ bool wait_three(uint64_t *a, int na, uint64_t *b, int nb, uint64_t *c, int nc,
                                           volatile int *abort, int *err, int code, uint32_t limit)
{
    const int which = (threadIdx.x & 31) % 3;
    return __all_sync(0xffffffffu, mbar_wait(which == 0 ? a : which == 1 ? b : c,
                                             (which == 0 ? na : which == 1 ? nb : nc) & 1, abort, err, code, limit));
}

// D[tmem] (+)= A[smem desc] * B[smem desc], bf16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate, uint32_t lead)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
                 : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem desc].
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate, uint32_t lead)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
                 : "memory");
}

// The lead's arrival on `bar` once all it has issued is complete.
__device__ __forceinline__ void commit(uint64_t *bar, uint32_t lead)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
                 ::"r"(smem_u32(bar)), "r"(lead) : "memory");
}

// acc[128 x 128] = X Y^T over the channels of two tiles.
template <int D>
__device__ __forceinline__ void mma_rows_rows(uint32_t acc, uint32_t x, uint32_t y, uint32_t lead)
{
    const uint64_t a = smem_desc(x, 16, 1024), b = smem_desc(y, 16, 1024);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = ((k >> 2) * kBlockBytes + (k & 3) * 32) >> 4;
        mma_ss(acc, a + off, b + off, idesc_bf16(128, 128, 0, 0), k > 0, lead);
    }
}

// acc[128 x 64] = X Y_h^T: half h of tile y's rows (64 of them).
template <int D>
__device__ __forceinline__ void mma_rows_half(uint32_t acc, uint32_t x, uint32_t y, int h,
                                              uint32_t lead)
{
    const uint64_t a = smem_desc(x, 16, 1024), b = smem_desc(y + h * 64 * 128, 16, 1024);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = ((k >> 2) * kBlockBytes + (k & 3) * 32) >> 4;
        mma_ss(acc, a + off, b + off, idesc_bf16(128, 64, 0, 0), k > 0, lead);
    }
}

// acc[128 x D] (+)= W Y_h over half h of tile y's tokens, of which the first 16 * groups count:
// W [128 x 64] bf16 in 32 columns.
template <int D>
__device__ __forceinline__ void mma_weights_half(uint32_t acc, uint32_t w, uint32_t y, int h, int groups,
                                                 bool accumulate, uint32_t lead)
{
    const uint64_t b = smem_desc(y + h * 4 * 2048, kBlockBytes, 1024);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        mma_ts(acc, w + k * 8, b + ((k * 2048) >> 4), idesc_bf16(128, D, 0, 1), accumulate || k > 0,
               k < groups ? lead : 0);
}

// acc[128 x D] (+)= W Y over 128 tokens: W [128 x 128] bf16 in TMEM, 32 columns for the
// first 64 tokens and 32 more that begin kHalf columns on; Y a tile read along its tokens.
template <int D, int kHalf>
__device__ __forceinline__ void mma_weights_rows(uint32_t acc, uint32_t w, uint32_t y,
                                                 bool accumulate, uint32_t lead)
{
    const uint64_t b = smem_desc(y, kBlockBytes, 1024);
#pragma unroll
    for (int k = 0; k < kTileRows / 16; ++k)
        mma_ts(acc, w + (k >> 2) * kHalf + (k & 3) * 8, b + ((k * 2048) >> 4),
               idesc_bf16(128, D, 0, 1), accumulate || k > 0, lead);
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define KDA_R4(v, i) "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3])
#define KDA_R16(v, i) KDA_R4(v, i), KDA_R4(v, i + 4), KDA_R4(v, i + 8), KDA_R4(v, i + 12)
#define KDA_RW4(v, i) "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3])
#define KDA_RW16(v, i) KDA_RW4(v, i), KDA_RW4(v, i + 4), KDA_RW4(v, i + 8), KDA_RW4(v, i + 12)

// Start reading 32 columns of this warp's 32 lanes: lane l gets its TMEM lane's values.
// The registers hold them after tmem_ready on the same array.
__device__ __forceinline__ void tmem_start(uint32_t taddr, float *v)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32"
                 " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : KDA_R16(v, 0), KDA_R16(v, 16) : "r"(taddr) : "memory");
}

// Wait for every read this thread started; no use of v moves before it.
__device__ __forceinline__ void tmem_ready(float *v)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : KDA_RW16(v, 0), KDA_RW16(v, 16) :: "memory");
}

// Write 16 columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *v)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16],"
                 " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
                 :: "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                    "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
                    "r"(taddr) : "memory");
}

// 16 columns and the wait in one.
__device__ __forceinline__ void tmem_ld16_sync(uint32_t taddr, float *v)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32"
                 " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : KDA_R16(v, 0) : "r"(taddr) : "memory");
}

// Two fp32 values in one 64-bit register pair.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 x, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// lo in the lower half: the operand's element order.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 4-byte asynchronous copy global -> shared, of zero where it is not `real`, and an arrival on
// `bar` once this thread's copies so far have landed (the barrier counts it like any arrival).
__device__ __forceinline__ void cp_async4(void *dst, const void *src, bool real)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(real ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

}  // namespace tc
#endif

}  // namespace kda
