// kda_cache.cu — pages of the full-attention layers' key/value cache: tables that
// fork, grow and shrink on the device, and the data moves that go with them.
//
// The table calls read and write a few hundred kilobytes at most and are bound by
// the latency of their dependent steps; the data calls are bound by HBM and move
// 16 bytes per thread and access, the pages of one (page, head) being contiguous.
// Reference counts are kept with integer atomics, whose order does not change the
// result; pages are handed out by prefix sums in row order.
#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int kWide = 1024;

__device__ __forceinline__ bool page_ok(int id, int P) { return (unsigned)id < (unsigned)P; }

// Tokens of a row, whatever the table's owner wrote: at least 0, at most M pages.
__device__ __forceinline__ int clamp_len(int len, int M, int shift)
{
    return min(max(len, 0), M << shift);
}

__device__ __forceinline__ int pages_of(int len, int shift)
{
    return (len >> shift) + ((len & ((1 << shift) - 1)) != 0);
}

// ---------------------------------------------------------------- fork
// One warp per row: the first N_out copy a row of the old table and take hold of its
// pages, the other N_in let go of an old row's pages.
__global__ void __launch_bounds__(256)
cache_fork_kernel(int32_t *refs, const int32_t *table, const int32_t *lens,
                  const int32_t *parents, int N_in, int N_out, int M, int P,
                  int32_t *new_table, int32_t *new_lens)
{
    const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (w >= (long long)N_out + N_in) return;
    if (w < N_out) {
        const int from = parents[w];
        const bool any = (unsigned)from < (unsigned)N_in;
        for (int m = lane; m < M; m += 32) {
            const int id = any ? table[(size_t)from * M + m] : -1;
            new_table[(size_t)w * M + m] = id;
            if (page_ok(id, P)) atomicAdd(refs + id, 1);
        }
        if (lane == 0) new_lens[w] = any ? lens[from] : 0;
        return;
    }
    const size_t n = (size_t)(w - N_out);
    for (int m = lane; m < M; m += 32) {
        const int id = table[n * M + m];
        if (page_ok(id, P)) atomicSub(refs + id, 1);
    }
}

// ---------------------------------------------------------------- reserve
// Inclusive scan over a block of kWide threads.
__device__ long long block_scan(long long x, long long *s_warp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        long long v = s_warp[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, v, off);
            if (lane >= off) v += y;
        }
        s_warp[lane] = v;
    }
    __syncthreads();
    if (warp > 0) x += s_warp[warp - 1];
    __syncthreads();
    return x;
}

struct Row {
    int len, have, tail;  // tail: the partly filled last page that is to be written, or -1
    long long want;       // pages after the call
};

__device__ __forceinline__ Row row_of(const int32_t *table, const int32_t *lens,
                                      const int32_t *add, int n, int M, int P, int shift)
{
    Row r;
    r.len = clamp_len(lens[n], M, shift);
    r.have = pages_of(r.len, shift);
    const int more = max(add[n], 0);
    r.want = ((long long)r.len + more + (1 << shift) - 1) >> shift;
    r.tail = -1;
    if (more > 0 && (r.len & ((1 << shift) - 1))) {
        const int id = table[(size_t)n * M + r.have - 1];
        if (page_ok(id, P)) r.tail = id;
    }
    return r;
}

constexpr int kEach = 8;             // pages that a thread looks at together
constexpr int kRowsShared = 4096;    // rows whose places are in shared memory

// Bit j: page at + j is free.
__device__ __forceinline__ unsigned free_pages(const int32_t *refs, int at, int P)
{
    unsigned bits = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j)
        if (at + j < P && refs[at + j] == 0) bits |= 1u << j;
    return bits;
}

// One block: rows and pages are few, and their order is what makes the result.
// A row copies its last page unless it is the page's only holder, or the last of
// rows of this call that are together all its holders; both follow from the number
// of such rows per page and the largest of them, which atomics count in any order.
// What takes the time are reads that depend on one another: so a thread keeps its first
// row in registers, the first free pages are looked for before anything else, and every
// page that is handed out finds its row by itself (256 rows: 7.8 us; a warp per row,
// eight rows one after another, 14 us).
__global__ void __launch_bounds__(kWide)
cache_reserve_kernel(int32_t *refs, int32_t *table, int32_t *lens, const int32_t *add, int N,
                     int M, int P, int shift, int32_t *copies, int32_t *status,
                     int32_t *ws)
{
    __shared__ long long s_warp[32];
    __shared__ long long s_carry;
    __shared__ int s_over;
    __shared__ int s_first[kRowsShared], s_slot[kRowsShared];
    int32_t *sharers = ws, *last = ws + P, *freed = ws + 2 * (size_t)P;
    // of a row: where its share of the free pages begins, and the table's place of the first
    int32_t *first = N <= kRowsShared ? s_first : ws + 3 * (size_t)P;
    int32_t *slot = N <= kRowsShared ? s_slot : ws + 3 * (size_t)P + N;
    const int tid = threadIdx.x;
    if (tid == 0) { s_over = INT32_MAX; s_carry = 0; }
    const unsigned free0 = free_pages(refs, tid * kEach, P);
    const Row row0 = tid < N ? row_of(table, lens, add, tid, M, P, shift) : Row{};
    auto row = [&](int n) { return n == tid ? row0 : row_of(table, lens, add, n, M, P, shift); };
    for (int n = tid; n < N; n += kWide) {
        const Row r = row(n);
        if (r.tail >= 0) { sharers[r.tail] = 0; last[r.tail] = -1; }
    }
    __syncthreads();
    for (int n = tid; n < N; n += kWide) {
        const Row r = row(n);
        if (r.want > M) atomicMin(&s_over, n);
        if (r.tail >= 0) { atomicAdd(sharers + r.tail, 1); atomicMax(last + r.tail, n); }
    }
    __syncthreads();
    // pages each row takes, and where its share of the free pages begins
    for (int base = 0; base < N; base += kWide) {
        const int n = base + tid;
        long long count = 0;
        Row r{};
        bool copy = false;
        if (n < N) {
            r = row(n);
            copy = r.tail >= 0 && refs[r.tail] > 1 &&
                   !(sharers[r.tail] >= refs[r.tail] && last[r.tail] == n);
            count = (copy ? 1 : 0) + (r.want - r.have);
        }
        const long long incl = block_scan(count, s_warp);
        const long long carry = s_carry;
        if (n < N) {
            first[n] = (int)min(carry + incl - count, (long long)INT32_MAX);
            slot[n] = r.have - copy;  // the copy takes the last page's place
        }
        __syncthreads();
        if (tid == kWide - 1) s_carry = carry + incl;
        __syncthreads();
    }
    const long long need = s_carry;
    __syncthreads();
    // the lowest free pages in order, as many as are needed
    if (tid == 0) s_carry = 0;
    __syncthreads();
    for (int base = 0; base < P; base += kWide * kEach) {
        const long long carry = s_carry;
        if (carry >= need) break;
        const int at = base + tid * kEach;
        unsigned bits = base ? free_pages(refs, at, P) : free0;
        const int mine = __popc(bits);
        const long long incl = block_scan(mine, s_warp);
        long long to = carry + incl - mine;
        for (; bits; bits &= bits - 1, ++to)
            if (to < need) freed[to] = at + __ffs(bits) - 1;
        __syncthreads();
        if (tid == kWide - 1) s_carry = carry + incl;
        __syncthreads();
    }
    const long long found = s_carry;
    const int over = s_over;
    const bool fails = over != INT32_MAX || found < need;
    if (tid == 0)
        *status = over != INT32_MAX ? -1 - over
                  : found < need    ? (int)min(need - found, (long long)INT32_MAX)
                                    : 0;
    for (int n = tid; n < N; n += kWide) {
        int from = -1, to = -1;
        if (!fails) {
            const Row r = row(n);
            if (slot[n] < r.have) {
                from = r.tail;
                to = freed[first[n]];
                atomicSub(refs + from, 1);
            }
            lens[n] = r.len + max(add[n], 0);
        }
        copies[2 * (size_t)n] = from;
        copies[2 * (size_t)n + 1] = to;
    }
    if (fails) return;
    __syncthreads();
    for (int k = tid; k < (int)need; k += kWide) {
        int n = 0;  // the last row whose share begins at or before k
        for (int end = N; end - n > 1;) {
            const int mid = (n + end) >> 1;
            if (first[mid] <= k) n = mid; else end = mid;
        }
        const int id = freed[k];
        table[(size_t)n * M + slot[n] + (k - first[n])] = id;
        refs[id] = 1;
    }
}

// ---------------------------------------------------------------- release
__global__ void __launch_bounds__(256)
cache_release_kernel(int32_t *refs, int32_t *table, int32_t *lens, const int32_t *new_lens,
                     int N, int M, int P, int shift)
{
    const long long n = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (n >= N) return;
    const int len = clamp_len(min(lens[n], new_lens[n]), M, shift);
    __syncwarp();
    if (lane == 0) lens[n] = len;
    for (int m = pages_of(len, shift) + lane; m < M; m += 32) {
        const int id = table[n * M + m];
        if (page_ok(id, P)) atomicSub(refs + id, 1);
        table[n * M + m] = -1;
    }
}

// ---------------------------------------------------------------- data
// Byte offset of position pos of a row, head hk, in a pool; -1 where it has no page.
__device__ __forceinline__ long long place(const PagePool &pool, const int32_t *row, int M,
                                           long long pos, int hk)
{
    if (pos < 0 || pos >= (long long)M << pool.page_shift) return -1;
    const int id = row[pos >> pool.page_shift];
    if (!page_ok(id, pool.P)) return -1;
    const long long slot = pos & ((1 << pool.page_shift) - 1);
    return ((((long long)id * pool.Hkv + hk) << pool.page_shift) + slot) * pool.d * pool.elem;
}

// 16 bytes of a token's keys and of its values: unit u, the x-th of head hk, at pos of sequence n.
__device__ __forceinline__ void append_unit(const PagePool &pool, const int32_t *table,
                                            const int32_t *start, const uint4 *k_new,
                                            const uint4 *v_new, int M, long long u, int n,
                                            long long pos, int hk, int x)
{
    const int at = start[n];
    const long long to = at < 0 ? -1 : place(pool, table + (size_t)n * M, M, at + pos, hk);
    if (to < 0) return;
    const uint4 a = __ldg(k_new + u), b = __ldg(v_new + u);
    *reinterpret_cast<uint4 *>(static_cast<char *>(pool.k) + to + x * 16) = a;
    *reinterpret_cast<uint4 *>(static_cast<char *>(pool.v) + to + x * 16) = b;
}

// One thread per unit.
__global__ void __launch_bounds__(256)
cache_append_kernel(PagePool pool, const int32_t *table, const int32_t *start,
                    const uint4 *k_new, const uint4 *v_new, int T, int M, long long units,
                    int head_units)
{
    const long long u = (long long)blockIdx.x * 256 + threadIdx.x;
    if (u >= units) return;
    const int per_token = pool.Hkv * head_units;
    const long long t = u / per_token;
    const int in = (int)(u % per_token);
    append_unit(pool, table, start, k_new, v_new, M, u, (int)(t / T), t % T, in / head_units,
                in % head_units);
}

// Packed sequences. The offsets are made non-decreasing as the prompt's plan makes them:
// sequence n begins at the largest of 0 and cu[0..n]. Up to kOffsets of them each block keeps;
// they hardly ever fall, which is seen as they come in, so the running maximum is hardly ever
// formed.
constexpr int kOffsets = 1024;
__global__ void __launch_bounds__(256)
cache_append_packed_kernel(PagePool pool, const int32_t *table, const int32_t *start,
                           const uint4 *k_new, const uint4 *v_new, const int32_t *cu, int N, int M,
                           long long units, int head_units)
{
    __shared__ int s_cu[kOffsets];
    const int tid = threadIdx.x;
    bool rises = true;
    for (int i = tid; i <= N; i += 256) {
        const int x = cu[i];
        s_cu[i] = max(x, 0);
        rises &= x >= (i ? cu[i - 1] : 0);
    }
    if (!__syncthreads_and(rises)) {
        if (tid < 32) {
            int most = 0;
            for (int base = 0; base <= N; base += 32) {
                int x = base + tid <= N ? s_cu[base + tid] : 0;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, off);
                    if (tid >= off) x = max(x, y);
                }
                x = max(x, most);
                if (base + tid <= N) s_cu[base + tid] = x;
                most = __shfl_sync(0xffffffffu, x, 31);
            }
        }
        __syncthreads();
    }
    const long long u = (long long)blockIdx.x * 256 + tid;
    const int per_token = pool.Hkv * head_units;
    const long long t = u / per_token;
    if (u >= units || t < s_cu[0] || t >= s_cu[N]) return;
    int n = 0;  // the last sequence that begins at or before t
    for (int end = N; end - n > 1;) {
        const int mid = (n + end) >> 1;
        if (s_cu[mid] <= t) n = mid; else end = mid;
    }
    const int in = (int)(u % per_token);
    append_unit(pool, table, start, k_new, v_new, M, u, n, t - s_cu[n], in / head_units,
                in % head_units);
}

// The same for more sequences than that. Token t belongs to the sequence before the first offset
// beyond t: a block looks for that of its first token together, kLooked offsets at a time from
// the first on, and its threads go on from there. What this reads grows with blocks times
// sequences, so no more blocks than run at a time (60000 tokens of one head of 64 in 20000
// sequences: 25 us, 31 with blocks of 1024; a search by every thread that trusted the offsets,
// 20).
constexpr int kMany = 256, kLooked = kMany * 16, kManyBlocks = 148 * 8;
__global__ void __launch_bounds__(kMany)
cache_append_many_kernel(PagePool pool, const int32_t *table, const int32_t *start,
                         const uint4 *k_new, const uint4 *v_new, const int32_t *cu, int N, int M,
                         long long units, long long each, int head_units)
{
    __shared__ int s_beyond, s_begin;
    const int per_token = pool.Hkv * head_units, tid = threadIdx.x;
    const long long first = blockIdx.x * each, end = min(first + each, units);
    const long long t0 = first / per_token;
    if (tid == 0) { s_beyond = N + 1; s_begin = 0; }
    __syncthreads();
    for (int base = 0; base <= N; base += kLooked) {
        int x[kLooked / kMany], found = N + 1, most = 0;
#pragma unroll
        for (int j = 0; j < kLooked / kMany; ++j) {
            const int i = base + j * kMany + tid;
            x[j] = i <= N ? __ldg(cu + i) : 0;
        }
#pragma unroll
        for (int j = kLooked / kMany - 1; j >= 0; --j) {
            const int i = base + j * kMany + tid;
            if (i <= N && x[j] > t0) found = i;
        }
        if (found <= N) atomicMin(&s_beyond, found);
        __syncthreads();
        const int beyond = s_beyond;
#pragma unroll
        for (int j = 0; j < kLooked / kMany; ++j)
            if (base + j * kMany + tid < beyond) most = max(most, x[j]);
        if (most > 0) atomicMax(&s_begin, most);
        __syncthreads();  // all have read it before the next offsets lower it
        if (beyond <= N) break;
    }
    int beyond = s_beyond, begin = s_begin;
    for (long long u = first + tid; u < end; u += kMany) {
        const long long t = u / per_token;
        for (; beyond <= N && cu[beyond] <= t; ++beyond) begin = max(begin, cu[beyond]);
        if (beyond > N) return;     // behind the last sequence
        if (beyond == 0) continue;  // before the first
        const int in = (int)(u % per_token);
        append_unit(pool, table, start, k_new, v_new, M, u, beyond - 1, t - begin, in / head_units,
                    in % head_units);
    }
}

// One block per sequence and 256 16-byte columns of (k or v, head). A thread moves its
// column's kept tokens in order, four reads ahead of four writes: path[j] >= j and the
// path increases, so a token is read before its place is written.
__global__ void __launch_bounds__(256)
cache_compact_kernel(PagePool pool, const int32_t *table, const int32_t *ctx_lens,
                     const int32_t *path, int R, int M, int head_units, int32_t *new_lens)
{
    __shared__ int s_path[1024];
    __shared__ int s_kept;
    const int n = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) s_kept = R;
    __syncthreads();
    for (int j = tid; j < R; j += 256) {
        const int a = path[(size_t)n * R + j];
        const int before = j ? path[(size_t)n * R + j - 1] : -1;
        s_path[j] = a;
        if (a <= before || a >= R || a < 0) atomicMin(&s_kept, j);
    }
    __syncthreads();
    const int kept = s_kept;
    const int ctx = clamp_len(ctx_lens[n], M, pool.page_shift);
    if (blockIdx.y == 0 && tid == 0) new_lens[n] = ctx + kept;
    const int u = blockIdx.y * 256 + tid, per_pool = pool.Hkv * head_units;
    if (u >= 2 * per_pool) return;
    char *base = static_cast<char *>(u < per_pool ? pool.k : pool.v) + (u % head_units) * 16;
    const int hk = u % per_pool / head_units;
    const int32_t *row = table + (size_t)n * M;
    constexpr int kAhead = 4;
    for (int j0 = 0; j0 < kept; j0 += kAhead) {
        uint4 x[kAhead];
        long long to[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            to[i] = -1;
            const int j = j0 + i;
            if (j >= kept || s_path[j] == j) continue;
            const long long from = place(pool, row, M, (long long)ctx + s_path[j], hk);
            if (from < 0) continue;
            to[i] = place(pool, row, M, (long long)ctx + j, hk);
            x[i] = *reinterpret_cast<const uint4 *>(base + from);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (to[i] >= 0) *reinterpret_cast<uint4 *>(base + to[i]) = x[i];
    }
}

// One block per pair, slice of the page, and pool. Whether a pair is left out is found
// from the whole list by every block of it, so a slice is at least half of the list (16384
// pages of 128 KB in each pool: 1.32 ms, in slices of 16 KB as few pages have them 2.23).
__global__ void __launch_bounds__(256)
cache_copy_kernel(PagePool pool, const int2 *copies, int C, long long page_units)
{
    const int c = blockIdx.x;
    const int2 me = copies[c];
    if (!page_ok(me.x, pool.P) || !page_ok(me.y, pool.P) || me.x == me.y) return;
    int out = 0;
    for (int i = threadIdx.x; i < C; i += 256) {
        const int2 o = copies[i];
        if (!page_ok(o.x, pool.P) || !page_ok(o.y, pool.P) || o.x == o.y) continue;
        out |= (i < c && o.y == me.y) || o.x == me.y;
    }
    if (__syncthreads_or(out)) return;
    char *p = static_cast<char *>(blockIdx.z ? pool.v : pool.k);
    const uint4 *src = reinterpret_cast<const uint4 *>(p) + (size_t)me.x * page_units;
    uint4 *dst = reinterpret_cast<uint4 *>(p) + (size_t)me.y * page_units;
    constexpr int kEach = 4;
    for (long long base = (long long)blockIdx.y * 256 * kEach; base < page_units;
         base += (long long)gridDim.y * 256 * kEach) {
        uint4 x[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const long long at = base + i * 256 + threadIdx.x;
            if (at < page_units) x[i] = src[at];
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const long long at = base + i * 256 + threadIdx.x;
            if (at < page_units) dst[at] = x[i];
        }
    }
}

cudaError_t launched()
{
    note_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_fork(int32_t *refs, const int32_t *table, const int32_t *lens,
                              const int32_t *parents, int N_in, int N_out, int M, int P,
                              int32_t *new_table, int32_t *new_lens, cudaStream_t st)
{
    const long long warps = (long long)N_in + N_out;
    cache_fork_kernel<<<(unsigned)((warps + 7) / 8), 256, 0, st>>>(
        refs, table, lens, parents, N_in, N_out, M, P, new_table, new_lens);
    return launched();
}

cudaError_t launch_cache_reserve(int32_t *refs, int32_t *table, int32_t *lens,
                                 const int32_t *add, int N, int M, int P, int page_shift,
                                 int32_t *copies, int32_t *status, void *workspace,
                                 cudaStream_t st)
{
    cache_reserve_kernel<<<1, kWide, 0, st>>>(refs, table, lens, add, N, M, P, page_shift, copies,
                                              status, static_cast<int32_t *>(workspace));
    return launched();
}

cudaError_t launch_cache_release(int32_t *refs, int32_t *table, int32_t *lens,
                                 const int32_t *new_lens, int N, int M, int P, int page_shift,
                                 cudaStream_t st)
{
    cache_release_kernel<<<(unsigned)(((long long)N + 7) / 8), 256, 0, st>>>(
        refs, table, lens, new_lens, N, M, P, page_shift);
    return launched();
}

cudaError_t launch_cache_append(const PagePool &pool, const int32_t *table, const int32_t *start,
                                const void *k_new, const void *v_new, const int32_t *cu_seqlens,
                                int N, int B, int T, int M, cudaStream_t st)
{
    const int head_units = pool.d * pool.elem / 16;
    const long long units = (long long)B * T * pool.Hkv * head_units;
    const long long blocks = (units + 255) / 256;
    const uint4 *k = static_cast<const uint4 *>(k_new), *v = static_cast<const uint4 *>(v_new);
    if (cu_seqlens && N >= kOffsets) {
        const long long all = (units + kMany - 1) / kMany, rounds = (all + kManyBlocks - 1) / kManyBlocks;
        cache_append_many_kernel<<<(unsigned)((all + rounds - 1) / rounds), kMany, 0, st>>>(
            pool, table, start, k, v, cu_seqlens, N, M, units, rounds * kMany, head_units);
        return launched();
    }
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (cu_seqlens)
        cache_append_packed_kernel<<<(unsigned)blocks, 256, 0, st>>>(
            pool, table, start, k, v, cu_seqlens, N, M, units, head_units);
    else
        cache_append_kernel<<<(unsigned)blocks, 256, 0, st>>>(pool, table, start, k, v, T, M, units,
                                                              head_units);
    return launched();
}

cudaError_t launch_cache_compact(const PagePool &pool, const int32_t *table,
                                 const int32_t *ctx_lens, const int32_t *path, int N, int R,
                                 int M, int32_t *new_lens, cudaStream_t st)
{
    const int head_units = pool.d * pool.elem / 16;
    const dim3 grid((unsigned)N, (unsigned)((2 * pool.Hkv * head_units + 255) / 256));
    cache_compact_kernel<<<grid, 256, 0, st>>>(pool, table, ctx_lens, path, R, M, head_units,
                                               new_lens);
    return launched();
}

cudaError_t launch_cache_copy(const PagePool &pool, const int32_t *copies, int C,
                              cudaStream_t st)
{
    const long long units = ((long long)pool.Hkv << pool.page_shift) * pool.d * pool.elem / 16;
    const long long each = C < 4096 ? 1024 : C / 4;  // 16-byte units of a slice; a pair is 8 bytes
    const long long slices = (units + each - 1) / each;
    const dim3 grid((unsigned)C, (unsigned)(slices < 64 ? slices : 64), 2);
    cache_copy_kernel<<<grid, 256, 0, st>>>(pool, reinterpret_cast<const int2 *>(copies), C,
                                            units);
    return launched();
}

}  // namespace kda
