// kda_attn_api.cu — the exported C ABI of the full-attention calls: argument
// checks, workspace sizing, dispatch. Every check runs on the host before any
// launch and touches no device state.
#include <math.h>
#include <stdlib.h>

#include <initializer_list>

#include "kda_attn.cuh"

namespace {

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool attn_dtype_ok(kda_dtype_t t) { return t == KDA_DTYPE_F32 || t == KDA_DTYPE_BF16; }
bool attn_head_ok(int d) { return d == 32 || d == 64 || d == 128; }
int elem_bytes(kda_dtype_t t) { return t == KDA_DTYPE_F32 ? 4 : 2; }

// Rows, pages, sequences and tiles are walked in 32 bits, up to 8192 at a time.
constexpr int kMostWalked = INT32_MAX - 16384;

// KDA_DEBUG_SYNC=1: wait for the call and report its status word.
bool attn_debug_sync()
{
    static const bool on = [] {
        const char *e = getenv("KDA_DEBUG_SYNC");
        return e != nullptr && e[0] != '\0' && e[0] != '0';
    }();
    return on;
}

kda_status_t heads_ok(int Hq, int Hkv, int d, kda_dtype_t dt)
{
    if (Hq < 1 || Hkv < 1 || d < 1) return KDA_ERR_INVALID_ARG;
    if (!attn_dtype_ok(dt) || !attn_head_ok(d)) return KDA_ERR_UNSUPPORTED;
    if (Hq % Hkv != 0) return KDA_ERR_INVALID_ARG;
    if (Hq > 65535) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// The packed time axis: sizes -> tokens and sequences.
kda_status_t sequences_ok(int B, int T, bool varlen, int n_seqs, long long *tokens, int *N)
{
    if (B < 1 || T < 0) return KDA_ERR_INVALID_ARG;
    if (varlen && (B != 1 || n_seqs < 1)) return KDA_ERR_INVALID_ARG;
    *tokens = (long long)B * T;
    *N = varlen ? n_seqs : B;
    if (*tokens > (long long)INT32_MAX - 1024 || *N > kMostWalked) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status_t describe_attn(int B, int T, int Hq, int Hkv, int d, int n_seqs, bool varlen,
                           kda_dtype_t dt, kda::AttnProblem *p)
{
    kda_status_t st = heads_ok(Hq, Hkv, d, dt);
    if (st != KDA_OK) return st;
    *p = kda::AttnProblem{};
    st = sequences_ok(B, T, varlen, n_seqs, &p->tokens, &p->N);
    if (st != KDA_OK) return st;
    p->B = B; p->T = T; p->Hq = Hq; p->Hkv = Hkv; p->d = d; p->dtype = dt;
    // any non-null value: only whether offsets are given matters before the call
    p->cu_seqlens = varlen ? reinterpret_cast<const int32_t *>(16) : nullptr;
    // one CTA per tile and head in a one-dimensional grid, at least 32 tokens a tile
    if ((kda::attn_tiles(*p, 32) + 1) * Hq > (long long)INT32_MAX || kda::attn_tiles(*p, 32) > kMostWalked ||
        p->tokens * Hq / 8 > (long long)INT32_MAX)  // and eight rows to a block at least
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

size_t attn_workspace(kda::AttnProblem &p, bool bwd)
{
    return kda::attn_workspace_layout(p, bwd ? kda::attn_bwd_rows(p) : kda::attn_fwd_rows(p), bwd)
        .total;
}

bool scale_ok(float s) { return isfinite(s) && s > 0.f; }

int log2_page(int page_size)
{
    if (page_size < 1 || page_size > 1024 || (page_size & (page_size - 1))) return -1;
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

// Sizes of a table and its pool.
kda_status_t table_ok(int N, int M, int P)
{
    if (N < 1 || M < 1 || P < 1) return KDA_ERR_INVALID_ARG;
    if ((long long)N * M > (long long)INT32_MAX || N > kMostWalked || P > kMostWalked)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status_t pool_ok(const void *k, const void *v, kda_dtype_t dt, int Hkv, int d, int P, int M,
                     int page_size, kda::PagePool *pool)
{
    kda_status_t st = heads_ok(Hkv, Hkv, d, dt);
    if (st != KDA_OK) return st;
    st = table_ok(1, M, P);
    if (st != KDA_OK) return st;
    const int shift = log2_page(page_size);
    if (shift < 0) return KDA_ERR_UNSUPPORTED;
    if ((long long)M * page_size > (long long)INT32_MAX - 1024) return KDA_ERR_UNSUPPORTED;
    if (!k || !v) return KDA_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16)) return KDA_ERR_ALIGNMENT;
    *pool = kda::PagePool{const_cast<void *>(k), const_cast<void *>(v), P, Hkv, d, shift,
                          elem_bytes(dt)};
    return KDA_OK;
}

bool overlap(const int32_t *a, long long na, const int32_t *b, long long nb)
{
    return a < b + nb && b < a + na;
}

// Null and 4-byte alignment of the int32 arguments of a table call.
kda_status_t ints_ok(std::initializer_list<const int32_t *> ptrs)
{
    for (const int32_t *p : ptrs)
        if (!p) return KDA_ERR_INVALID_ARG;
    for (const int32_t *p : ptrs)
        if (!aligned(p, 4)) return KDA_ERR_ALIGNMENT;
    return KDA_OK;
}

kda_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace

extern "C" {

size_t kda_attn_fwd_workspace_size(int B, int T, int Hq, int Hkv, int d, int n_seqs,
                                   kda_dtype_t dt)
{
    kda::AttnProblem p;
    if (describe_attn(B, T, Hq, Hkv, d, n_seqs, n_seqs > 0 && B == 1, dt, &p) != KDA_OK) return 0;
    return attn_workspace(p, false);
}

size_t kda_attn_bwd_workspace_size(int B, int T, int Hq, int Hkv, int d, int n_seqs,
                                   kda_dtype_t dt)
{
    kda::AttnProblem p;
    if (describe_attn(B, T, Hq, Hkv, d, n_seqs, n_seqs > 0 && B == 1, dt, &p) != KDA_OK) return 0;
    return attn_workspace(p, true);
}

kda_status_t kda_attn_status(const void *workspace, size_t workspace_bytes, int *device_code,
                             void *stream)
{
    return kda_chunk_fwd_status(workspace, workspace_bytes, device_code, stream);
}

kda_status_t kda_attn_fwd(const void *q, const void *k, const void *v, kda_dtype_t dt,
                          const int32_t *cu_seqlens, int n_seqs, int B, int T, int Hq, int Hkv,
                          int d, float scale, void *o, float *lse, void *workspace,
                          size_t workspace_bytes, void *stream)
{
    kda::AttnProblem p;
    kda_status_t st = describe_attn(B, T, Hq, Hkv, d, n_seqs, cu_seqlens != nullptr, dt, &p);
    if (st != KDA_OK) return st;
    if (!scale_ok(scale)) return KDA_ERR_INVALID_ARG;
    if (p.tokens == 0) return KDA_OK;
    if (!q || !k || !v || !o) return KDA_ERR_INVALID_ARG;
    for (const void *ptr : {q, k, v, (const void *)o, (const void *)lse, (const void *)workspace})
        if (!aligned(ptr, 16)) return KDA_ERR_ALIGNMENT;
    if (!aligned(cu_seqlens, 4)) return KDA_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < attn_workspace(p, false)) return KDA_ERR_WORKSPACE;
    p.q = q; p.k = k; p.v = v; p.cu_seqlens = cu_seqlens; p.scale = scale;
    st = from_cuda(kda::launch_attn_fwd(p, o, lse, workspace, static_cast<cudaStream_t>(stream)));
    if (st != KDA_OK || !attn_debug_sync()) return st;
    int code = 0;
    return kda_attn_status(workspace, workspace_bytes, &code, stream);
}

kda_status_t kda_attn_bwd(const void *q, const void *k, const void *v, const void *o,
                          const float *lse, const void *dO, kda_dtype_t dt,
                          const int32_t *cu_seqlens, int n_seqs, int B, int T, int Hq, int Hkv,
                          int d, float scale, void *grad_q, void *grad_k, void *grad_v,
                          void *workspace, size_t workspace_bytes, void *stream)
{
    kda::AttnProblem p;
    kda_status_t st = describe_attn(B, T, Hq, Hkv, d, n_seqs, cu_seqlens != nullptr, dt, &p);
    if (st != KDA_OK) return st;
    if (!scale_ok(scale)) return KDA_ERR_INVALID_ARG;
    if (p.tokens == 0) return KDA_OK;
    if (!q || !k || !v || !o || !lse || !dO || !grad_q || !grad_k || !grad_v)
        return KDA_ERR_INVALID_ARG;
    for (const void *ptr : {q, k, v, o, (const void *)lse, dO, (const void *)grad_q,
                            (const void *)grad_k, (const void *)grad_v, (const void *)workspace})
        if (!aligned(ptr, 16)) return KDA_ERR_ALIGNMENT;
    if (!aligned(cu_seqlens, 4)) return KDA_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < attn_workspace(p, true)) return KDA_ERR_WORKSPACE;
    p.q = q; p.k = k; p.v = v; p.cu_seqlens = cu_seqlens; p.scale = scale;
    st = from_cuda(kda::launch_attn_bwd(p, o, lse, dO, grad_q, grad_k, grad_v, workspace,
                                        static_cast<cudaStream_t>(stream)));
    if (st != KDA_OK || !attn_debug_sync()) return st;
    int code = 0;
    return kda_attn_status(workspace, workspace_bytes, &code, stream);
}

static kda_status_t describe_tree(int N, int R, int Hq, int Hkv, int d, int M, int page_size,
                                  kda_dtype_t dt, kda::TreeProblem *p)
{
    kda_status_t st = heads_ok(Hq, Hkv, d, dt);
    if (st != KDA_OK) return st;
    if (N < 1 || R < 0 || M < 1) return KDA_ERR_INVALID_ARG;
    if (R > 64) return KDA_ERR_UNSUPPORTED;
    const int shift = log2_page(page_size);
    if (shift < 0) return KDA_ERR_UNSUPPORTED;
    if ((long long)M * page_size > (long long)INT32_MAX - 1024 ||
        (long long)N * M > (long long)INT32_MAX || (long long)N * 64 * Hq > (long long)INT32_MAX)
        return KDA_ERR_UNSUPPORTED;
    *p = kda::TreeProblem{};
    p->N = N; p->R = R; p->Hq = Hq; p->Hkv = Hkv; p->d = d; p->M = M; p->page_shift = shift;
    p->dtype = dt;
    return KDA_OK;
}

size_t kda_attn_tree_workspace_size(int N, int R, int Hq, int Hkv, int d, int M, int page_size,
                                    kda_dtype_t dt)
{
    kda::TreeProblem p;
    if (describe_tree(N, R, Hq, Hkv, d, M, page_size, dt, &p) != KDA_OK) return 0;
    return kda::tree_workspace_bytes(p);
}

kda_status_t kda_attn_tree(const void *q, const void *k_pages, const void *v_pages,
                           kda_dtype_t dt, const int32_t *block_table, const int32_t *ctx_lens,
                           const int32_t *parents, int N, int R, int Hq, int Hkv, int d, int P,
                           int M, int page_size, float scale, void *o, float *lse,
                           void *workspace, size_t workspace_bytes, void *stream)
{
    kda::TreeProblem p;
    kda_status_t st = describe_tree(N, R, Hq, Hkv, d, M, page_size, dt, &p);
    if (st != KDA_OK) return st;
    if (P < 1 || !scale_ok(scale)) return KDA_ERR_INVALID_ARG;
    if ((long long)P * Hkv * page_size > (long long)INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (R == 0) return KDA_OK;
    if (!q || !k_pages || !v_pages || !block_table || !ctx_lens || !o) return KDA_ERR_INVALID_ARG;
    for (const void *ptr : {q, k_pages, v_pages, (const void *)o, (const void *)workspace})
        if (!aligned(ptr, 16)) return KDA_ERR_ALIGNMENT;
    for (const void *ptr : {(const void *)block_table, (const void *)ctx_lens,
                            (const void *)parents, (const void *)lse})
        if (!aligned(ptr, 4)) return KDA_ERR_ALIGNMENT;
    const size_t need = kda::tree_workspace_bytes(p);
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    p.q = q; p.k_pages = k_pages; p.v_pages = v_pages; p.table = block_table;
    p.ctx_lens = ctx_lens; p.parents = parents; p.P = P; p.scale = scale; p.o = o; p.lse = lse;
    st = from_cuda(kda::launch_attn_tree(p, workspace, static_cast<cudaStream_t>(stream)));
    if (st != KDA_OK || !attn_debug_sync()) return st;
    int code = 0;
    return kda_attn_status(workspace, workspace_bytes, &code, stream);
}

kda_status_t kda_cache_fork(int32_t *refs, const int32_t *block_table, const int32_t *lens,
                            const int32_t *parents, int N_in, int N_out, int M, int P,
                            int32_t *new_table, int32_t *new_lens, void *stream)
{
    kda_status_t st = table_ok(N_in, M, P);
    if (st == KDA_OK) st = table_ok(N_out, M, P);
    if (st == KDA_OK) st = ints_ok({refs, block_table, lens, parents, new_table, new_lens});
    if (st != KDA_OK) return st;
    const long long in = (long long)N_in * M, out = (long long)N_out * M;
    if (overlap(block_table, in, new_table, out) || overlap(lens, N_in, new_lens, N_out))
        return KDA_ERR_INVALID_ARG;
    return from_cuda(kda::launch_cache_fork(refs, block_table, lens, parents, N_in, N_out, M, P,
                                            new_table, new_lens,
                                            static_cast<cudaStream_t>(stream)));
}

size_t kda_cache_reserve_workspace_size(int N, int M, int P)
{
    if (table_ok(N, M, P) != KDA_OK) return 0;
    return sizeof(int32_t) * (3 * (size_t)P + 3 * (size_t)N + 16);
}

kda_status_t kda_cache_reserve(int32_t *refs, int32_t *block_table, int32_t *lens,
                               const int32_t *add, int N, int M, int P, int page_size,
                               int32_t *copies, int32_t *status, void *workspace,
                               size_t workspace_bytes, void *stream)
{
    kda_status_t st = table_ok(N, M, P);
    if (st != KDA_OK) return st;
    const int shift = log2_page(page_size);
    if (shift < 0 || (long long)M * page_size > (long long)INT32_MAX - 1024)
        return KDA_ERR_UNSUPPORTED;
    st = ints_ok({refs, block_table, lens, add, copies, status});
    if (st != KDA_OK) return st;
    if (!aligned(workspace, 16)) return KDA_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < kda_cache_reserve_workspace_size(N, M, P))
        return KDA_ERR_WORKSPACE;
    return from_cuda(kda::launch_cache_reserve(refs, block_table, lens, add, N, M, P, shift,
                                               copies, status, workspace,
                                               static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_cache_release(int32_t *refs, int32_t *block_table, int32_t *lens,
                               const int32_t *new_lens, int N, int M, int P, int page_size,
                               void *stream)
{
    kda_status_t st = table_ok(N, M, P);
    if (st != KDA_OK) return st;
    const int shift = log2_page(page_size);
    if (shift < 0 || (long long)M * page_size > (long long)INT32_MAX - 1024)
        return KDA_ERR_UNSUPPORTED;
    st = ints_ok({refs, block_table, lens, new_lens});
    if (st != KDA_OK) return st;
    return from_cuda(kda::launch_cache_release(refs, block_table, lens, new_lens, N, M, P, shift,
                                               static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_cache_append(void *k_pages, void *v_pages, kda_dtype_t dt,
                              const int32_t *block_table, const int32_t *start,
                              const void *k_new, const void *v_new, const int32_t *cu_seqlens,
                              int n_seqs, int B, int T, int Hkv, int d, int P, int M,
                              int page_size, void *stream)
{
    kda::PagePool pool;
    kda_status_t st = pool_ok(k_pages, v_pages, dt, Hkv, d, P, M, page_size, &pool);
    if (st != KDA_OK) return st;
    long long tokens;
    int N;
    st = sequences_ok(B, T, cu_seqlens != nullptr, n_seqs, &tokens, &N);
    if (st == KDA_OK) st = table_ok(N, M, P);
    if (st != KDA_OK) return st;
    st = ints_ok({block_table, start});
    if (st != KDA_OK) return st;
    if (tokens == 0) return KDA_OK;
    if (!k_new || !v_new) return KDA_ERR_INVALID_ARG;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(cu_seqlens, 4))
        return KDA_ERR_ALIGNMENT;
    return from_cuda(kda::launch_cache_append(pool, block_table, start, k_new, v_new, cu_seqlens,
                                              N, B, T, M, static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_cache_compact(void *k_pages, void *v_pages, kda_dtype_t dt,
                               const int32_t *block_table, const int32_t *ctx_lens,
                               const int32_t *path, int N, int R, int Hkv, int d, int P, int M,
                               int page_size, int32_t *new_lens, void *stream)
{
    kda::PagePool pool;
    kda_status_t st = pool_ok(k_pages, v_pages, dt, Hkv, d, P, M, page_size, &pool);
    if (st == KDA_OK) st = table_ok(N, M, P);
    if (st != KDA_OK) return st;
    if (R < 1) return KDA_ERR_INVALID_ARG;
    if (R > 1024 || Hkv > 65535) return KDA_ERR_UNSUPPORTED;
    st = ints_ok({block_table, ctx_lens, path, new_lens});
    if (st != KDA_OK) return st;
    // blocks of one row read these while one of them writes its new length
    if (overlap(new_lens, N, ctx_lens, N) || overlap(new_lens, N, path, (long long)N * R) ||
        overlap(new_lens, N, block_table, (long long)N * M))
        return KDA_ERR_INVALID_ARG;
    return from_cuda(kda::launch_cache_compact(pool, block_table, ctx_lens, path, N, R, M,
                                               new_lens, static_cast<cudaStream_t>(stream)));
}

kda_status_t kda_cache_copy_pages(void *k_pages, void *v_pages, kda_dtype_t dt,
                                  const int32_t *copies, int C, int Hkv, int d, int P,
                                  int page_size, void *stream)
{
    kda::PagePool pool;
    kda_status_t st = pool_ok(k_pages, v_pages, dt, Hkv, d, P, 1, page_size, &pool);
    if (st != KDA_OK) return st;
    if (C < 0) return KDA_ERR_INVALID_ARG;
    if (C > 16384) return KDA_ERR_UNSUPPORTED;
    if (C == 0) return KDA_OK;
    st = ints_ok({copies});
    if (st != KDA_OK) return st;
    return from_cuda(kda::launch_cache_copy(pool, copies, C, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
