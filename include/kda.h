/*
 * kda.h — C ABI of the KDA (Kimi Delta Attention) library for NVIDIA B200 (sm_100a).
 *
 * The operation. "Kimi Linear：让长上下文大模型真正实用的线性注意力架构" (juejin.cn),
 * section 三 5️⃣ gives the KDA update rule
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *
 * (beta = learning rate, alpha = forget rate, S = memory state); section 三 1️⃣
 * says the forget rate is per channel (alpha_t[i], one per key channel). The
 * library reads out with the updated state, o_t = scale * S_t^T q_t, and takes
 * the gate in log space, alpha_t = exp(log_alpha_t). S is dk x dv per head, so
 * Diag(alpha_t) scales the dk rows of S.
 *
 * Layouts. Every tensor is a dense, row-major DEVICE buffer, 16-byte aligned:
 *   q, k        [B, T, H, dk]   dtype given by qkv_dtype (fp32 or bf16)
 *   v, o        [B, T, H, dv]   qkv_dtype (o has the same dtype as q, k, v)
 *   log_alpha   [B, T, H, dk]   fp32, expected <= 0 (alpha in (0, 1])
 *   beta        [B, T, H]       fp32
 *   S0, S_final [N, H, dk, dv]  fp32, dv contiguous
 * Sequences: without cu_seqlens, N = B and row b of the batch is one sequence of
 * T tokens. With cu_seqlens (int32 [n_seqs + 1], device memory, cu_seqlens[0] = 0,
 * non-decreasing, cu_seqlens[n_seqs] = T) the batch must have B = 1 and sequence
 * n owns the packed tokens [cu_seqlens[n], cu_seqlens[n+1]); N = n_seqs. Zero-
 * length sequences are allowed (their S_final equals their S0).
 *
 * Supported sizes: dk = dv in {32, 64, 128}. bf16 inputs with dk = dv = 128 run on
 * the tcgen05 tensor-core path; all other supported cases run on the fp32 SIMT
 * path (see kda_chunk_fwd_ex).
 *
 * Ownership and asynchrony. The caller owns every buffer, including the
 * workspace; the library allocates no device memory and never synchronises the
 * stream. Calls are enqueued on `stream` (a cudaStream_t passed as void*; NULL is
 * the legacy default stream) and return once the launches are queued. Buffers
 * must stay valid until the stream reaches that point. Concurrent calls on
 * different streams need separate workspaces.
 *
 * Errors. Arguments are checked on the host before anything is launched; a bad
 * argument returns an error status and launches nothing. A failed launch returns
 * KDA_ERR_CUDA. The library never aborts, exits or traps. Every wait inside the
 * tensor-core kernels is bounded; a wait that runs out makes the kernel return
 * early and records a nonzero code in the prefill workspace's status word, so
 * the results of that call are not valid. The word is read by
 * kda_chunk_fwd_status (after the call) or, with KDA_DEBUG_SYNC=1 in the
 * environment, by every prefill call itself, which then waits for its work and
 * returns KDA_ERR_DEVICE_STATUS.
 */
#ifndef KDA_B200_H
#define KDA_B200_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,   /* null pointer, non-positive size, bad cu_seqlens shape */
    KDA_ERR_UNSUPPORTED = 2,   /* head size or dtype the library does not implement */
    KDA_ERR_ALIGNMENT = 3,     /* a buffer is not 16-byte aligned */
    KDA_ERR_WORKSPACE = 4,     /* workspace missing or smaller than required */
    KDA_ERR_CUDA = 5,          /* a CUDA runtime call or kernel launch failed */
    KDA_ERR_DEVICE_STATUS = 6  /* a kernel gave up a bounded wait: results invalid */
} kda_status_t;

typedef enum { KDA_DTYPE_F32 = 0, KDA_DTYPE_BF16 = 1 } kda_dtype_t;

/* Prefill algorithm selector for kda_chunk_fwd_ex. */
typedef enum {
    KDA_ALGO_AUTO = 0,    /* tcgen05 path when supported, else SIMT */
    KDA_ALGO_SIMT = 1,    /* fp32 CUDA-core path: any supported dtype and size */
    KDA_ALGO_TCGEN05 = 2, /* tensor-core path: bf16, dk = dv = 128 only */
    KDA_ALGO_TCGEN05_SEQUENTIAL = 3  /* tensor-core path without the time split */
} kda_algo_t;

/* Human-readable name of a status code (static storage; never NULL). */
const char *kda_status_string(kda_status_t status);

/* Library version as major*10000 + minor*100 + patch. */
int kda_version(void);

/* Number of kernels this library has launched in this process so far (all
 * entry points, all devices). Differences of two readings count the launches
 * of the calls made in between. */
unsigned long long kda_launch_count(void);

/*
 * Device status of the last prefill that used `workspace` (any kda_*chunk_fwd*
 * entry point, either phase). The library defines no counterpart on the pages;
 * it reports whether the kernels' own failure detection fired. Reads the
 * workspace's status word on `stream` and waits for the stream. The prepare
 * phase clears the word; a later failure in either phase sets it to a nonzero
 * code (the first failing wait's), which stays until the next prepare.
 *   workspace, workspace_bytes  the prefill's workspace (>= 256 bytes)
 *   device_code                 receives the word (0: no wait ran out)
 * Returns KDA_OK, KDA_ERR_DEVICE_STATUS when the word is nonzero, or an
 * argument / CUDA error.
 */
kda_status_t kda_chunk_fwd_status(const void *workspace, size_t workspace_bytes,
                                  int *device_code, void *stream);

/*
 * Debugging aid for the failure path (process-wide; not needed in normal use):
 * `polls` replaces the poll limit of every bounded wait in the tensor-core
 * kernels launched afterwards (0 restores the default of 2^20 polls), and a
 * nonzero `starve_carry` makes the sequential kernel's copy producer (and the
 * tensor-core attention kernels' loading warps) issue no copies, so that the
 * first wait on a copy runs out while nothing asynchronous is in flight. The kernels then return early and the status word
 * reports the failure. Always returns KDA_OK.
 */
kda_status_t kda_debug_set_wait_limit(unsigned int polls, int starve_carry);

/*
 * Workspace bytes that kda_chunk_fwd needs for this problem, i.e. for the path
 * KDA_ALGO_AUTO selects (0 on invalid sizes). The workspace holds the per-chunk intermediate matrices of the
 * chunked form between the chunk-parallel and the sequential kernel; it is
 * device memory owned by the caller, needs no initialisation and may be reused
 * across calls on the same stream. For varlen calls pass B = 1, T = total
 * packed tokens and n_seqs = number of sequences; otherwise n_seqs is ignored.
 */
size_t kda_chunk_fwd_workspace_size(int B, int T, int H, int dk, int dv, int n_seqs,
                                    kda_dtype_t qkv_dtype);

/* Workspace bytes kda_chunk_fwd_ex needs with the given kda_algo_t (the size for
 * the path that algo selects; KDA_ALGO_AUTO gives the same value as
 * kda_chunk_fwd_workspace_size). 0 on invalid sizes or an unsupported algo. */
size_t kda_chunk_fwd_workspace_size_ex(int B, int T, int H, int dk, int dv, int n_seqs,
                                       kda_dtype_t qkv_dtype, int algo);

/*
 * Chunked prefill: runs the recurrence over every sequence from S0 (NULL = zero
 * state), writes o for every token and, if S_final is not NULL, the state after
 * each sequence's last token. Source: the update rule above ("Kimi Linear"
 * juejin.cn page, section 三 5️⃣), evaluated in the exact chunked form (64-token
 * chunks, a triangular solve per chunk, fp32 state carried on chip between
 * chunks); results equal the token-by-token recurrence up to rounding.
 *
 *   q, k, v, o       qkv_dtype device buffers (layouts above)
 *   log_alpha, beta  fp32 device buffers
 *   S0, S_final      fp32 [N, H, dk, dv] or NULL; S0 and S_final may alias
 *   cu_seqlens       int32 device buffer [n_seqs + 1] or NULL (then n_seqs is ignored)
 *   scale            read-out scale (commonly dk^-0.5)
 *   workspace        >= kda_chunk_fwd_workspace_size(...) bytes of device memory
 *   stream           cudaStream_t or NULL
 * T = 0 is allowed and only copies S0 to S_final (zeros without S0).
 */
kda_status_t kda_chunk_fwd(const void *q, const void *k, const void *v, kda_dtype_t qkv_dtype,
                           const float *log_alpha, const float *beta, const float *S0,
                           const int32_t *cu_seqlens, int n_seqs, int B, int T, int H,
                           int dk, int dv, float scale, void *o, float *S_final,
                           void *workspace, size_t workspace_bytes, void *stream);

/* kda_chunk_fwd with an explicit algorithm choice (kda_algo_t). Asking for
 * KDA_ALGO_TCGEN05 on a problem it does not support returns KDA_ERR_UNSUPPORTED.
 * On the tensor-core path (AUTO and TCGEN05) the sequential phase is split in
 * time when a problem has so few (sequence, head) chains that most SMs would
 * idle (see kda_chunk_fwd_timesplit); KDA_ALGO_TCGEN05_SEQUENTIAL never splits. */
kda_status_t kda_chunk_fwd_ex(const void *q, const void *k, const void *v, kda_dtype_t qkv_dtype,
                              const float *log_alpha, const float *beta, const float *S0,
                              const int32_t *cu_seqlens, int n_seqs, int B, int T, int H,
                              int dk, int dv, float scale, void *o, float *S_final,
                              void *workspace, size_t workspace_bytes, int algo,
                              void *stream);

/*
 * Chunked prefill on the tensor-core path (bf16, dk = dv = 128) with the
 * sequential phase split into `segments` time segments per sequence, so that
 * a long sequence with few heads keeps more SMs busy. The
 * sequential chunk walk of one (sequence, head) only runs on as many SMs as
 * there are 64-column halves of its state; the split runs it in two parallel
 * passes instead. Pass 1: segment 0 from S0 with outputs, and for every later
 * segment the state from a zero start and the segment's transition (the
 * product of the chunk steps' linear parts, a 128 x 128 matrix carried like a
 * state that starts at the identity). A combine kernel then forms each
 * segment's true entry state in fp32 (end = transition x entry + zero-start
 * state). Pass 2: every later segment again from its entry state, with
 * outputs. Results equal kda_chunk_fwd_ex's up to rounding. The recurrence is
 * the one of the "Kimi Linear" juejin.cn page, section 三 5️⃣; the pages give no
 * time split (the chunk-parallel form is section 三 2️⃣'s remark).
 *   segments   0: choose automatically (as KDA_ALGO_TCGEN05), 1: no split,
 *              2..64: that many segments per sequence (sequences with fewer
 *              chunks get empty segments)
 * Other arguments, layouts and errors as kda_chunk_fwd_ex; the workspace is
 * kda_chunk_fwd_timesplit_workspace_size bytes (it grows by 192 KB per segment,
 * sequence and head). Unsupported problems return KDA_ERR_UNSUPPORTED.
 */
size_t kda_chunk_fwd_timesplit_workspace_size(int B, int T, int H, int dk, int dv, int n_seqs,
                                              kda_dtype_t qkv_dtype, int segments);
kda_status_t kda_chunk_fwd_timesplit(const void *q, const void *k, const void *v,
                                     kda_dtype_t qkv_dtype, const float *log_alpha,
                                     const float *beta, const float *S0,
                                     const int32_t *cu_seqlens, int n_seqs, int B, int T, int H,
                                     int dk, int dv, float scale, void *o, float *S_final,
                                     void *workspace, size_t workspace_bytes, int segments,
                                     void *stream);

/*
 * The two phases of kda_chunk_fwd_ex, exported separately (same arguments, same
 * workspace). kda_chunk_fwd_ex(...) is exactly kda_chunk_fwd_prepare(...)
 * followed by kda_chunk_fwd_carry(...) on the same stream.
 *   prepare: the chunk-parallel phase. Plans the sequences and, for every
 *            64-token chunk and head, forms the gate cumulative sums, the
 *            intra-chunk matrices and the triangular solve, storing the chunk's
 *            intermediates in the workspace. Reads q, k, v, log_alpha, beta.
 *   carry:   the sequential phase. Walks each sequence's chunks in order with
 *            the fp32 state on chip, writing o and S_final. Reads the workspace,
 *            S0 and cu_seqlens-derived plan; does not read q, k, v or the gates.
 * Useful to time the phases or to run the chunk-parallel phase ahead of time.
 */
kda_status_t kda_chunk_fwd_prepare(const void *q, const void *k, const void *v,
                                   kda_dtype_t qkv_dtype, const float *log_alpha,
                                   const float *beta, const float *S0,
                                   const int32_t *cu_seqlens, int n_seqs, int B, int T, int H,
                                   int dk, int dv, float scale, void *o, float *S_final,
                                   void *workspace, size_t workspace_bytes, int algo,
                                   void *stream);
kda_status_t kda_chunk_fwd_carry(const void *q, const void *k, const void *v,
                                 kda_dtype_t qkv_dtype, const float *log_alpha,
                                 const float *beta, const float *S0,
                                 const int32_t *cu_seqlens, int n_seqs, int B, int T, int H,
                                 int dk, int dv, float scale, void *o, float *S_final,
                                 void *workspace, size_t workspace_bytes, int algo,
                                 void *stream);

/*
 * Recurrent decode: one new token for each of N independent sequences. Applies
 * the update rule once per (sequence, head) to the state S in place and writes
 * o = scale * S_new^T q. Source: the same update rule; the kernel evaluates it
 * in one pass over S using o = scale * (S'^T q + (k^T q) u) with
 * S' = Diag(alpha) S and u = beta (v - S'^T k), so S is read once and written
 * once.
 *
 *   q, k        qkv_dtype [N, H, dk]      v, o   qkv_dtype [N, H, dv]
 *   log_alpha   fp32 [N, H, dk]           beta   fp32 [N, H]
 *   S           fp32 [N, H, dk, dv], read and overwritten
 */
kda_status_t kda_decode_step(const void *q, const void *k, const void *v, kda_dtype_t qkv_dtype,
                             const float *log_alpha, const float *beta, float *S, int N,
                             int H, int dk, int dv, float scale, void *o, void *stream);

/*
 * Multi-token decode: T new tokens for each of N independent sequences, applied
 * in order with the state held on chip between them; S is read once and
 * written once per call. Source: the same update rule, applied T times (each
 * token as in kda_decode_step). Equals T chained kda_decode_step calls, and
 * kda_chunk_fwd with B = N, S0 = S_final = S (up to rounding); meant for small
 * T (speculative verification, continuing a prefill by a few tokens), where the
 * chunked prefill would spend most of its time on per-chunk intermediates.
 *
 *   q, k        qkv_dtype [N, T, H, dk]   v, o   qkv_dtype [N, T, H, dv]
 *   log_alpha   fp32 [N, T, H, dk]        beta   fp32 [N, T, H]
 *   S           fp32 [N, H, dk, dv], read and overwritten
 * Errors as kda_decode_step; T = 0 returns KDA_OK without touching anything
 * (only S must then be non-null). N * T must fit in a signed 32-bit int.
 */
kda_status_t kda_decode_tokens(const void *q, const void *k, const void *v,
                               kda_dtype_t qkv_dtype, const float *log_alpha,
                               const float *beta, float *S, int N, int T, int H, int dk,
                               int dv, float scale, void *o, void *stream);

/*
 * Gated DeltaNet (GDN) variants: the same update rule with one forget rate per
 * token and head instead of one per channel, i.e. Diag(alpha_t) = alpha_t I.
 * Source: "Kimi Linear：让长上下文大模型真正实用的线性注意力架构" (juejin.cn),
 * section 三 1️⃣ (GDN has a single forget rate per head; KDA refines it per
 * channel) with the rule of section 三 5️⃣. Results equal the KDA entry points
 * given log_alpha broadcast over the dk channels.
 *
 * kda_gdn_chunk_fwd: arguments, layouts, workspace (kda_chunk_fwd_workspace_size_ex
 * with the same algo), errors and paths as kda_chunk_fwd_ex, except
 *   log_alpha   fp32 [B, T, H]  (one log forget rate per token and head, <= 0)
 * On the tensor-core path (bf16, dk = dv = 128) the scalar decay comes out of
 * the channel contraction, so its chunk-parallel phase is a lighter kernel than
 * the per-channel one; the sequential phase is shared.
 *
 * kda_gdn_chunk_fwd_prepare: its chunk-parallel phase alone; the sequential
 * phase, which reads only the workspace, S0 and the plan, is kda_chunk_fwd_carry
 * with the same arguments.
 *
 * kda_gdn_decode_tokens: as kda_decode_tokens, except
 *   log_alpha   fp32 [N, T, H]
 */
kda_status_t kda_gdn_chunk_fwd(const void *q, const void *k, const void *v,
                               kda_dtype_t qkv_dtype, const float *log_alpha,
                               const float *beta, const float *S0, const int32_t *cu_seqlens,
                               int n_seqs, int B, int T, int H, int dk, int dv, float scale,
                               void *o, float *S_final, void *workspace,
                               size_t workspace_bytes, int algo, void *stream);
kda_status_t kda_gdn_chunk_fwd_prepare(const void *q, const void *k, const void *v,
                                       kda_dtype_t qkv_dtype, const float *log_alpha,
                                       const float *beta, const float *S0,
                                       const int32_t *cu_seqlens, int n_seqs, int B, int T,
                                       int H, int dk, int dv, float scale, void *o,
                                       float *S_final, void *workspace, size_t workspace_bytes,
                                       int algo, void *stream);
kda_status_t kda_gdn_decode_tokens(const void *q, const void *k, const void *v,
                                   kda_dtype_t qkv_dtype, const float *log_alpha,
                                   const float *beta, float *S, int N, int T, int H, int dk,
                                   int dv, float scale, void *o, void *stream);

/*
 * Backward of the prefill (for training; the pages state only the forward rule,
 * so this is the rule's derivative): the gradients of
 *     L = <dO, o> + <dS_final, S_final>
 * with respect to q, k, v, log_alpha, beta and S0, for the arguments of
 * kda_chunk_fwd (same layouts, sequences and scale). Computed in fp32 on CUDA
 * cores for every supported head size, by the chunk-parallel form below
 * (KDA_BWD_AUTO; results are deterministic). The token walk (KDA_BWD_TOKEN,
 * through kda_chunk_bwd_ex) replays the states from checkpoints kept every 32
 * tokens and adds per-slice partial gradients (dk / 32 slices of 32 value
 * columns) in a fixed order; at d = 128 its workspace is about 8.2 KB per
 * token and head plus 2.2 MB per (sequence, head), e.g. 2.2 GB for B = 1,
 * H = 32, T = 8192.
 *   dO              qkv_dtype [B, T, H, dv]
 *   dS_final        fp32 [N, H, dk, dv] or NULL (zero)
 *   grad_q, grad_k  fp32 [B, T, H, dk]       grad_v     fp32 [B, T, H, dv]
 *   grad_log_alpha  fp32 [B, T, H, dk]       grad_beta  fp32 [B, T, H]
 *   grad_S0         fp32 [N, H, dk, dv] or NULL (not returned)
 * Workspace: kda_chunk_bwd_workspace_size bytes (that of KDA_BWD_AUTO). Errors as
 * kda_chunk_fwd_ex.
 * Tokens outside every sequence (cu_seqlens ending before B*T) are not written.
 * kda_gdn_chunk_bwd: the same for one gate per token and head (log_alpha and
 * grad_log_alpha fp32 [B, T, H]).
 */
size_t kda_chunk_bwd_workspace_size(int B, int T, int H, int dk, int dv, int n_seqs,
                                    kda_dtype_t qkv_dtype);
/*
 * Backward algorithms. KDA_BWD_TOKEN walks every sequence token by token (the
 * states replayed from checkpoints). KDA_BWD_CHUNKED goes through the chunked
 * form of the rule (what kda_chunk_bwd and kda_gdn_chunk_bwd run, and
 * KDA_BWD_AUTO): per-chunk records (W, U~, e^g q, e^{g_C - g} k, P, e^{g_C}), a forward
 * and a reverse walk over the chunks (one CTA per sequence, head and 32 value
 * columns), then the token gradients of all chunks in parallel; fp32 CUDA-core
 * arithmetic where every exponential is of a non-positive number, so any gate
 * is safe. Its workspace holds, per (chunk, head) at d = 128, the record
 * (148 KB), the entry state and chunk-end gradient (64 KB each), U and dU
 * (32 KB each) and the token-gradient products (115 KB): about 7.1 KB per
 * token and head.
 */
enum { KDA_BWD_AUTO = 0, KDA_BWD_TOKEN = 1, KDA_BWD_CHUNKED = 2 };
/* Workspace bytes for a backward algorithm (0 on invalid sizes or algo). */
size_t kda_chunk_bwd_workspace_size_ex(int B, int T, int H, int dk, int dv, int n_seqs,
                                       kda_dtype_t qkv_dtype, int algo);
/* kda_chunk_bwd (gate_per_channel 1) or kda_gdn_chunk_bwd (0) with an explicit
 * algorithm; the workspace is kda_chunk_bwd_workspace_size_ex(..., algo) bytes.
 * An unknown algo returns KDA_ERR_INVALID_ARG before any device work. */
kda_status_t kda_chunk_bwd_ex(const void *q, const void *k, const void *v, kda_dtype_t qkv_dtype,
                              const float *log_alpha, const float *beta, const float *S0,
                              const int32_t *cu_seqlens, int n_seqs, int B, int T, int H,
                              int dk, int dv, float scale, const void *dO,
                              const float *dS_final, float *grad_q, float *grad_k,
                              float *grad_v, float *grad_log_alpha, float *grad_beta,
                              float *grad_S0, void *workspace, size_t workspace_bytes,
                              int gate_per_channel, int algo, void *stream);
kda_status_t kda_chunk_bwd(const void *q, const void *k, const void *v, kda_dtype_t qkv_dtype,
                           const float *log_alpha, const float *beta, const float *S0,
                           const int32_t *cu_seqlens, int n_seqs, int B, int T, int H, int dk,
                           int dv, float scale, const void *dO, const float *dS_final,
                           float *grad_q, float *grad_k, float *grad_v, float *grad_log_alpha,
                           float *grad_beta, float *grad_S0, void *workspace,
                           size_t workspace_bytes, void *stream);
kda_status_t kda_gdn_chunk_bwd(const void *q, const void *k, const void *v,
                               kda_dtype_t qkv_dtype, const float *log_alpha,
                               const float *beta, const float *S0, const int32_t *cu_seqlens,
                               int n_seqs, int B, int T, int H, int dk, int dv, float scale,
                               const void *dO, const float *dS_final, float *grad_q,
                               float *grad_k, float *grad_v, float *grad_log_alpha,
                               float *grad_beta, float *grad_S0, void *workspace,
                               size_t workspace_bytes, void *stream);

/*
 * kda_chunk_fwd_noalloc — the chunked prefill for callers that cannot allocate
 * device memory (no counterpart in the paper; it exists for callers such as a
 * plugin whose host application owns all device memory, or code that must not
 * trigger the device synchronisation an allocation can cause).
 *
 * Same arguments and results as kda_chunk_fwd_ex, minus the workspace: the
 * library uses a fixed scratch array of KDA_NOALLOC_SCRATCH_BYTES in its own
 * device memory, held by every GPU that loads the library until the process
 * exits. The caller still provides every input and output buffer. The call
 * allocates nothing (no cudaMalloc, no cudaFree, no allocating library call).
 *   - Problems whose workspace for the same algo
 *     (kda_chunk_fwd_workspace_size_ex with this call's algo) exceeds
 *     KDA_NOALLOC_SCRATCH_BYTES are rejected on the host with
 *     KDA_ERR_WORKSPACE before anything is launched; invalid arguments are
 *     rejected on the host as kda_chunk_fwd_ex rejects them.
 *   - The first call on each device (and the first after the device's
 *     context was reset) looks up the scratch array's device address
 *     (cudaGetSymbolAddress, with that device current); make that first call
 *     before any stream capture on the device.
 *   - With KDA_DEBUG_SYNC=1 in the environment the call waits for its work
 *     and reports a bounded wait that ran out as KDA_ERR_DEVICE_STATUS, as
 *     kda_chunk_fwd_ex does.
 *   - Every call shares the one array and leaves its contents behind. The
 *     kernels initialise every part of it they read, so nothing carries over
 *     from one call to the next; but calls whose execution overlaps on the GPU
 *     (different streams, or different host threads) race on the array and
 *     must be serialised by the caller.
 */
#define KDA_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

kda_status_t kda_chunk_fwd_noalloc(const void *q, const void *k, const void *v,
                                   kda_dtype_t qkv_dtype, const float *log_alpha,
                                   const float *beta, const float *S0,
                                   const int32_t *cu_seqlens, int n_seqs, int B, int T, int H,
                                   int dk, int dv, float scale, void *o, float *S_final,
                                   int algo, void *stream);

/*
 * Full attention. A hybrid model interleaves the KDA layers with full-attention
 * layers without position encoding ("Kimi Linear" juejin.cn page, section 三 3️⃣ and
 * 4️⃣); the calls below are that layer's token mixing with grouped heads: query
 * head h reads key/value head h / (Hq / Hkv). The pages give the definition only
 * (softmax(Q K^T / sqrt(d)) V); the paged cache is this library's own.
 *
 * Layouts (dense, row-major, 16-byte aligned device buffers; dtype fp32 or bf16;
 * d in {32, 64, 128}; Hq a multiple of Hkv):
 *   q, o, dO, grad_q          [B, T, Hq, d]      dtype
 *   k, v, grad_k, grad_v      [B, T, Hkv, d]     dtype
 *   lse                       [B, T, Hq]         fp32, natural logarithm
 * Sequences (cu_seqlens, n_seqs) as for the prefill; offsets are sanitised on the
 * device in the same way. `scale` must be positive and finite. Sums, softmax
 * statistics and accumulators are fp32; with bf16 inputs the probabilities (and
 * in the backward the score gradients) are rounded to bf16 as operands of the
 * tensor-core products. Results do not depend on the order of execution: the same call gives
 * the same bits. How sums are split (dK and dV over a group's heads, a tree's over its keys)
 * goes by the sizes of the whole call, so a sequence may be rounded differently next to others.
 *
 * kda_attn_fwd: causal attention of every sequence,
 *     s_rc = scale <q_r, k_c> (c <= r),  lse_r = log sum_c e^(s_rc),
 *     o_r = sum_c e^(s_rc - lse_r) v_c.
 * What keys and values that a row does not see hold (infinities and NaN included) cannot
 * change its result beyond rounding. Tokens outside every sequence are not written.
 * lse may be NULL. T = 0 returns KDA_OK without touching anything.
 *
 * kda_attn_bwd: the gradients of <dO, o> with respect to q, k and v in the inputs'
 * dtype, from the forward's inputs, its o and its lse:
 *     p_rc = e^(s_rc - lse_r),  D_r = <dO_r, o_r>,  ds_rc = scale p_rc (<dO_r, v_c> - D_r),
 *     grad_q_r = sum_c ds_rc k_c,  grad_k_c = sum_r ds_rc q_r,  grad_v_c = sum_r p_rc dO_r
 * (grad_k and grad_v summed over the group's query heads in fp32 before rounding). D comes
 * from the o that is given, rounded as it is; in bf16 p and ds are rounded to bf16 for the
 * products that sum them, which are in fp32. Gradients of tokens outside every sequence are not
 * written; what q, k, v, o, lse and dO hold there does not matter.
 *
 * Errors as for kda_chunk_fwd. kda_attn_status reads the status word of the last
 * kda_attn_fwd, kda_attn_bwd or kda_attn_tree on a workspace, as kda_chunk_fwd_status does.
 */
size_t kda_attn_fwd_workspace_size(int B, int T, int Hq, int Hkv, int d, int n_seqs,
                                   kda_dtype_t dtype);
kda_status_t kda_attn_fwd(const void *q, const void *k, const void *v, kda_dtype_t dtype,
                          const int32_t *cu_seqlens, int n_seqs, int B, int T, int Hq, int Hkv,
                          int d, float scale, void *o, float *lse, void *workspace,
                          size_t workspace_bytes, void *stream);
size_t kda_attn_bwd_workspace_size(int B, int T, int Hq, int Hkv, int d, int n_seqs,
                                   kda_dtype_t dtype);
kda_status_t kda_attn_bwd(const void *q, const void *k, const void *v, const void *o,
                          const float *lse, const void *dO, kda_dtype_t dtype,
                          const int32_t *cu_seqlens, int n_seqs, int B, int T, int Hq, int Hkv,
                          int d, float scale, void *grad_q, void *grad_k, void *grad_v,
                          void *workspace, size_t workspace_bytes, void *stream);
kda_status_t kda_attn_status(const void *workspace, size_t workspace_bytes, int *device_code,
                             void *stream);

/*
 * The paged key/value cache of one full-attention layer:
 *   k_pages, v_pages  [P, Hkv, page_size, d]  dtype; page_size a power of two, 1..1024
 *   block_table       int32 [N, M]   page of each page_size tokens of a sequence (row);
 *                                    entries behind the last page hold -1
 *   lens              int32 [N]      tokens in each row
 *   refs              int32 [P]      rows that hold each page; 0: the page is free
 * One block_table, lens and refs serve the pools of all layers. A page number outside
 * [0, P) reads as no page: its tokens are not attended to, not written and not counted.
 *
 * kda_attn_tree: attention of R drafted tokens per sequence over its cache. Token i of
 * sequence n sits at position ctx_lens[n] + i, where its key and value already are
 * (kda_cache_append). It attends to the positions [0, ctx_lens[n]), to itself and to
 * the drafted tokens above it in the tree: parents[n, i] is its parent's index (less
 * than i), or -1 where the parent is the last cached token. Any other value makes the
 * token absent, and with it all tokens that descend from it: absent tokens, and tokens
 * that find no key at all, get o = 0 and lse = -inf. parents = NULL is a chain (parent
 * i - 1); R = 1 with it is the ordinary decode step.
 *   q, o      [N, R, Hq, d]  dtype          lse  fp32 [N, R, Hq] or NULL
 *   ctx_lens  int32 [N], clamped to [0, M * page_size]
 *   parents   int32 [N, R] or NULL          R <= 64
 * R = 0 returns KDA_OK without touching anything.
 */
size_t kda_attn_tree_workspace_size(int N, int R, int Hq, int Hkv, int d, int M, int page_size,
                                    kda_dtype_t dtype);
kda_status_t kda_attn_tree(const void *q, const void *k_pages, const void *v_pages,
                           kda_dtype_t dtype, const int32_t *block_table, const int32_t *ctx_lens,
                           const int32_t *parents, int N, int R, int Hq, int Hkv, int d, int P,
                           int M, int page_size, float scale, void *o, float *lse,
                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * Pages of the cache. The table calls work on block_table, lens and refs once for all
 * layers; the data calls move keys and values of one layer's pools. Everything stays on
 * the device and is deterministic.
 *
 * kda_cache_fork (table): row n of the new table (N_out rows) becomes a copy of row
 * parents[n] of the old one, sharing all its pages (parents outside [0, N_in) give an
 * empty row); then the old rows end. A row taken twice is forked, one taken by nobody
 * is freed. The new table and lens must not overlap the old ones.
 *
 * kda_cache_reserve (table): makes room for add[n] >= 0 more tokens in every row and
 * adds them to lens. Pages are the lowest-numbered free ones, handed out row after
 * row. A last page that is partly filled and held by other rows too is replaced by a
 * new one first; copies[n] = (old page, new page) then, else (-1, -1): pass it to
 * kda_cache_copy_pages for every layer (of more than 16384 rows in parts: these pairs do not
 * depend on one another). Of several rows that share such a page and
 * together are all its holders, the last one keeps it. All or nothing: status[0] = 0,
 * or the number of pages that are missing, or -1 - n for the first row n that would
 * need more than M pages; where it is not 0, nothing has changed and copies is all -1.
 *
 * kda_cache_release (table): cuts every row to min(lens[n], new_lens[n]) tokens and
 * lets go of the pages behind (new_lens = 0 frees the row).
 *
 * kda_cache_append (data): writes k_new and v_new ([B, T, Hkv, d], sequences as for the
 * prefill, offsets sanitised like the prompt calls') into the rows' pages, sequence n from
 * position start[n] on.
 *
 * kda_cache_compact (data): keeps the drafted tokens path[n, 0], path[n, 1], ... (an
 * increasing list of indices below R, ended by the first entry that is not one) of row
 * n, whose drafts begin at position ctx_lens[n]: moves them together to ctx_lens[n],
 * ctx_lens[n] + 1, ..., and writes ctx_lens[n] plus their number to new_lens[n]. new_lens
 * must not overlap ctx_lens, path or block_table.
 *
 * kda_cache_copy_pages (data): copies page copies[c, 0] to page copies[c, 1] for every
 * c < C (at most 16384). A pair with a number outside [0, P), with a destination that
 * an earlier pair already has, or with one that is the source of another pair is left out.
 */
kda_status_t kda_cache_fork(int32_t *refs, const int32_t *block_table, const int32_t *lens,
                            const int32_t *parents, int N_in, int N_out, int M, int P,
                            int32_t *new_table, int32_t *new_lens, void *stream);
size_t kda_cache_reserve_workspace_size(int N, int M, int P);
kda_status_t kda_cache_reserve(int32_t *refs, int32_t *block_table, int32_t *lens,
                               const int32_t *add, int N, int M, int P, int page_size,
                               int32_t *copies, int32_t *status, void *workspace,
                               size_t workspace_bytes, void *stream);
kda_status_t kda_cache_release(int32_t *refs, int32_t *block_table, int32_t *lens,
                               const int32_t *new_lens, int N, int M, int P, int page_size,
                               void *stream);
kda_status_t kda_cache_append(void *k_pages, void *v_pages, kda_dtype_t dtype,
                              const int32_t *block_table, const int32_t *start,
                              const void *k_new, const void *v_new, const int32_t *cu_seqlens,
                              int n_seqs, int B, int T, int Hkv, int d, int P, int M,
                              int page_size, void *stream);
kda_status_t kda_cache_compact(void *k_pages, void *v_pages, kda_dtype_t dtype,
                               const int32_t *block_table, const int32_t *ctx_lens,
                               const int32_t *path, int N, int R, int Hkv, int d, int P, int M,
                               int page_size, int32_t *new_lens, void *stream);
kda_status_t kda_cache_copy_pages(void *k_pages, void *v_pages, kda_dtype_t dtype,
                                  const int32_t *copies, int C, int Hkv, int d, int P,
                                  int page_size, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_B200_H */
