/*
 * nsp.h -- C ABI of the GB300 (sm_103a) varlen attention hot path.
 *
 * One GPU, caller-owned device memory, caller stream.  The library computes:
 *
 *   - document-masked ("varlen") causal self-attention over a packed token
 *     stream, forward and backward, with grouped-query heads;
 *   - the chunk-partial attention of ring-style sequence parallelism (a query
 *     range against a key range) and the log-sum-exp merge of such partials;
 *   - the Ulysses seq-sharded -> head-sharded layout permutation;
 *   - a differential attention layer's operators: rotary positions, the
 *     learned difference weight, differential attention forward and backward,
 *     and the norm of each head's output;
 *   - a packed post-training step's operators next to attention: the norm of
 *     query and key heads with the rotation in the same pass, log-probabilities
 *     of given tokens, the clipped policy loss, the preference loss over pairs of
 *     documents, and the norm and clipping of many gradients.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Layouts (row-major, innermost last):
 *   q, out, dout, dq : [tokens, Hq,  d]      k, v, dk, dv : [tokens, Hkv, d]
 *   lse              : [Hq, tokens] float32 (natural log of the scaled scores)
 *   cu_seqlens       : int32 [ndoc + 1], device memory, cu[0] = 0,
 *                      non-decreasing, cu[ndoc] = total tokens of the stream.
 *                      Zero-length documents are allowed.
 * Element types: NSP_BF16 inputs are computed with float32 accumulation;
 *   NSP_F32 inputs with true float32 arithmetic (no TF32).
 * Ownership: the caller allocates and frees every buffer, including the
 *   workspace.  The library allocates no device or host memory, never
 *   synchronises the stream (except nsp_status_query) and enqueues all work
 *   on `stream`.  Calls on different streams with different workspaces may
 *   run concurrently.
 * Alignment: every device pointer must be 16-byte aligned; the bf16 outputs
 * of attention (out of a forward, dq / dk / dv of a backward) must be
 * 32-byte aligned (they are written as 32-byte vectors).
 * Errors: scalar, alignment and size errors are detected on the host and
 *   returned before anything is enqueued.  Errors in device data (a bad
 *   cu_seqlens) are detected by the first kernel, recorded in the status word
 *   at the start of the workspace, and make every later kernel of the call a
 *   no-op; nsp_status_query() returns that word.  A CUDA launch failure
 *   returns NSP_ERR_CUDA.  Every device-side wait is bounded: if a bound
 *   expires the kernel records NSP_ERR_TIMEOUT and returns (it never traps).
 *
 * Pages the operations come from (cited by title and section):
 *   [NSP]  "NSP: Accelerating Variable-Length LLM Training via Nested Sequence
 *          Parallelism" -- Sec. 2.2 Sequence Packing, Sec. 2.3 recomputation.
 *   [BASP] "BASP: Communication-Efficient Batch-Aware Sequence Parallelism for
 *          LLM Training" -- Sec. II-A Scaled Dot-Product Attention, Sec. II-C
 *          DeepSpeed Ulysses.
 *   [HSAP] "HSAP: A Hierachical Sequence-aware Parallelism for Hybrid-Context
 *          Generative Models" -- Sec. 2.1 Sequence Packing (cu_len),
 *          Sec. 2.2.1 InterSP (ring, online accumulation), Sec. 2.2.2 IntraSP
 *          (all-to-all), Sec. 3.2 attention-block patterns, Limitations
 *          (fusing copy and rescale).
 */
#ifndef NSP_H_
#define NSP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t; 0 is the legacy default stream. */
typedef struct CUstream_st* nsp_stream_t;

typedef enum {
  NSP_OK = 0,
  NSP_ERR_INVALID = 1,      /* bad scalar argument or bad cu_seqlens contents */
  NSP_ERR_UNSUPPORTED = 2,  /* valid but not implemented (e.g. d not 64/128)  */
  NSP_ERR_WORKSPACE = 3,    /* workspace missing or smaller than required     */
  NSP_ERR_CUDA = 4,         /* a CUDA call or launch failed                   */
  NSP_ERR_TIMEOUT = 5,      /* a bounded device-side wait expired             */
  NSP_ERR_ALIGN = 6         /* a pointer is not 16 (bf16 outputs: 32)-byte aligned */
} nsp_status;

typedef enum { NSP_F32 = 0, NSP_BF16 = 1 } nsp_dtype;

/* Human-readable name of a status code (static string, never NULL). */
const char* nsp_status_str(int32_t status);

/* Library version string, e.g. "nsp 0.1 sm_103a". */
const char* nsp_version(void);

/* Number of kernels this library has launched in this process so far (all
 * devices, all streams; a relaxed atomic counter).  Lets callers and
 * benchmarks count the library's own launches. */
int64_t nsp_kernel_launches(void);

/* Number of attention kernels (forward, dK/dV and dQ kernels) this library
 * has launched in this process on the tensor-core path (tensor_core = 1:
 * tcgen05, TMEM, TMA) or on the CUDA-core path (tensor_core = 0: float32
 * I/O, or no tensor-map support in the driver).
 * Lets a caller see which path its calls took. */
int64_t nsp_path_launches(int32_t tensor_core);

/* Bound, in GPU clock cycles, of every wait inside the tensor-core attention
 * kernels (a thread waiting for a copy, a product or another role of its
 * block).  When a wait runs longer, the kernel records NSP_ERR_TIMEOUT in the
 * workspace status word (read it with nsp_status_query), every role of the
 * block stops, waits for the copies and products it already issued, frees its
 * tensor memory and returns: the context stays usable and the next call on
 * the same workspace starts afresh.  The outputs of the failed call are
 * unspecified.
 *
 * It makes the kernels' failure detection testable: the default (cycles < 0
 * restores it) is 4e9 cycles, about 2 s,
 * far beyond any legitimate wait; a tiny bound (0 to a few hundred cycles)
 * makes a call's first wait that is not already satisfied expire.
 * Process-wide; applies to calls issued after it returns (not to calls
 * already enqueued).  Returns the previous bound.  No counterpart on the
 * pages, which describe no device-side failure handling. */
int64_t nsp_set_wait_timeout_cycles(int64_t cycles);

/* ------------------------------------------------------------------------
 * Varlen attention forward  ([BASP] Sec. II-A; [HSAP] Sec. 2.1, 2.2.1).
 *
 * For every query row t in [q_start, q_start + q_len) of the packed stream,
 * every query head h and g = h / (Hq / Hkv):
 *   J(t)  = keys of t's document, restricted to positions <= t if causal,
 *           intersected with [kv_start, kv_start + kv_len);
 *   x_j   = scale * <q[t,h], k[j,g]>,   lse[h,t] = ln sum_{j in J(t)} exp(x_j),
 *   out[t,h] = sum_{j in J(t)} exp(x_j - lse[h,t]) v[j,g].
 * A row with empty J(t) gets out = 0 and lse = -inf.
 *
 * Whole-stream attention: q_start = kv_start = 0, q_len = kv_len = T.
 * Ring chunk partial ([HSAP] Sec. 2.2.1 / 3.2): `q` points at the first row
 * of the query shard ([q_len, Hq, d]) and `k`, `v` at the first row of the
 * key shard ([kv_len, Hkv, d]); q_start / kv_start are the shards' global
 * token offsets, used only to compare positions with cu_seqlens.  Request
 * out_dtype = NSP_F32 for partials that will be merged.
 *
 * Arguments: q, k, v device, io_dtype; cu_seqlens device int32 [ndoc+1];
 *   Hq % Hkv == 0; d in {64, 128}; scale > 0 and finite; causal 0/1; out device [q_len, Hq, d] of
 *   out_dtype (NSP_F32 or io_dtype); lse device float32 [Hq, q_len] (may be
 *   NULL when not needed); workspace device, at least
 *   nsp_attn_fwd_workspace_size(...) bytes, contents need no initialisation.
 *
 * Kernel choice: bf16 (d = 128 or 64) runs on the tensor cores (tcgen05,
 * TMEM, TMA), any Hq / Hkv (an even ratio pairs two query heads of a KV
 * group per work item, an odd one, multi-head attention among them, pairs
 * two adjacent query tiles of one head).  float32 I/O runs on the CUDA
 * cores: a correct but much slower path (nsp_path_launches tells which
 * ran).
 * ---------------------------------------------------------------------- */
size_t nsp_attn_fwd_workspace_size(int64_t q_len, int64_t kv_len, int32_t Hq, int32_t Hkv,
                                   int32_t d);

int32_t nsp_attn_fwd(const void* q, const void* k, const void* v, const int32_t* cu_seqlens,
                     int32_t ndoc, int64_t q_start, int64_t q_len, int64_t kv_start,
                     int64_t kv_len, int32_t Hq, int32_t Hkv, int32_t d, float scale,
                     int32_t causal, int32_t io_dtype, void* out, int32_t out_dtype,
                     float* lse, void* workspace, size_t workspace_bytes, nsp_stream_t stream);

/* Host-only argument check of nsp_attn_fwd (no CUDA call): returns the
 * status nsp_attn_fwd would return before enqueuing anything. */
int32_t nsp_attn_fwd_validate(const void* q, const void* k, const void* v,
                              const int32_t* cu_seqlens, int32_t ndoc, int64_t q_start,
                              int64_t q_len, int64_t kv_start, int64_t kv_len, int32_t Hq,
                              int32_t Hkv, int32_t d, int32_t causal, int32_t io_dtype,
                              const void* out, int32_t out_dtype, const void* workspace,
                              size_t workspace_bytes);

/* ------------------------------------------------------------------------
 * Ring partial accumulated in place: the partial block of nsp_attn_fwd
 * merged into a running result inside the attention kernel itself (the
 * running result enters the online softmax as one more weighted term).
 * This is the ring's online accumulation (HSAP Sec. 2.2.1) with the
 * receive-side rescale fused into the attention computation, as HSAP's
 * Limitations section proposes; nsp_lse_merge is the same combine as a
 * separate pass.  Results agree with partials + nsp_lse_merge to well
 * inside the stated tolerances, not bit for bit (P is rounded to bf16
 * against a different reference maximum).
 *
 * For the query rows [q_start, q_start + q_len) against the keys
 * [kv_start, kv_start + kv_len) (global token ids, checked against
 * cu_seqlens exactly as in nsp_attn_fwd) it forms the partial (o_p, lse_p)
 * and updates, per (row t, head h):
 *   lse' = log(exp(lse_acc) + exp(lse_p)),
 *   acc' = exp(lse_acc - lse') acc + exp(lse_p - lse') o_p.
 * Rows that see no key of the range (lse_p = -inf) are left unchanged.
 *   q, k, v, cu_seqlens, ndoc, ranges, Hq, Hkv, d, scale, causal, io_dtype,
 *     workspace: as nsp_attn_fwd (workspace sized by
 *     nsp_attn_fwd_workspace_size(q_len, kv_len, ...)).
 *   acc: device float32 [q_len, Hq, d], read and written.
 *   lse_acc: device float32 [Hq, q_len] (natural log), read and written;
 *     required.
 * Start a ring with lse_acc = -inf and acc = 0 everywhere; after the last
 * block acc holds the attention output and lse_acc its log-sum-exp (a row
 * that never saw a key keeps acc = 0, lse_acc = -inf).  Blocks may come in
 * any order.  Errors: as nsp_attn_fwd (with out_dtype = NSP_F32); a NULL
 * lse_acc is NSP_ERR_INVALID.
 * ---------------------------------------------------------------------- */
int32_t nsp_attn_fwd_accumulate(const void* q, const void* k, const void* v,
                                const int32_t* cu_seqlens, int32_t ndoc, int64_t q_start,
                                int64_t q_len, int64_t kv_start, int64_t kv_len, int32_t Hq,
                                int32_t Hkv, int32_t d, float scale, int32_t causal,
                                int32_t io_dtype, float* acc, float* lse_acc, void* workspace,
                                size_t workspace_bytes, nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Whole-stream forward with q and out in the head-group-major layout an
 * Ulysses-style all-to-all delivers ([HSAP] Sec. 2.2.2: IntraSP moves
 * R^{n x H x d} per rank to R^{N x h x d}, h = H / P; [BASP] Sec. II-C):
 *   q, out: device [P][T][Hq / P][d] (group g holds query heads
 *     g Hq/P .. (g + 1) Hq/P - 1 of every token, i.e.
 *     nsp_seq2head_permute's output);
 *   k, v: device [T][Hkv][d] (the packed layout, not permuted: a group's
 *     query heads find their key/value head as h / (Hq / Hkv));
 *   lse: device float32 [Hq, T] or NULL.
 * The result equals nsp_attn_fwd on the packed layout followed by
 * nsp_seq2head_permute of out, bit for bit (same kernels, same order of
 * arithmetic), without either permutation pass: the kernels address the
 * grouped rows directly (TMA coordinates of a [P T, (Hq/P) d] map).
 * P must divide Hq; P T must fit in int32.  Kernel choice as nsp_attn_fwd
 * (tensor cores for bf16; CUDA cores for float32 I/O).
 * Other arguments and errors: as nsp_attn_fwd
 * with q_start = kv_start = 0, q_len = kv_len = T (workspace sized by
 * nsp_attn_fwd_workspace_size(T, T, ...)); a bad P is NSP_ERR_INVALID.
 * ---------------------------------------------------------------------- */
int32_t nsp_attn_fwd_headgroups(const void* q, const void* k, const void* v,
                                const int32_t* cu_seqlens, int32_t ndoc, int64_t T, int32_t Hq,
                                int32_t Hkv, int32_t d, int32_t P, float scale, int32_t causal,
                                int32_t io_dtype, void* out, int32_t out_dtype, float* lse,
                                void* workspace, size_t workspace_bytes, nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Batched ring blocks: several (query range, key range) blocks of the same
 * packed stream in one call ([HSAP] Sec. 2.2.1, InterSP: each rank's query
 * shard meets every key/value shard; Sec. 3.2, attention blocks A1-A5).  On
 * one GPU holding every shard, a ring step (or a whole ring) is one schedule
 * and one persistent launch instead of one call per block.
 *
 *   q: device [T][Hq][d], k, v: device [T][Hkv][d]: the whole packed stream;
 *      a block's rows are addressed by global token ids.
 *   blocks: host array of nblocks (1..64) descriptors, read during the call:
 *      q_start, q_len: the block's query rows; kv_start, kv_len: its keys;
 *      out: device float32 [q_len][Hq][d]; lse: device float32 [Hq][q_len]
 *      (required when accumulate = 1, else optional).
 *   accumulate = 0: each block's out / lse are written with the partial of
 *      its rows against its keys, exactly as nsp_attn_fwd with out_dtype =
 *      NSP_F32, q / k / v pointing at the block's rows and
 *      q_start / kv_start as given (bit-identical results).
 *   accumulate = 1: each block's partial is merged into its out / lse in
 *      place, as nsp_attn_fwd_accumulate does.
 * The blocks' outputs must not share bytes (NSP_ERR_INVALID otherwise): a
 * ring step's blocks have distinct query shards.  Rows of a block that see
 * no key of it get out = 0, lse = -inf (accumulate: left unchanged).
 * Workspace: at least nsp_attn_fwd_blocks_workspace_size(nblocks, blocks,
 * ...) bytes.  Other arguments, kernel choice and errors as nsp_attn_fwd;
 * ranges outside [0, T) are NSP_ERR_INVALID.
 * ---------------------------------------------------------------------- */
typedef struct {
  int64_t q_start, q_len, kv_start, kv_len;
  void* out;
  float* lse;
} nsp_block_t;

size_t nsp_attn_fwd_blocks_workspace_size(int32_t nblocks, const nsp_block_t* blocks, int32_t Hq,
                                          int32_t Hkv, int32_t d);

int32_t nsp_attn_fwd_blocks(const void* q, const void* k, const void* v,
                            const int32_t* cu_seqlens, int32_t ndoc, int64_t T, int32_t nblocks,
                            const nsp_block_t* blocks, int32_t Hq, int32_t Hkv, int32_t d,
                            float scale, int32_t causal, int32_t io_dtype, int32_t accumulate,
                            void* workspace, size_t workspace_bytes, nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Batched ring-block backward: the gradient contributions of many
 * (query range, key range) blocks of one packed stream, as
 * nsp_attn_bwd_accumulate computes them for each block (full-row
 * probabilities and delta, sums restricted to the block; [HSAP] Sec. 2.2.1
 * ring InterSP, Sec. 3.2 blocks), in one schedule and one launch of each
 * backward kernel: a whole ring's backward as one call.
 *
 *   q, out, dout: device [T][Hq][d]; k, v: device [T][Hkv][d]: the whole
 *     stream, rows addressed by global token ids; lse: device float32 [Hq][T],
 *     the rows' final lse (the forward's over all keys).
 *   ranges: host array of nranges (1..64) {q_start, q_len, kv_start, kv_len},
 *     read during the call; blocks may share rows or overlap.
 *   dq_acc: device float32 [T][Hq][d]; dk_acc, dv_acc: device float32
 *     [T][Hkv][d]: every block's contributions are ADDED at global rows with
 *     float atomics (the caller zeroes them first; the order of the
 *     additions, hence the last bits, may vary between runs).
 * Tensor cores only: bf16 with d = 128 or 64 (float32: NSP_ERR_UNSUPPORTED;
 * use nsp_attn_bwd_accumulate per block).  Every q_start must be a multiple
 * of 4 (NSP_ERR_UNSUPPORTED otherwise).  Workspace: at least
 * nsp_attn_bwd_blocks_workspace_size(T, nranges, ranges, Hq, Hkv, d) bytes;
 * bytes past it (from the next 1024-byte boundary) are a dS cache as for
 * nsp_attn_bwd, used when it holds every visible tile pair of every block
 * (nsp_attn_bwd_blocks_ds_cache_size bytes).
 * Other arguments and errors as nsp_attn_bwd_accumulate.
 * ---------------------------------------------------------------------- */
typedef struct {
  int64_t q_start, q_len, kv_start, kv_len;
} nsp_range_t;

size_t nsp_attn_bwd_blocks_workspace_size(int64_t T, int32_t nranges, const nsp_range_t* ranges,
                                          int32_t Hq, int32_t Hkv, int32_t d);

/* Bytes of dS cache that let nsp_attn_bwd_blocks compute dq from cached
 * tiles: Hq x (visible 128 x 128 tile pairs of every block, tiles aligned to
 * the block's q_start and kv_start) x 32768, from HOST cu_seqlens [ndoc + 1].
 * 0 for a bad argument. */
size_t nsp_attn_bwd_blocks_ds_cache_size(const int32_t* cu_seqlens_host, int32_t ndoc,
                                         int32_t nranges, const nsp_range_t* ranges, int32_t Hq,
                                         int32_t causal);

int32_t nsp_attn_bwd_blocks(const void* q, const void* k, const void* v, const void* out,
                            const void* dout, const float* lse, const int32_t* cu_seqlens,
                            int32_t ndoc, int64_t T, int32_t nranges, const nsp_range_t* ranges,
                            int32_t Hq, int32_t Hkv, int32_t d, float scale, int32_t causal,
                            int32_t io_dtype, float* dq_acc, float* dk_acc, float* dv_acc,
                            void* workspace, size_t workspace_bytes, nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * nsp_attn_fwd without a workspace argument.  No page has a counterpart of
 * this entry point: it exists for callers that cannot allocate device
 * memory where they run attention (code inside a custom allocator or
 * memory-pool callback, plugins whose host framework owns every device
 * allocation, processes that must keep a fixed footprint after start-up).
 *
 * Same arguments, semantics, layouts and results as nsp_attn_fwd, minus
 * workspace / workspace_bytes.  The scheduler scratch lives in a 1 MiB
 * static __device__ array of the library instead, present on every GPU that
 * loads the library until the process exits; nothing is allocated (no
 * cudaMalloc, cudaFree or allocating library call).
 *   Limit: nsp_attn_fwd_workspace_size(q_len, kv_len, ...) must not exceed
 *   1 MiB (about 8.3 million query tokens when q_len = kv_len); larger
 *   problems return NSP_ERR_WORKSPACE before anything is enqueued.
 *   device_status: optional device int32; receives (stream-ordered) the
 *   status word the kernels recorded (NSP_OK, NSP_ERR_INVALID for a bad
 *   cu_seqlens, NSP_ERR_TIMEOUT); NULL to skip.
 *   The first call on each device looks up the array's device address with
 *   cudaGetSymbolAddress (with that device current) and caches it; make that
 *   first call before any stream capture.
 *   Every call shares the one array per device: calls whose kernels overlap
 *   on the GPU (other streams, other host threads) race and must be
 *   serialised by the caller.  Each call rewrites all the scratch it reads.
 * ---------------------------------------------------------------------- */
int32_t nsp_attn_fwd_noalloc(const void* q, const void* k, const void* v,
                             const int32_t* cu_seqlens, int32_t ndoc, int64_t q_start,
                             int64_t q_len, int64_t kv_start, int64_t kv_len, int32_t Hq,
                             int32_t Hkv, int32_t d, float scale, int32_t causal,
                             int32_t io_dtype, void* out, int32_t out_dtype, float* lse,
                             int32_t* device_status, nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Varlen attention backward over the whole stream ([NSP] Sec. 2.3: the
 * backward recomputes attention; only out and lse are kept).
 *
 * Gradients of L = sum(dout * out) for the forward above (q_start =
 * kv_start = 0, q_len = kv_len = T):
 *   delta_t = <dout[t,h], out[t,h]>,  p_tj = exp(x_tj - lse[h,t]),
 *   dS_tj = p_tj (<dout[t,h], v[j,g]> - delta_t),
 *   dq[t,h] = scale sum_j dS_tj k[j,g],
 *   dk[j,g] = scale sum_{h in g} sum_t dS_tj q[t,h],
 *   dv[j,g] = sum_{h in g} sum_t p_tj dout[t,h].
 * out and lse must be the forward's results for the same inputs.
 * dq, dk, dv are written (not accumulated) in io_dtype.  The workspace (at
 * least nsp_attn_bwd_workspace_size bytes for the same T, heads, d and
 * io_dtype) holds the tile schedules, delta and lse * log2(e); its contents
 * need no initialisation.  bf16 (d = 128 or 64) runs on the tensor cores
 * (dq, dk, dv each written once, deterministic); float32 runs on CUDA cores,
 * whose dq is summed with float atomics in a float32 accumulator that the
 * workspace then also holds (last bits may vary).
 *
 * dS cache (tensor-core path only; storing instead of recomputing, the
 * trade NSP Sec. 2.3 weighs for attention's backward).  Workspace bytes past
 * nsp_attn_bwd_workspace_size (from the next 1024-byte boundary on) are a
 * cache for dS = P (dP - delta), the probabilities' gradient: when it holds
 * every visible (128-row query tile, 128-key tile) pair of every query head
 * (nsp_attn_bwd_ds_cache_size bytes), the dK/dV kernel copies each dS tile
 * it builds into the cache and dq is computed from the cached tiles (one
 * 128 x 128 x 128 product per pair instead of recomputing S and dP: three).
 * Otherwise, or with no such bytes, dq recomputes them.  The decision is
 * taken on the device from cu_seqlens; results agree within rounding (dq
 * then uses the dS rounded to bf16 that dk uses; deterministic either way).
 * ---------------------------------------------------------------------- */
size_t nsp_attn_bwd_workspace_size(int64_t T, int32_t Hq, int32_t Hkv, int32_t d,
                                   int32_t io_dtype);

/* Bytes of dS cache that let nsp_attn_bwd / nsp_attn_bwd_headgroups compute
 * dq from cached tiles: Hq x (visible 128 x 128 tile pairs) x 32768, from
 * HOST cu_seqlens [ndoc + 1] (int32, non-decreasing from 0).  Pass at least
 * nsp_attn_bwd_workspace_size rounded up to 1024, plus this, as the
 * workspace.  0 for a bad argument. */
size_t nsp_attn_bwd_ds_cache_size(const int32_t* cu_seqlens_host, int32_t ndoc, int32_t Hq,
                                  int32_t causal);

/* Whether the last backward on this workspace computed dq from the dS cache:
 * *used = 1 or 0, read from the workspace header (a copy to the host on
 * stream, then a synchronisation of stream).  NSP_ERR_INVALID for a NULL
 * argument, NSP_ERR_CUDA if the copy fails. */
int32_t nsp_bwd_ds_cache_used(const void* workspace, int32_t* used, nsp_stream_t stream);

int32_t nsp_attn_bwd(const void* q, const void* k, const void* v, const void* out,
                     const void* dout, const float* lse, const int32_t* cu_seqlens,
                     int32_t ndoc, int64_t T, int32_t Hq, int32_t Hkv, int32_t d, float scale,
                     int32_t causal, int32_t io_dtype, void* dq, void* dk, void* dv,
                     void* workspace, size_t workspace_bytes, nsp_stream_t stream);

int32_t nsp_attn_bwd_validate(const void* q, const void* k, const void* v, const void* out,
                              const void* dout, const float* lse, const int32_t* cu_seqlens,
                              int32_t ndoc, int64_t T, int32_t Hq, int32_t Hkv, int32_t d,
                              int32_t causal, int32_t io_dtype, const void* dq,
                              const void* dk, const void* dv, const void* workspace,
                              size_t workspace_bytes);

/* ------------------------------------------------------------------------
 * Whole-stream backward in the Ulysses receive layout, the backward of
 * nsp_attn_fwd_headgroups ([HSAP] Sec. 2.2.2; [BASP] Sec. II-C):
 *   q, out, dout, dq: device [P][T][Hq / P][d] (head-group-major);
 *   k, v, dk, dv: device [T][Hkv][d] (packed);
 *   lse: device float32 [Hq, T].
 * The gradients equal nsp_attn_bwd on the packed layout with dq moved by
 * nsp_seq2head_permute, bit for bit, without the permutation passes.
 * P must divide Hq; P T must fit in int32.  Other arguments, workspace
 * (nsp_attn_bwd_workspace_size(T, ...)) and errors: as nsp_attn_bwd; a bad P
 * is NSP_ERR_INVALID.
 * ---------------------------------------------------------------------- */
int32_t nsp_attn_bwd_headgroups(const void* q, const void* k, const void* v, const void* out,
                                const void* dout, const float* lse,
                                const int32_t* cu_seqlens, int32_t ndoc, int64_t T, int32_t Hq,
                                int32_t Hkv, int32_t d, int32_t P, float scale, int32_t causal,
                                int32_t io_dtype, void* dq, void* dk, void* dv, void* workspace,
                                size_t workspace_bytes, nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Ring-block backward: one (query range, key range) block's share of the
 * gradients, added into float32 accumulators.  In ring-style InterSP
 * ([HSAP] Sec. 2.2.1) each rank keeps its query shard and the key/value
 * blocks circulate; the backward meets every block once, adds the block's
 * dq into its own accumulator and sends the block's dk/dv contribution on
 * with the block.  Summing the blocks of any chunking of queries and keys
 * gives nsp_attn_bwd's gradients.
 *
 * For the query rows [q_start, q_start + q_len) and the keys
 * [kv_start, kv_start + kv_len) (global token ids, checked against
 * cu_seqlens as in nsp_attn_fwd), with p_tj and delta_t those of the whole
 * row (lse and out are the row's final results over all its keys):
 *   dq_acc[t - q_start, h] += scale sum_{j in block} dS_tj k[j, g],
 *   dk_acc[j - kv_start, g] += scale sum_{t in block, h in g} dS_tj q[t, h],
 *   dv_acc[j - kv_start, g] += sum_{t in block, h in g} p_tj dout[t, h].
 *   q, out, dout: device io_dtype [q_len, Hq, d] (the query shard, its final
 *     attention output and the output gradient).
 *   lse: device float32 [Hq, q_len], the rows' final log-sum-exp.
 *   k, v: device io_dtype [kv_len, Hkv, d] (the key/value block).
 *   dq_acc: device float32 [q_len, Hq, d]; dk_acc, dv_acc: device float32
 *     [kv_len, Hkv, d]; read and written (start them at zero).
 *   workspace: device, at least nsp_attn_bwd_accumulate_workspace_size(q_len,
 *     kv_len, ...) bytes, no initialisation.
 * Pairs no query of the block can see add nothing; a block with no visible
 * pair leaves the accumulators unchanged.  bf16 (d = 128 or 64) runs on the
 * tensor cores (each accumulator element read and written once per call);
 * float32 runs on CUDA cores (dq_acc summed with float atomics).
 * Errors: as nsp_attn_bwd (NULL or misaligned buffers, bad scalars before
 * any launch; a bad cu_seqlens through the workspace status word).
 * ---------------------------------------------------------------------- */
size_t nsp_attn_bwd_accumulate_workspace_size(int64_t q_len, int64_t kv_len, int32_t Hq,
                                              int32_t Hkv, int32_t d, int32_t io_dtype);

int32_t nsp_attn_bwd_accumulate(const void* q, const void* k, const void* v, const void* out,
                                const void* dout, const float* lse,
                                const int32_t* cu_seqlens, int32_t ndoc, int64_t q_start,
                                int64_t q_len, int64_t kv_start, int64_t kv_len, int32_t Hq,
                                int32_t Hkv, int32_t d, float scale, int32_t causal,
                                int32_t io_dtype, float* dq_acc, float* dk_acc, float* dv_acc,
                                void* workspace, size_t workspace_bytes, nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Log-sum-exp merge of n partials of the same T query rows over disjoint
 * key sets ([HSAP] Sec. 2.2.1 online accumulation; Limitations "rescale"):
 *   m = max_i lse_i;  m = -inf -> out = 0, lse = -inf;  otherwise
 *   lse = m + ln sum_i exp(lse_i - m),  out = sum_i exp(lse_i - lse) out_i.
 *
 * outs, lses: HOST arrays of n DEVICE pointers (1 <= n <= 64); outs[i] is
 *   float32 [T, H, d], lses[i] float32 [H, T].  out: device [T, H, d] of
 *   out_dtype (NSP_F32 or NSP_BF16, round-to-nearest-even); lse: device
 *   float32 [H, T] (may be NULL).  out and lse must not overlap any input.
 * ---------------------------------------------------------------------- */
int32_t nsp_lse_merge(const float* const* outs, const float* const* lses, int32_t n,
                      int64_t T, int32_t H, int32_t d, void* out, int32_t out_dtype,
                      float* lse, nsp_stream_t stream);

int32_t nsp_lse_merge_validate(const float* const* outs, const float* const* lses, int32_t n,
                               int64_t T, int32_t H, int32_t d, const void* out,
                               int32_t out_dtype, const float* lse);

/* ------------------------------------------------------------------------
 * Several independent LSE merges in one launch: segment g combines its
 * counts[g] partials into out[g] / lse[g], exactly as nsp_lse_merge would
 * (same arithmetic, same results).  For a ring on one GPU this merges every
 * query shard at once ([HSAP] Sec. 2.2.1), so the launch ramps up and
 * drains once instead of once per shard.
 *   nseg: 1 .. 16 segments, each of T tokens, H heads, head dim d.
 *   counts: HOST int32 [nseg], each >= 1, sum <= 64.
 *   outs, lses: HOST arrays of sum(counts) device pointers, segment after
 *     segment (layouts as in nsp_lse_merge).
 *   out: HOST array of nseg device pointers [T, H, d] (out_dtype);
 *   lse: HOST array of nseg device pointers [H, T] (entries may be NULL),
 *     or NULL.
 * Errors: as nsp_lse_merge, per segment; bad nseg / counts are
 * NSP_ERR_INVALID.
 * ---------------------------------------------------------------------- */
int32_t nsp_lse_merge_batch(int32_t nseg, const int32_t* counts, const float* const* outs,
                            const float* const* lses, int64_t T, int32_t H, int32_t d,
                            void* const* out, int32_t out_dtype, float* const* lse,
                            nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Ulysses seq -> head permutation ([HSAP] Sec. 2.2.2: blocks in
 * R^{n x H x d} per group become R^{N x h x d}, h = H / P; [BASP] Sec. II-C).
 * With the P sequence shards stacked on this device as in = [T, H, d]:
 *   inverse = 0:  out[g][t][j][:] = in[t][g*h + j][:]    out = [P, T, h, d]
 *   inverse = 1:  out[t][g*h + j][:] = in[g][t][j][:]    (head -> seq)
 * Elements are elem_bytes wide (1, 2, 4 or 8) and copied bit-exactly.
 * H % P == 0; in and out must not overlap.
 * ---------------------------------------------------------------------- */
int32_t nsp_seq2head_permute(const void* in, void* out, int64_t T, int32_t H, int32_t d,
                             int32_t P, int32_t elem_bytes, int32_t inverse,
                             nsp_stream_t stream);

int32_t nsp_seq2head_permute_validate(const void* in, const void* out, int64_t T, int32_t H,
                                      int32_t d, int32_t P, int32_t elem_bytes);

/* ------------------------------------------------------------------------
 * Batch-aware subgroup all-to-all layout ([BASP] Sec. IV, "Batch-aware
 * group formation", "Batch Aware Sequence Partitioning" (Alg. 2),
 * "Subgroup all-to-all"): a micro-batch of B sequences of L tokens on
 * N = B K ranks, where each sequence is sharded over its own group of K ranks
 * and each group runs an independent K-way all-to-all.  With the batch
 * stacked on one device, the receive side of all B groups:
 *   inverse = 0:  out[b][g][t][j][:] = in[b L + t][g H/K + j][:]
 *   inverse = 1:  in[b L + t][g H/K + j][:] = out[b][g][t][j][:] (roles of
 *                 the buffers swapped: `in` is [B][K][L][H/K][d])
 *   in:  device [B L][H][d] elements of elem_bytes (1, 2, 4 or 8 bytes);
 *   out: device [B][K][L][H/K][d].
 * Each group's block is the nsp_seq2head_permute of its own sequence with
 * P = K (B = 1 is exactly that call); no data crosses sequences.  Bit-exact
 * data movement, one launch for all B groups.  Errors as
 * nsp_seq2head_permute on the whole [B L, H, d] batch (K must divide H;
 * in, out 16-byte aligned, not overlapping); B < 1 or L < 0 is
 * NSP_ERR_INVALID.
 * ---------------------------------------------------------------------- */
int32_t nsp_seq2head_permute_groups(const void* in, void* out, int32_t B, int64_t L, int32_t H,
                                    int32_t d, int32_t K, int32_t elem_bytes, int32_t inverse,
                                    nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * The operators between the projections of a differential attention layer
 * on a packed stream.  No page has a counterpart of them; they follow the
 * conventions above (caller-owned buffers, caller stream, nothing allocated,
 * host errors before anything is enqueued).
 *
 * Rotary positions
 * ----------------
 * Every head of every token is rotated by angles that grow with the token's
 * position inside its own document.  With rot rotated columns of a head's d,
 * pair i < rot / 2 is columns (i, i + rot / 2) (interleaved = 0) or
 * (2 i, 2 i + 1) (interleaved = 1), and for x_a, x_b of the pair
 *   angle = position * freqs[i],
 *   y_a = mscale (x_a cos - x_b sin),  y_b = mscale (x_a sin + x_b cos);
 * columns [rot, d) are copied.  inverse = 1 rotates by -angle (times mscale
 * as well): the transpose, which takes gradients of y to gradients of x.
 *
 *   tensors: HOST array of n (1..4) descriptors, read during the call: in and
 *     out device [len, heads, d] of io_dtype, tokens in_stride / out_stride
 *     elements apart (0: heads * d), so that in or out can be columns of a
 *     fused projection's tensor.  in and out may be the same buffer with the
 *     same stride (in place); any other overlap of an output with another
 *     array of the call is NSP_ERR_INVALID.  groups = P > 1: the rotated side (out,
 *     or in when inverse = 1) is in the head-group-major layout
 *     [P][len][heads / P][d] of nsp_attn_fwd_headgroups, packed.
 *   positions: device int32 [len], or NULL: row r is then global token
 *     start + r of the stream, its position the distance from its document's
 *     start in cu_seqlens (device int32 [ndoc + 1]; unused, may be NULL, when
 *     positions is given).  Rows at or past cu_seqlens[ndoc] are not written.
 *     The contents of cu_seqlens are not checked here (there is no status
 *     word); they never lead outside the buffers.
 *   freqs: device float64 [rot / 2], finite, radians per position.  The angle's whole
 *     turns are taken off in integer arithmetic, at any position; what is left is
 *     off by 2^-52 of the whole angle (the float64 frequency as a fraction of a
 *     turn) and by its own rounding to float32, 2^-26 turns at most.
 *   d in 2..1024; rot even, 2..d; sums and products in float32.  Pointers
 *     need their element's alignment; 16-byte aligned ones with strides, d
 *     and rot (halves: rot / 2) of whole 16-byte pieces are several times
 *     faster.
 * ---------------------------------------------------------------------- */
typedef struct {
  const void* in;
  void* out;
  int64_t in_stride, out_stride;
  int32_t heads, groups;
} nsp_rope_tensor_t;

int32_t nsp_rope(const nsp_rope_tensor_t* tensors, int32_t n, const int32_t* cu_seqlens,
                 int32_t ndoc, const int32_t* positions, int64_t start, int64_t len, int32_t d,
                 int32_t rot, const double* freqs, int32_t interleaved, float mscale,
                 int32_t inverse, int32_t io_dtype, nsp_stream_t stream);

/* Frequencies for nsp_rope, written to HOST freqs_host [rot / 2]:
 *   f_i = base^(-2 i / rot), and for contexts longer than the trained one
 *   NSP_ROPE_LINEAR: f_i / factor;
 *   NSP_ROPE_BASE:   base * factor^(rot / (rot - 2)) in place of base (the
 *                    slowest pair slows by factor, the fastest stays);
 *   NSP_ROPE_PARTS:  k f_i + (1 - k) f_i / factor, where pair i turns
 *                    n_i = orig_len f_i / 2 pi times over the trained context
 *                    and k = clamp((n_i - low) / (high - low), 0, 1).
 * factor >= 1; unused arguments of a kind are ignored.  Host only. */
typedef enum {
  NSP_ROPE_PLAIN = 0, NSP_ROPE_LINEAR = 1, NSP_ROPE_BASE = 2, NSP_ROPE_PARTS = 3
} nsp_rope_scaling;

int32_t nsp_rope_freqs(int32_t rot, double base, int32_t scaling, double factor, double low,
                       double high, double orig_len, double* freqs_host);

/* ------------------------------------------------------------------------
 * Weight of the second map, from four learned vectors of each head:
 *   lambda[h] = exp(<q1, k1>) - exp(<q2, k2>) + init.
 *   q1, k1, q2, k2: device [n][dl] of io_dtype, n = heads, or n = 1: one set
 *   that every head shares.  lambda: device [heads] of io_dtype.
 * The backward writes dq1 = g e1 k1, dk1 = g e1 q1, dq2 = -g e2 k2,
 * dk2 = -g e2 q2 ([n][dl], io_dtype), e1, e2 the two exponentials and g =
 * dlambda[h] (io_dtype), or its sum over the heads when n = 1.  Sums in
 * float32.  Pointers need their element's alignment.  A lambda that overlaps a
 * vector, or a gradient that overlaps an input or another gradient, is
 * NSP_ERR_INVALID.
 * ---------------------------------------------------------------------- */
int32_t nsp_diff_lambda_fwd(const void* q1, const void* k1, const void* q2, const void* k2,
                            int32_t n, int32_t dl, int32_t heads, float init, int32_t io_dtype,
                            void* lambda, nsp_stream_t stream);

int32_t nsp_diff_lambda_bwd(const void* dlambda, const void* q1, const void* k1, const void* q2,
                            const void* k2, int32_t n, int32_t dl, int32_t heads,
                            int32_t io_dtype, void* dq1, void* dk1, void* dq2, void* dk2,
                            nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Differential attention of a whole packed stream, document-masked as
 * nsp_attn_fwd with q_start = kv_start = 0, q_len = kv_len = T.  Columns
 * [0, d/2) of a head's q and k are its first map, [d/2, d) its second:
 *   x^m_j = scale <q^m[t,h], k^m[j,g]>,  lse[h,m,t] = ln sum_j exp(x^m_j),
 *   o^m[t,h] = sum_j exp(x^m_j - lse[h,m,t]) v[j,g],
 *   out = o^1 - lambda o^2,                       g = h / (Hq / Hkv).
 *   q, out, out2: device [T, Hq, d]; k, v: device [T, Hkv, d]; d in {64, 128}.
 *   lambda: device [Hq][n_lambda] of io_dtype; n_lambda = 1 (one of each
 *     head) or T (one of each head and token).
 *   out2: o^2, or NULL when no backward follows.  lse: device float32
 *     [Hq][2][T], or NULL likewise.  out and out2 are of io_dtype.
 * All pointers 16-byte aligned, bf16 out and out2 32-byte aligned.  Outputs
 * must not overlap any input or one another (not checked).  Errors and the
 * status word as nsp_attn_fwd; a cu_seqlens that reaches past T is cut there.
 * v has to be finite in every row, those of padding documents too: masked
 * keys have probability zero, which times a non-finite value is NaN, so that
 * such a value makes NaN of rows that do not see it, in its own document and in
 * those around it that share its tiles of 128 rows or keys, or a neighbour's.
 * A non-finite q or k reaches the rows that have or see it and no others.
 * ---------------------------------------------------------------------- */
size_t nsp_diff_attn_fwd_workspace_size(int64_t T);

int32_t nsp_diff_attn_fwd(const void* q, const void* k, const void* v, const void* lambda,
                          int64_t n_lambda, const int32_t* cu_seqlens, int32_t ndoc, int64_t T,
                          int32_t Hq, int32_t Hkv, int32_t d, float scale, int32_t causal,
                          int32_t io_dtype, void* out, void* out2, float* lse, void* workspace,
                          size_t workspace_bytes, nsp_stream_t stream);

/* Its backward.  out, out2 and lse as the forward wrote them; dout and dq
 * device [T, Hq, d], dk and dv [T, Hkv, d], dlambda [Hq][n_lambda], all of
 * io_dtype.  With p^m the probabilities recomputed from lse,
 * delta^m = <dout, o^m> and dp_j = <dout, v_j>:
 *   ds^1 = p^1 (dp - delta^1),  ds^2 = -lambda p^2 (dp - delta^2),
 *   dq^m = scale sum_j ds^m_j k^m_j,  dk^m = scale sum_t ds^m_t q^m_t,
 *   dv = sum_t (p^1_t - lambda p^2_t) dout_t  (dk, dv over the group's heads),
 *   dlambda = -sum_j p^2_j dp_j of each token, or its sum over the tokens.
 * bf16: delta^m are sums over the rounded out and out2, dlambda is summed in
 * float32 from p and dp before they are rounded.  Every output is written whole,
 * and sums run in one fixed order: results are the same bits on every run.
 * q, k, v and dout have to be finite in every row, for the forward's reason. */
size_t nsp_diff_attn_bwd_workspace_size(int64_t T, int32_t Hq, int32_t Hkv, int32_t d,
                                        int32_t io_dtype);

int32_t nsp_diff_attn_bwd(const void* q, const void* k, const void* v, const void* lambda,
                          int64_t n_lambda, const void* out, const void* out2, const void* dout,
                          const float* lse, const int32_t* cu_seqlens, int32_t ndoc, int64_t T,
                          int32_t Hq, int32_t Hkv, int32_t d, float scale, int32_t causal,
                          int32_t io_dtype, void* dq, void* dk, void* dv, void* dlambda,
                          void* workspace, size_t workspace_bytes, nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Root-mean-square norm of every head's row (the difference of two maps is
 * normed head by head before the output projection; q and k before the
 * rotation), scaled and optionally gated:
 *   y = scale * weight * x / sqrt(mean(x^2) + eps) [* sigmoid(gate)].
 *   x: device [tokens, heads, d], tokens x_stride elements apart (0:
 *     heads * d); weight: device [d] or NULL (ones); gate: device
 *     [tokens, heads, d] or NULL; y: device [tokens, heads, d]; all of
 *     io_dtype, statistics and products in float32.
 *   d <= 512 with whole 16-byte pieces (bf16: a multiple of 8, float32: of 4),
 *     other d are NSP_ERR_UNSUPPORTED; eps > 0.  Pointers 16-byte aligned,
 *     x_stride a multiple of 16 bytes.  y may be gate's or a packed x's
 *     buffer.
 * The backward writes dx (packed), dgate (required with a gate) and, unless
 * NULL, dweight [d]; dweight needs nsp_head_norm_bwd_workspace_size bytes of
 * workspace and is summed in one fixed order.  dx may be dy's buffer, dgate
 * gate's.  Any other overlap of an output (or the workspace) with another
 * array is NSP_ERR_INVALID.
 * ---------------------------------------------------------------------- */
int32_t nsp_head_norm_fwd(const void* x, int64_t x_stride, const void* weight, const void* gate,
                          int64_t tokens, int32_t heads, int32_t d, float eps, float scale,
                          int32_t io_dtype, void* y, nsp_stream_t stream);

size_t nsp_head_norm_bwd_workspace_size(int64_t tokens, int32_t heads, int32_t d);

int32_t nsp_head_norm_bwd(const void* x, int64_t x_stride, const void* weight, const void* gate,
                          const void* dy, int64_t tokens, int32_t heads, int32_t d, float eps,
                          float scale, int32_t io_dtype, void* dx, void* dgate, void* dweight,
                          void* workspace, size_t workspace_bytes, nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * The operators of a packed post-training step next to attention.  No page has
 * a counterpart of them; they follow the conventions above.
 *
 * Norm of query and key heads with the rotation in the same pass
 * --------------------------------------------------------------
 * Every head's row is normed by its root mean square, weighted, and rotated by
 * its token's position as nsp_rope does:
 *   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = rotated(weight * n).
 *   tensors: HOST array of n (1..4) descriptors, read during the call: x device
 *     [len, heads, d] and y of io_dtype, tokens x_stride / y_stride elements
 *     apart (0: heads * d), so that x can be columns of a fused projection;
 *     weight device [d] of io_dtype or NULL (ones).  groups = P > 1: y is in the
 *     head-group-major layout [P][len][heads / P][d], packed.  y may take x's
 *     place (the same buffer and stride, groups = 1).
 *   cu_seqlens, ndoc, positions, start, len, rot, freqs, interleaved, mscale:
 *     as nsp_rope, rows at or past cu_seqlens[ndoc] not written among them.
 *   d in 2..512, eps > 0; statistics, sums and products in float32.  Pointers
 *     need their element's alignment; 16-byte aligned ones with strides, d
 *     and rot (halves: rot / 2) of whole 16-byte pieces are several times
 *     faster.
 * A non-finite element makes its own row's results non-finite or zero, in any
 * column, and in the backward dweight; no other row's.
 * The backward reads x and the gradient dy of y (y's stride and groups) and
 * writes, with z = dy rotated back and u = weight * z,
 *   dx = r (u - n mean(u n)), tokens dx_stride elements apart, and, unless
 *   NULL, dweight [d] = sum over rows of n z.
 * dx may take x's place, or with groups = 1 dy's (the same buffer and stride).
 * The workspace (nsp_qk_norm_rope_bwd_workspace_size bytes, which reads only
 * the descriptors' heads; required) holds dweight's partial sums, added in one
 * fixed order.  Rows at or past cu_seqlens[ndoc] are not written and add
 * nothing.  Any other overlap of an output or the workspace with another array
 * of the call is NSP_ERR_INVALID.
 * ---------------------------------------------------------------------- */
typedef struct {
  const void* x;
  const void* weight;
  void* y;              /* forward */
  const void* dy;       /* backward */
  void* dx;
  void* dweight;
  int64_t x_stride, y_stride, dx_stride;
  int32_t heads, groups;
} nsp_qk_tensor_t;

int32_t nsp_qk_norm_rope_fwd(const nsp_qk_tensor_t* tensors, int32_t n, const int32_t* cu_seqlens,
                             int32_t ndoc, const int32_t* positions, int64_t start, int64_t len,
                             int32_t d, int32_t rot, const double* freqs, int32_t interleaved,
                             float mscale, float eps, int32_t io_dtype, nsp_stream_t stream);

size_t nsp_qk_norm_rope_bwd_workspace_size(const nsp_qk_tensor_t* tensors, int32_t n, int64_t len,
                                           int32_t d);

int32_t nsp_qk_norm_rope_bwd(const nsp_qk_tensor_t* tensors, int32_t n, const int32_t* cu_seqlens,
                             int32_t ndoc, const int32_t* positions, int64_t start, int64_t len,
                             int32_t d, int32_t rot, const double* freqs, int32_t interleaved,
                             float mscale, float eps, int32_t io_dtype, void* workspace,
                             size_t workspace_bytes, nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Log-probability of a given token of every row of logits:
 *   x_j = scale * logits[t][j],  lse[t] = ln sum_j exp(x_j),
 *   logp[t] = x_{targets[t]} - lse[t].
 *   logits: device [rows][vocab] of io_dtype, rows row_stride elements apart (0:
 *     vocab); targets: device int32 [rows]; a negative target is none: the row is
 *     not read, whatever it holds, its logp and lse are 0.  A target at or past
 *     vocab makes its logp NaN.  scale in [1e-30, 1e30]: the inverse of a sampling temperature.
 *   logp, lse: device float32 [rows]; lse may be NULL.
 *   workspace: nsp_token_logp_workspace_size(rows) bytes.
 * Logits of minus infinity have probability zero (a row of nothing else, a NaN or
 * a plus infinity in a row give NaN).  Statistics in float32.
 * The backward writes
 *   dlogits[t][j] = scale * dlogp[t] * ([j = targets[t]] - exp(x_j - lse[t])),
 * rows out_stride elements apart (0: vocab), zeros for a row without a target (whose
 * dlogp is not used) and NaN for a target at or past vocab.  lse as the forward
 * wrote it, dlogp device float32 [rows].  dlogits may be the logits' own buffer
 * with the same stride.  Columns past vocab of a strided tensor are neither read
 * nor written.
 * vocab <= 2^20.  Pointers need their element's alignment; logits and dlogits at
 * the same distance from a 16-byte border, row by row, are several times faster.
 * Any other overlap of an output with another array is NSP_ERR_INVALID.
 * ---------------------------------------------------------------------- */
size_t nsp_token_logp_workspace_size(int64_t rows);

int32_t nsp_token_logp_fwd(const void* logits, int64_t row_stride, const int32_t* targets, int64_t rows,
                           int32_t vocab, double scale, int32_t io_dtype, float* logp, float* lse,
                           void* workspace, size_t workspace_bytes, nsp_stream_t stream);

int32_t nsp_token_logp_bwd(const void* logits, int64_t row_stride, const int32_t* targets,
                           const float* lse, const float* dlogp, int64_t rows, int32_t vocab,
                           double scale, int32_t io_dtype, void* dlogits, int64_t out_stride,
                           nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Clipped policy loss of a packed stream, with its gradient.  A row is scored if
 * it has a target (targets[t] >= 0) and lies in a document.  With rho =
 * exp(logp - old_logp), A the advantage and z = ref_logp - logp:
 *   surrogate = -min(rho A, min(max(rho, 1 - clip_low), 1 + clip_high) A),
 *   kl = exp(z) - z - 1 (0 without ref_logp),
 *   loss = sum over scored rows of w (surrogate + kl_coef kl),
 * w = 1 / N (mean = NSP_MEAN_TOKENS, N scored rows) or 1 / (D n) (NSP_MEAN_DOCUMENTS:
 * n scored rows of the row's document, D documents that have one); total > 0
 * takes the place of N or D (the whole batch's, where a step has several calls).
 *   logp: device float32 [rows]; old_logp, ref_logp likewise (ref_logp may be NULL
 *     if kl_coef = 0); advantages: device float32 [ndoc], or [rows] (per_token = 1).
 *     What rows without a score hold is not used.
 *   stats: device float32 [4]: loss, and the weighted sums of surrogate, kl and
 *     clipped (1 where the clip decides: A > 0 and rho > 1 + clip_high, or A < 0
 *     and rho < 1 - clip_low; such a row's surrogate has no gradient).
 *   dlogp: device float32 [rows], the loss's gradient; 0 for rows not scored.
 * nsp_policy_loss_logits does nsp_token_logp_fwd, this and nsp_token_logp_bwd in
 * one pass over the logits: logp (may be NULL; 0 for rows not scored) and dlogits
 * as they write them, dlogits the loss's gradient, zeros for rows not scored; it
 * may be the logits' buffer with the same stride.
 *   rows: of all arrays; a cu_seqlens that reaches past it is cut there.  A bad
 *   cu_seqlens sets the status word, and nothing else is written.
 *   workspace: nsp_policy_loss_workspace_size(rows, ndoc, logits = 0 / 1) bytes.
 *   0 <= clip_low <= 1, clip_high >= 0.  Sums in one fixed order, to more than
 *   float32's precision.  An output or workspace that overlaps another array (but
 *   dlogits as said) is NSP_ERR_INVALID.
 * ---------------------------------------------------------------------- */
typedef enum { NSP_MEAN_TOKENS = 0, NSP_MEAN_DOCUMENTS = 1 } nsp_mean;

typedef struct {
  const float* old_logp;
  const float* ref_logp;
  const float* advantages;
  int32_t per_token;
  int32_t mean;
  float clip_low, clip_high, kl_coef, total;
} nsp_policy_t;

size_t nsp_policy_loss_workspace_size(int64_t rows, int32_t ndoc, int32_t logits);

int32_t nsp_policy_loss(const float* logp, const int32_t* targets, const int32_t* cu_seqlens,
                        int32_t ndoc, int64_t rows, const nsp_policy_t* policy, float* stats,
                        float* dlogp, void* workspace, size_t workspace_bytes, nsp_stream_t stream);

int32_t nsp_policy_loss_logits(const void* logits, int64_t row_stride, const int32_t* targets,
                               const int32_t* cu_seqlens, int32_t ndoc, int64_t rows, int32_t vocab,
                               double scale, int32_t io_dtype, const nsp_policy_t* policy, float* stats,
                               float* logp, void* dlogits, int64_t out_stride, void* workspace,
                               size_t workspace_bytes, nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Preference loss over pairs of documents, with its gradient: documents 2 i and
 * 2 i + 1 are the chosen and the rejected answer of pair i.
 *   score_b = sum over document b's scored rows of (logp - ref_logp), divided by
 *   their number if average = 1 (0 without any),
 *   rewards[b] = beta score_b,  h = rewards[2 i] - rewards[2 i + 1] - margin,
 *   loss = mean over pairs of
 *     NSP_PREFERENCE_SIGMOID: -(1 - smoothing) ln sigma(h) - smoothing ln sigma(-h),
 *     NSP_PREFERENCE_HINGE:   max(0, 1 - h),
 *     NSP_PREFERENCE_SQUARE:  (h / beta - 1 / (2 beta))^2.
 *   logp, ref_logp (NULL: zeros): device float32 [rows]; targets: device int32
 *   [rows], only their sign is used; ndoc even.
 *   stats: device float32 [2]: the loss, and the share of pairs whose chosen
 *   answer's reward is the larger; rewards: device float32 [ndoc]; dlogp: device
 *   float32 [rows], 0 for rows not scored.
 * Rows, cu_seqlens, status word, sums and overlaps as nsp_policy_loss (after a bad
 * cu_seqlens the outputs are unspecified).
 * ---------------------------------------------------------------------- */
typedef enum {
  NSP_PREFERENCE_SIGMOID = 0, NSP_PREFERENCE_HINGE = 1, NSP_PREFERENCE_SQUARE = 2
} nsp_preference;

size_t nsp_preference_loss_workspace_size(int32_t ndoc);

int32_t nsp_preference_loss(const float* logp, const float* ref_logp, const int32_t* targets,
                            const int32_t* cu_seqlens, int32_t ndoc, int64_t rows, int32_t kind,
                            float beta, float smoothing, float margin, int32_t average, float* stats,
                            float* rewards, float* dlogp, void* workspace, size_t workspace_bytes,
                            nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Norm of many gradients taken together, and their clipping:
 *   norm = |unscale| (sum of all g^2)^(1/2) (NSP_NORM_2) or |unscale| max |g|
 *   (NSP_NORM_INF),
 *   out = g * unscale * min(1, max_norm / (norm + eps)).
 *   grads, out, counts, dtypes, out_dtypes: HOST arrays of n (1..16384) device
 *     pointers, element counts (0 to 2^40) and nsp_dtypes, read during the call.
 *     Gradients of both types may be mixed, and out may be of the other type
 *     than its gradient; out[i] may be grads[i] (same type: in place).
 *   unscale: what the gradients have to be multiplied by (1 / the number of
 *     micro-batches summed in them, or 1 / a loss scale).
 *   norm: device float32 [1].  The norm of no elements is 0.
 * One multiplication in float32 and one rounding to out's type; in place, where the
 * factor is 1, nothing is read or written again.  The factor is decided on the
 * device.  A NaN anywhere makes the norm and every output NaN; an infinite norm
 * makes finite gradients 0 and infinite ones NaN.  Squares are float32: a
 * gradient past 1.8e19 makes an infinite norm, one below 1e-23 adds nothing.
 * Sums in one fixed order.  max_norm >= 0, eps > 0.  Pointers need their element's
 * alignment; grads[i] and out[i] at the same number of elements from a 16-byte
 * border are faster.  An output, the norm or the workspace
 * (nsp_grad_norm_workspace_size) that overlaps another array of the call is
 * NSP_ERR_INVALID (the same gradient twice among them, where it is written).
 * ---------------------------------------------------------------------- */
typedef enum { NSP_NORM_2 = 0, NSP_NORM_INF = 1 } nsp_norm;

size_t nsp_grad_norm_workspace_size(const int64_t* counts, int32_t n);

int32_t nsp_grad_norm(const void* const* grads, const int64_t* counts, const int32_t* dtypes, int32_t n,
                      int32_t kind, float unscale, float* norm, void* workspace, size_t workspace_bytes,
                      nsp_stream_t stream);

int32_t nsp_grad_clip(const void* const* grads, void* const* out, const int64_t* counts,
                      const int32_t* dtypes, const int32_t* out_dtypes, int32_t n, int32_t kind,
                      float unscale, float max_norm, float eps, float* norm, void* workspace,
                      size_t workspace_bytes, nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Status word of the last call that used `workspace`.  Synchronises `stream`
 * first (the only synchronising call).  Returns NSP_OK, the recorded device
 * error (NSP_ERR_INVALID for bad cu_seqlens, NSP_ERR_TIMEOUT), or
 * NSP_ERR_CUDA if the synchronisation itself failed.
 * ---------------------------------------------------------------------- */
int32_t nsp_status_query(const void* workspace, nsp_stream_t stream);

/* ------------------------------------------------------------------------
 * Useful work of a whole-stream causal/bidirectional attention, from a HOST
 * copy of cu_seqlens (NSP's cost model takes "attention FLOPs" of the routed
 * inputs, [NSP] Sec. 4.1): pairs = allowed (query, key) pairs per query head.
 * Writes *pairs; returns NSP_ERR_INVALID for a malformed cu_seqlens.
 * ---------------------------------------------------------------------- */
int32_t nsp_attn_pairs(const int32_t* cu_seqlens_host, int32_t ndoc, int32_t causal,
                       double* pairs);

/* ------------------------------------------------------------------------
 * Cost of one attention call, from a HOST copy of cu_seqlens: the hook a
 * planner that balances attention work over ranks or pipelines needs (NSP
 * Sec. 4.1: the backend reports the attention FLOPs of the inputs routed to
 * it; HSAP Sec. 3.2 balances ranks by attention block counts).  For the
 * query rows [q_start, q_start + q_len) against the keys
 * [kv_start, kv_start + kv_len) (the whole stream: 0, T, 0, T):
 *   pairs      allowed (query, key) pairs per query head;
 *   fwd_flop   4 d Hq pairs (Q K^T and P V);
 *   bwd_flop   10 d Hq pairs (the recomputed Q K^T, dOut V^T, P^T dOut,
 *              dS^T Q, dS K);
 *   tiles      (128-row query tile, 128-key tile) pairs holding at least one
 *              allowed pair: the tiles the kernels schedule, per query head
 *              (executed tensor-core work is 4 d Hq 128^2 tiles forward);
 *   fwd_bytes  compulsory HBM bytes of nsp_attn_fwd: q, k, v read, out
 *              written in io_dtype, lse written (float32);
 *   bwd_bytes  compulsory HBM bytes of nsp_attn_bwd: q, k, v, out, dout and
 *              lse read, dq, dk, dv written.
 * Returns NSP_ERR_INVALID for a malformed cu_seqlens, ranges outside it or
 * bad head counts; *cost is written only on NSP_OK.  No device work.
 * ---------------------------------------------------------------------- */
typedef struct {
  double pairs, fwd_flop, bwd_flop, tiles, fwd_bytes, bwd_bytes;
} nsp_attn_cost_t;

int32_t nsp_attn_cost(const int32_t* cu_seqlens_host, int32_t ndoc, int64_t q_start,
                      int64_t q_len, int64_t kv_start, int64_t kv_len, int32_t Hq, int32_t Hkv,
                      int32_t d, int32_t causal, int32_t io_dtype, nsp_attn_cost_t* cost);

#ifdef __cplusplus
}
#endif

#endif /* NSP_H_ */
