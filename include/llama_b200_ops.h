/*
 * llama_b200_ops.h — single-kernel entry points of libllama_b200.so.
 *
 * Each call runs one of the kernels the model path uses, on caller device
 * buffers, so that a kernel can be checked against the CPU oracle on its own
 * and timed in isolation, or an operator of a serving step over a paged KV
 * cache (llama_paged_*).  Conventions (device pointers, void* stream,
 * LLAMA_OK / LLAMA_ERR_* return codes, llama_last_error) are those of
 * llama_b200.h.
 */
#ifndef LLAMA_B200_OPS_H
#define LLAMA_B200_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "llama_b200.h"

#ifdef __cplusplus
extern "C" {
#endif

/* RMSNorm of M rows: out[m,:] = x[m,:] / sqrt(mean(x[m,:]^2) + eps) * w
 * (Admin Guide §8.4, RMSNorm), fp32 arithmetic.
 *   x fp32 [M, dim]; w fp32 [dim]; out [M, dim] in out_dtype (LLAMA_F32,
 *   LLAMA_BF16 or LLAMA_F16, rounded once).  dim % 4 == 0. */
LLAMA_API int llama_op_rmsnorm(const float* x, const float* w, int M, int dim, float eps,
                     void* out, int out_dtype, void* stream);

/* Dense projection out[m,n] = sum_k A[m,k] * W[n,k]  (nn.Linear, y = x W^T).
 *   A [M, K] and W [N, K] in `dtype` (LLAMA_F32: SIMT fp32 FMA, no TF32;
 *   LLAMA_BF16 or LLAMA_F16: tcgen05 tensor cores, both operands of that
 *   type, fp32 accumulation in TMEM); out fp32 [M, N] (row-major,
 *   overwritten).  K % 8 == 0 for the 16-bit types; any other dtype code is
 *   LLAMA_ERR_INVALID_ARG.
 * The 16-bit kernels are the ones the model path uses: for M <= 64 the
 * persistent weight-streaming kernel (the weight is the 128-row MMA operand,
 * K split across CTAs), else the persistent 128 x 256-tile kernel.
 *   workspace  device scratch of llama_op_linear_workspace_bytes(), 256-byte
 *              aligned, zero-filled before its first use (the kernels leave
 *              their counters at zero again).  Required for the 16-bit
 *              types with M <= 64.  Optional for M > 64: with it the last
 *              wave of tiles is split along K over all SMs (stream-K), with
 *              NULL every tile runs whole.  A non-NULL workspace that is too small or
 *              misaligned is rejected (LLAMA_ERR_INVALID_ARG).  Calls sharing
 *              a workspace must not overlap on the device. */
LLAMA_API size_t llama_op_linear_workspace_bytes(void);
LLAMA_API int llama_op_linear(const void* A, const void* W, int M, int N, int K, int dtype,
                    float* out, void* workspace, size_t workspace_bytes, void* stream);

/* Allocation-free decode-shaped projection.  The source pages have no
 * counterpart: it exists for callers that cannot allocate device memory --
 * code running where cudaMalloc is not allowed (inside an allocator or memory
 * pool owned by someone else, a locked-down process, a plug-in that must not
 * touch the device heap) and so cannot provide the scratch workspace that
 * llama_op_linear needs.
 * Computes exactly what llama_op_linear computes for dtype LLAMA_BF16:
 *   out[m,n] = sum_k A[m,k] * W[n,k], A bf16 [M, K], W bf16 [N, K], out fp32
 *   [M, N] (device pointers owned by the caller), with the same persistent
 *   weight-streaming kernel, but its split-tile scratch is a fixed array in
 *   the library's device image (4 MiB + 16 KiB, held on every GPU that loads
 *   the library until the process exits).  Nothing is allocated on any call.
 * Limits: 1 <= M <= 16 token rows, N <= 4096 * 128, K a multiple of 8;
 *   larger M or N returns LLAMA_ERR_CAPACITY with a message.
 * The first call on a device, made with that device current, looks up the
 *   array's device address (a host-side symbol lookup); make that first call
 *   before any stream capture.  Every call clears the array's counters on
 *   `stream` before its kernel.
 * All calls share the one array: calls that overlap on the GPU (different
 *   streams, or threads without ordering) race and give wrong results. */
LLAMA_API int llama_op_linear_noalloc(const void* A, const void* W, int M, int N, int K, float* out,
                                      void* stream);

/* ---- a serving step over a paged KV cache -----------------------------------
 * The model's cache holds max_batch_size rows of max_seq_len positions
 * (llama_get_kv).  These operators serve requests of any mix of lengths from
 * a caller-owned pool of pages instead; one step runs
 *   llama_paged_plan -> llama_paged_append -> llama_paged_attention
 * (append and attention once per layer, on that layer's pools), and
 * llama_sample_rows draws the next tokens.  Shapes shared by the calls:
 *   pools         k_pages, v_pages [n_pages, n_kv_heads, page_size, head_dim] in
 *                 the cache's dtype; page_size 16, 32, 64, 128 or 256
 *   block_tables  int32 [B, max_pages]: entry i of row b is the page that holds
 *                 positions i*page_size .. of request b
 *   slot          page * page_size + position % page_size: a position's place in a pool
 *   packed rows   the new tokens of request b are rows cu_new[b] .. cu_new[b+1]-1
 * head_dim is 32, 64 or 128, n_heads / n_kv_heads 1, 2, 4 or 8, B at most 1024.
 * All lengths live in device memory: a step can be captured in a CUDA graph
 * and replayed.  `status` is a caller-owned device int32 (or NULL) that keeps
 * the first error code a kernel reports; the caller clears it. */

/* Block tables, slots, positions and offsets of one step, from its lengths.
 *   ctx_lens    int32 [B]: tokens of each request already in the cache
 *   new_lens    int32 [B]: tokens each request adds (0 allowed); negative: the
 *               request has ended and its ceil(ctx/page_size) pages go back to the list
 *   free_pages  int32 [n_pages]: a stack of free page ids, *free_count of them
 * Pages of ended requests are pushed in request order, then every growing
 * request takes ceil((ctx+new)/page_size) - ceil(ctx/page_size) pages from
 * the top, in request order, appended to its row of block_tables; the row of
 * an ended request and entries behind a request's pages are left as they were.
 *   seq_lens    int32 [B] out: ctx + new, 0 for an ended request (may be ctx_lens itself)
 *   cu_new      int32 [B+1] out: packed rows before each request, total at the end
 *   slots       int64 [T] out, positions int32 [T] out: of every packed row; -1
 *               behind the last row.  T is the arrays' length, at least the step's total
 *   free_left   int32 [1] out: free pages after the step (may be free_count itself)
 * All or nothing: if the step needs more pages than are free, more than
 * max_pages (or 2^30 tokens) per request or more than T rows (LLAMA_ERR_CAPACITY in
 * status), or a
 * ctx or free_count is negative or more pages are free than n_pages
 * (LLAMA_ERR_INVALID_ARG), nothing is taken or returned: every request adds no
 * token (cu_new all 0, slots and positions -1) and seq_lens and free_left repeat
 * their inputs.  Other outputs must not overlap inputs. */
LLAMA_API int llama_paged_plan(const int32_t* ctx_lens, const int32_t* new_lens, int B, int page_size,
                               int32_t* block_tables, int max_pages, int32_t* free_pages, int n_pages,
                               const int32_t* free_count, int T, int32_t* seq_lens, int32_t* cu_new, int64_t* slots,
                               int32_t* positions, int32_t* free_left, int32_t* status, void* stream);

/* The rotation table llama_paged_append reads: rope fp32 [len, head_dim/2, 2] =
 * (cos, sin)(t * theta^(-2j/head_dim)), in fp64 rounded once (Admin Guide §8.4). */
LLAMA_API int llama_rope_table(float* rope, int len, int head_dim, float theta, void* stream);

/* Per-head RMSNorm of queries and keys, rotation by position (adjacent pairs,
 * Admin Guide §8.4) and the write of K and V into their slots, in one pass.
 *   q, k, v     T rows of n_heads (n_kv_heads) * head_dim values, q_stride ...
 *               elements apart (three views of one fused projection, say), of
 *               in_dtype: LLAMA_F32 or the cache's dtype
 *   q_norm, k_norm  fp32 [head_dim] or NULL (no norm)
 *   rope        fp32 [rope_len, head_dim/2, 2];  positions int32 [T];  slots int64 [T]
 *   q_out       [T, n_heads, head_dim] in the cache's dtype (may be q itself if
 *               that has this type and layout); K and V go to k_pages, v_pages
 * fp32 arithmetic, one rounding; v of the cache's dtype is copied.  A row with
 * slot < 0 is padding: nothing of it is written.  A row with a slot
 * outside the pool or a position outside the table writes nothing and sets
 * LLAMA_ERR_CAPACITY in status.  The slots of one call must differ.  Bases,
 * rows, rope and norm weights 16-byte aligned. */
LLAMA_API int llama_paged_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                 int64_t v_stride, int in_dtype, int T, int n_heads, int n_kv_heads, int head_dim,
                                 const float* q_norm, const float* k_norm, float eps, const float* rope, int rope_len,
                                 const int32_t* positions, const int64_t* slots, void* q_out, void* k_pages,
                                 void* v_pages, int n_pages, int page_size, int dtype, int32_t* status, void* stream);

/* Causal grouped-query attention of each request's new tokens over its pages.
 *   q, out      [T, n_heads, head_dim] in the cache's dtype.  Scores, softmax
 *               statistics and sums are fp32; with a 16-bit cache the weights
 *               exp(score - maximum) are rounded once to its type for the
 *               product with V (their sum is taken before), as in the model's
 *               own attention, and the output is rounded once
 *   seq_lens    int32 [B]: tokens of each request in the cache, the new ones
 *               included: row i of request b's n new tokens sits at position
 *               seq_lens[b] - n + i and sees keys 0 .. that position
 *   max_new     most new tokens of one request (host): it chooses the kernel
 *               and sizes the workspace; a request with more is still right,
 *               but one far too high gives single tokens the chunk kernel's
 *               256-row tiles
 *   scale       factor of the scores (1/sqrt(head_dim) for the model's attention)
 *   workspace   llama_paged_attention_workspace_bytes() of device scratch,
 *               256-byte aligned, zero-filled before its first use (the kernels
 *               leave their counters at zero); calls sharing one must not
 *               overlap on the device.  A workspace for one max_new serves smaller
 *               ones.  Zero it again after LLAMA_ERR_DEVICE_TIMEOUT in status (a
 *               bounded wait of the chunk kernel gave up; outputs unspecified).
 * A row that sees no key (seq_lens[b] < n) gives zeros; rows behind the last
 * request are left as they were.  Keys behind a request's last token and keys
 * a row may not see do not reach its output, whatever their slots hold (NaN
 * included).  A request with rows outside 0..T is skipped
 * (LLAMA_ERR_INVALID_ARG in status); seq_lens[b] is cut to 0 ..
 * max_pages*page_size (LLAMA_ERR_CAPACITY); keys of a page outside the pool read
 * as zeros (LLAMA_ERR_INVALID_ARG). */
LLAMA_API size_t llama_paged_attention_workspace_bytes(int n_heads, int n_kv_heads, int head_dim, int dtype,
                                                       int max_new);
LLAMA_API int llama_paged_attention(const void* q, const void* k_pages, const void* v_pages, int dtype, int T,
                                    int n_heads, int n_kv_heads, int head_dim, int B, const int32_t* cu_new,
                                    const int32_t* seq_lens, const int32_t* block_tables, int max_pages, int n_pages,
                                    int page_size, int max_new, float scale, void* out, void* workspace,
                                    size_t workspace_bytes, int32_t* status, void* stream);

/* Per-launch timing of a model's projection kernels (for benchmarks).
 * llama_profile_start: from now on every projection launch the model enqueues
 *   (wq/wk/wv, wo, w1/w3, w2, output) is bracketed by two CUDA events recorded
 *   on the launch's own stream, for the first `capacity` launches.  Timed
 *   launches do not overlap their neighbours (no early launch).
 * llama_profile_stop: synchronises the events, writes up to `max` records
 *   (host arrays, any may be NULL): ms[i] = duration of launch i, bytes[i] =
 *   its algorithmic bytes (every weight once, the bf16 input rows once, the
 *   epilogue's outputs), flops[i] = 2*M*N*K summed over its projections,
 *   rows[i] = M; sets *n to the number of timed launches and stops timing.
 *   Events are created by start and destroyed by stop or llama_model_destroy. */
LLAMA_API int llama_profile_start(llama_model* m, int capacity);
LLAMA_API int llama_profile_stop(llama_model* m, float* ms, int64_t* bytes, int64_t* flops, int32_t* rows, int max,
                                 int* n);

/* Timeline of a model's decode steps (for benchmarks): where the time of a
 * step goes when its kernels overlap (programmatic dependent launch, CUDA
 * graph replay), which events between launches cannot show.
 * llama_timeline_start: zeroes the timeline on `stream` and, from now on,
 *   gives every kernel that llama_decode_step enqueues the next of up to 8192
 *   slots (embedding, RMSNorm, projection, attention, sampling launches).  A
 *   launch's CTAs leave in its slot the %globaltimer value (ns) at which the
 *   last of them finished (an atomic maximum), so launch i ran, exclusive of
 *   its predecessor, for end_ns[i] - end_ns[i-1].  A CUDA graph captured while
 *   the timeline records keeps its slots: each replay stamps them again
 *   (later replays leave later times).
 * llama_timeline_stop: stops giving out slots, synchronises the model's last
 *   stream and writes up to `max` records of the slots given out since the
 *   last start (host arrays, any may be NULL); it may be called again, e.g.
 *   after replaying a graph captured while recording, to read them anew:
 *   end_ns[i], kind[i] (LLAMA_TL_*), bytes[i] = the launch's algorithmic
 *   bytes where the host knows them (projections: every weight once, the
 *   16-bit input rows, the epilogue's outputs; embedding rows; sampling: the
 *   logits read), else 0; sets *n to the number of slots given out. */
#define LLAMA_TL_EMBED       0
#define LLAMA_TL_PROJECTION  1
#define LLAMA_TL_ATTENTION   2
#define LLAMA_TL_SAMPLE      3
#define LLAMA_TL_RMSNORM     4
LLAMA_API int llama_timeline_start(llama_model* m, void* stream);
LLAMA_API int llama_timeline_stop(llama_model* m, uint64_t* end_ns, int32_t* kind, int64_t* bytes, int max, int* n);

/* A stalled producer, for tests of the device-side timeout (failure
 * detection without a GPU fault).  Every wait of a kernel on another agent is
 * bounded; when one gives up, the kernel lets its own copies and tensor-core
 * operations in flight finish, releases its tensor memory, records
 * LLAMA_ERR_DEVICE_TIMEOUT in the model's device status word and returns.
 * llama_debug_stall arms that path once: in the next launch of the chosen
 * kernel by this model (16-bit models; LLAMA_STALL_PROJECTION: the next
 * projection, decode-shaped or prefill-shaped, on single SMs or CTA pairs;
 * LLAMA_STALL_ATTENTION: the next decode attention), CTA 0 never issues the
 * copies of pipeline stage `unit` of its run nor the barrier signal that
 * would announce them, and every wait of that launch gives up after wait_limit_ns
 * (1 us .. 2 s).  A unit past the end of CTA 0's run stalls nothing.  The
 * outputs of that step are unspecified; llama_model_status then returns the
 * timeout code and resets the model's internal counters, after which the next
 * call computes correctly.  LLAMA_STALL_NONE disarms a stall not yet taken.
 * Without a model (m NULL), LLAMA_STALL_PAGED arms the next llama_paged_attention
 * call of this process that takes the chunk kernel: stage 2i is the K tile of
 * CTA 0's i-th unit, 2i + 1 its V tile; the code arrives in that call's status,
 * and its workspace is zeroed before the next call. */
#define LLAMA_STALL_NONE        0
#define LLAMA_STALL_PROJECTION  1
#define LLAMA_STALL_ATTENTION   2
#define LLAMA_STALL_PAGED       3
LLAMA_API int llama_debug_stall(llama_model* m, int which, int unit, int64_t wait_limit_ns);

#ifdef __cplusplus
}
#endif

#endif /* LLAMA_B200_OPS_H */
