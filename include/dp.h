/*
 * dp.h -- C ABI of the GB300 (sm_103a) data-parallel collective data path.
 *
 * K data-parallel ranks are "virtual": K rank buffers that live in the one
 * GPU's device memory.  Every call enqueues hand-written CUDA kernels on the
 * caller's stream and returns; no call synchronises, except
 * dp_get_device_error().
 *
 * Shared conventions
 * ------------------
 *  - Pointer arrays (bufs, shards, out_*, w_shards, grads) are HOST arrays
 *    whose entries are DEVICE pointers, one per rank, in the manner of the
 *    per-device send/receive buffers of an NCCL all-reduce ("CMU 11-868
 *    L14-L15: Distributed Training and Data Parallelism, and Where Gradient
 *    Sync Costs Come From", section "NCCL's five building blocks" and the
 *    ncclAllReduce listing after "Ring AllReduce: ReduceScatter, then
 *    AllGather").  The host arrays are read during the call only; the
 *    pointers are passed by value to the kernels, so no host->device copy
 *    happens and the caller may reuse the host array at once.
 *  - Ownership: the caller owns all memory; no call allocates device memory.
 *    The library's state is a 4-byte device error word and the 8 MiB scratch
 *    array of dp_wgrad_reduce_scatter_noalloc (file-scope __device__
 *    variables, placed by the CUDA runtime when it loads the library), a
 *    cached driver entry point, four streams with their events per device
 *    for dp_all_gather_copy_engine (created on its first call), and the
 *    host-side bookkeeping (with their own streams and events) of the
 *    reducer, settle-pipe and AdamW objects the caller creates and destroys.
 *  - Chunks: a rank buffer of N elements is split into K chunks of
 *    C = ceil(N/K) elements; chunk c is [c*C, min((c+1)*C, N)) (the page's
 *    "each worker splits its gradient into K chunks").
 *  - Ring order: the reduced chunk c ends on rank c and is the fp32 left
 *    fold x_{c+1} + x_{c+2} + ... + x_{c} (rank indices mod K): at step s
 *    rank r passes chunk (r-s-1) mod K to rank r+1, which adds it to its own
 *    matching chunk (section "Ring AllReduce: ReduceScatter, then
 *    AllGather").  Results are bit-identical to that ring for every input,
 *    because the kernels keep this order for every element.
 *  - Arithmetic: bf16 inputs are widened exactly to fp32; the fold is fp32
 *    round-to-nearest-even; `scale` (1/K for the average of "Intuition: data
 *    parallelism has only one thing to synchronize", step 3) multiplies the
 *    folded fp32 value once; the result is rounded once to the output type
 *    (bf16: round-to-nearest-even).
 *  - Limits: 1 <= K <= DP_MAX_K.  N == 0 is a no-op returning DP_OK.
 *  - Memory: any address the GPU can dereference -- device memory, or pinned
 *    host memory (cudaHostAlloc / cudaMallocHost), which the kernels then
 *    read and write across the host link (zero-copy).  The alias checks
 *    compare addresses only.
 *  - Alignment: any element-aligned pointer is accepted; 16-byte-aligned
 *    buffers (with 16-byte-aligned chunk starts) take the vector path,
 *    anything else a slower scalar path with the same results.
 *  - Errors: a status is returned; DP_ERR_CUDA means a launch failed (the
 *    CUDA error is left for cudaGetLastError to report).  Invalid arguments
 *    are rejected before anything is enqueued.
 *  - Threads: every entry point is reentrant and may be called from several
 *    host threads (dp_wgrad_reduce_scatter_noalloc shares one scratch array:
 *    its calls must not overlap on the GPU).
 */
#ifndef DP_GB300_H
#define DP_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define DP_API __attribute__((visibility("default")))
#else
#define DP_API
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st* dp_stream_t;

typedef enum {
  DP_OK = 0,
  DP_ERR_INVALID_ARG = 1, /* null pointer, K out of range, N % K != 0, ...   */
  DP_ERR_UNSUPPORTED = 2, /* dtype or shape this entry point does not take   */
  DP_ERR_ALIAS = 3,       /* buffers that must be disjoint overlap           */
  DP_ERR_CUDA = 4,        /* a CUDA call failed (no device, launch failure)  */
  DP_ERR_TIMEOUT = 5      /* a bounded device-side wait expired (see below)  */
} dp_status_t;

typedef enum { DP_FP32 = 0, DP_BF16 = 1 } dp_dtype_t;

/* Microscaled 4-bit formats (see dp_mx4_quantize). */
typedef enum { DP_MXFP4 = 0, DP_NVFP4 = 1 } dp_mx4_format_t;

/* What dp_rms_norm quantises its output to. */
typedef enum {
  DP_NORM_PLAIN = 0,  /* nothing: y only */
  DP_NORM_MXFP4 = 1,
  DP_NORM_NVFP4 = 2,
  DP_NORM_MXFP8 = 3
} dp_norm_format_t;

/* How an optimizer keeps its states. */
typedef enum { DP_STATE_FP32 = 0, DP_STATE_8BIT = 1 } dp_state_t;

#define DP_MAX_K 16
#define DP_MAX_MICROBATCHES 16

/*
 * Ring all-reduce, in place ("CMU 11-868 L14-L15 ...", section "Ring
 * AllReduce: ReduceScatter, then AllGather": the reduce-scatter phase, then
 * the all-gather phase; section "NCCL's five building blocks": AllReduce =
 * ReduceScatter + AllGather; ring bound T_AR >= 2B(X-1)/(XW) in "Sharding
 * and Parallelism", section "The cost of the inserted collectives").
 *
 * bufs: K device buffers of N elements of `dtype`, pairwise disjoint.
 * After the call every bufs[r][e] = cast(scale * fold_c(e)), with c the chunk
 * of e.  Any N (C = ceil(N/K); trailing chunks may be short or empty).
 * One kernel reads and writes every element once.
 * Errors: DP_ERR_INVALID_ARG (null, K), DP_ERR_UNSUPPORTED (dtype),
 * DP_ERR_ALIAS (two ranks' buffers overlap), DP_ERR_CUDA.
 */
DP_API dp_status_t dp_ring_allreduce(void* const* bufs, int K, size_t N, dp_dtype_t dtype, float scale,
                              dp_stream_t stream);

/*
 * Ring reduce-scatter ("CMU 11-868 L14-L15 ...", section "Ring AllReduce:
 * ReduceScatter, then AllGather", phase 1; the FSDP backward's per-layer
 * gradient reduce-scatter of "Using ODC to Accelerate AMD SFT Training",
 * section "Why FSDP is Slow"; bound T_RS >= B(X-1)/(XW) in "Sharding and
 * Parallelism", section "The cost of the inserted collectives").
 *
 * bufs: K device buffers of N elements of in_dtype (not modified).
 * out_shards: K device buffers of N/K elements of out_dtype; out_shards[c]
 * receives cast(scale * fold_c) for chunk c (rank c's shard).
 * Requires N % K == 0 (even partition; padding indivisible sizes is the
 * caller's job).  Outputs must not overlap inputs or each other.
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA.
 */
DP_API dp_status_t dp_reduce_scatter(const void* const* bufs, int K, size_t N, dp_dtype_t in_dtype,
                              void* const* out_shards, float scale, dp_dtype_t out_dtype,
                              dp_stream_t stream);

/*
 * Ring reduce-scatter emitting both an fp32 and a bf16 shard from the same
 * scaled fp32 value, reading the inputs once (the FSDP gradient
 * reduce-scatter with a master-precision and a compute-precision copy; the
 * page "Sharding and Parallelism", section "Communication predictions",
 * notes that fp32 gradients double the bf16 byte counts).
 *
 * out_f32 (K buffers of N/K floats) or out_bf16 (K buffers of N/K bf16) may
 * be NULL, not both.  Otherwise as dp_reduce_scatter.
 */
DP_API dp_status_t dp_reduce_scatter_dual(const void* const* bufs, int K, size_t N, dp_dtype_t in_dtype,
                                   float* const* out_f32, void* const* out_bf16, float scale,
                                   dp_stream_t stream);

/*
 * Ring all-gather ("CMU 11-868 L14-L15 ...", section "Ring AllReduce:
 * ReduceScatter, then AllGather", phase 2; FSDP's parameter all-gather in
 * "Using ODC to Accelerate AMD SFT Training", section "Why FSDP is Slow";
 * bound T_AG >= B(X-1)/(XW) in "Sharding and Parallelism", section "The
 * cost of the inserted collectives").
 *
 * shards: K device buffers of shard_elems elements of dtype (rank c's
 * finished chunk c).  out: K device buffers of K*shard_elems elements; each
 * receives shard_0 .. shard_{K-1} concatenated, bit for bit.  Outputs must
 * not overlap each other or the shards.
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA.
 */
DP_API dp_status_t dp_all_gather(const void* const* shards, int K, size_t shard_elems, dp_dtype_t dtype,
                          void* const* out, dp_stream_t stream);

/*
 * FSDP forward: parameter all-gather fused into the local matmul ("Sharding
 * and Parallelism", section "Real HLO before and after partitioning": the
 * partitioned program all-gathers w[64,512] shards to w[512,512] before the
 * local dot with x[128,512]; section "FSDP and ZeRO": the forward pass
 * gathers W before the dot).
 *
 * x_local: device, row-major [M, D] bf16.  w_shards: K device buffers,
 * each row-major [F_shard, D] bf16; row f of the gathered weight w[F, D]
 * (F = K*F_shard) is row f mod F_shard of shard f / F_shard.  y: device,
 * row-major [M, F] of y_dtype (DP_BF16 or DP_FP32):
 *   y[m, f] = sum_d x[m, d] * w[f, d]   (y = x . w^T),
 * bf16 products accumulated in fp32 on the tensor cores; the gathered w is
 * never materialised (tiles are loaded by TMA straight from the shards).
 * Requires D % 8 == 0 and F_shard % 16 == 0, all base pointers 16-byte
 * aligned, M, D, F_shard < 2^31.  y must not overlap the operands.
 * The summation order over d is the tensor core's, so y matches an fp64
 * reference to within fp32 accumulation error, not bit for bit.
 *
 * workspace (optional, NULL / 0 bytes: none): caller-owned device memory of
 * workspace_bytes, 16-byte aligned, overlapping no operand or output, any
 * contents.  With at least dp_allgather_matmul_workspace_size() bytes, the
 * output tiles of a last round of the persistent grid that is at most half
 * full have their k-blocks split between several otherwise idle CTAs that
 * hand the fp32 accumulator on
 * through the workspace (the same chained split as dp_wgrad_reduce_scatter:
 * the result is bitwise the same with or without it, under any CTA limit).
 * Calls that may overlap on the GPU need separate workspaces.  Flags carry
 * a per-call value as for dp_wgrad_reduce_scatter: no clearing between
 * calls; after a captured call's replay reported DP_ERR_TIMEOUT, zero the
 * workspace before replaying again.
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED (shape/alignment, or a
 * device that is not sm_103), DP_ERR_ALIAS, DP_ERR_CUDA; DP_ERR_TIMEOUT is
 * reported later by dp_get_device_error if a pipeline wait expired.
 */
DP_API dp_status_t dp_allgather_matmul(const void* x_local, int M, int D, const void* const* w_shards,
                                int K, int F_shard, void* y, dp_dtype_t y_dtype,
                                void* workspace, size_t workspace_bytes, dp_stream_t stream);

/*
 * Workspace bytes with which dp_allgather_matmul(M, D, K, F_shard) splits its
 * last round on the current device under the current CTA limit; 0 when the
 * shape has no last round at most half full.  A smaller workspace is not an
 * error: the call then runs without the split.
 * Errors: DP_ERR_INVALID_ARG (bytes NULL, K out of range, negative sizes),
 * DP_ERR_CUDA (no device).
 */
DP_API dp_status_t dp_allgather_matmul_workspace_size(int M, int D, int K, int F_shard,
                                                      size_t* bytes);

/*
 * Tensor-parallel partial products summed across the ranks, fused into one
 * GEMM ("Sharding and Parallelism", section "Real HLO before and after
 * partitioning", TP-style fixture: the contracting dimension of both
 * operands is split over the ranks, each computes a partial dot, and an
 * eight-way all-reduce sums the partials; section "Parallelism strategies":
 * tensor parallelism communicates by AllReduce or AllGather/ReduceScatter).
 *
 * Rank r holds x_shards[r]: device, row-major [M, D_shard] bf16, and
 * w_shards[r]: device, row-major [F, D_shard] bf16 (the weight in the
 * [out, in] layout, so both operands are contiguous along the contracted
 * dimension).  The result is
 *   y[m, f] = scale * sum_r sum_d x_r[m, d] * w_r[f, d]
 * with every partial product accumulated in the same fp32 tensor-core
 * accumulator (the psum happens in TMEM; the partials are never written).
 *
 * dp_matmul_allreduce: y_out holds K device buffers [M, F] of y_dtype; every
 *   rank's buffer receives the whole result.
 * dp_matmul_reduce_scatter: requires M % K == 0; y_out[c] is a device buffer
 *   [M/K, F] receiving rows [c*M/K, (c+1)*M/K) -- chunk c of the row-major
 *   result, as the ring reduce-scatter of the flattened partials would leave
 *   on rank c.
 * Requires D_shard % 8 == 0, F % 16 == 0, 16-byte-aligned base pointers;
 * outputs must not overlap the operands or each other.  Accuracy as for
 * dp_allgather_matmul (fp32 accumulation, not bit-defined).  workspace /
 * workspace_bytes: optional, as for dp_allgather_matmul (size from
 * dp_matmul_workspace_size; bitwise the same result with or without).
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA.
 */
DP_API dp_status_t dp_matmul_allreduce(const void* const* x_shards, const void* const* w_shards,
                                       int K, int M, int D_shard, int F, void* const* y_out,
                                       dp_dtype_t y_dtype, float scale, void* workspace,
                                       size_t workspace_bytes, dp_stream_t stream);
DP_API dp_status_t dp_matmul_reduce_scatter(const void* const* x_shards,
                                            const void* const* w_shards, int K, int M,
                                            int D_shard, int F, void* const* y_out,
                                            dp_dtype_t y_dtype, float scale, void* workspace,
                                            size_t workspace_bytes, dp_stream_t stream);

/*
 * The same two calls in the x . w orientation of the page's fixture ("Sharding
 * and Parallelism", section "Real HLO before and after partitioning", TP-style
 * fixture x[1024,64] @ w[64,512] per rank: the weight is sharded along its
 * contracted rows): w_shards[r] is device, row-major [D_shard, F] bf16, and
 *   y[m, f] = scale * sum_r sum_d x_r[m, d] * w_r[d, f].
 * The tensor core reads w_r column-major from shared memory (the
 * instruction's B transpose), so nothing is transposed in memory.  Requires
 * F % 64 == 0 in addition to the conditions of dp_matmul_allreduce; outputs,
 * workspace (size from dp_matmul_xw_workspace_size) and errors as there.
 */
DP_API dp_status_t dp_matmul_allreduce_xw(const void* const* x_shards,
                                          const void* const* w_shards, int K, int M,
                                          int D_shard, int F, void* const* y_out,
                                          dp_dtype_t y_dtype, float scale, void* workspace,
                                          size_t workspace_bytes, dp_stream_t stream);
DP_API dp_status_t dp_matmul_reduce_scatter_xw(const void* const* x_shards,
                                               const void* const* w_shards, int K, int M,
                                               int D_shard, int F, void* const* y_out,
                                               dp_dtype_t y_dtype, float scale, void* workspace,
                                               size_t workspace_bytes, dp_stream_t stream);
DP_API dp_status_t dp_matmul_xw_workspace_size(int K, int M, int D_shard, int F, size_t* bytes);

/*
 * Workspace bytes with which dp_matmul_allreduce / dp_matmul_reduce_scatter
 * (K, M, D_shard, F) split their last round on the current device under the
 * current CTA limit (the two forms share their tiling); 0 when there is no
 * last round at most half full.  Errors as dp_allgather_matmul_workspace_size.
 */
DP_API dp_status_t dp_matmul_workspace_size(int K, int M, int D_shard, int F, size_t* bytes);

/*
 * The FSDP backward weight gradient fused with its reduce-scatter ("Using
 * ODC to Accelerate AMD SFT Training", section "Why FSDP is Slow": in the
 * backward pass each layer computes its full gradient and reduce-scatters it
 * to the rank's shard; "Sharding and Parallelism", section "Real HLO before
 * and after partitioning": an FSDP training step's backward adds a gradient
 * ReduceScatter).  For a linear layer y = x . w^T with w [F, D], rank r's
 * local weight gradient is dW_r = dY_r^T . X_r over its own T tokens, and the
 * data-parallel gradient is their sum ("CMU 11-868 L14-L15", section
 * "Intuition: data parallelism has only one thing to synchronize").
 *
 * Rank r holds dy[r]: device, row-major [T, F] bf16 (the layer's output
 * gradients, tokens x output features) and x[r]: device, row-major [T, D]
 * bf16 (its inputs).  The result is
 *   dW[f, d] = scale * sum_r sum_t dy_r[t, f] * x_r[t, d]
 * with every rank's products accumulated in the same fp32 tensor-core
 * accumulator (the per-rank dW_r are never written).  dw_shards[c] is a
 * device buffer [F/K, D] of dw_dtype receiving rows [c*F/K, (c+1)*F/K) of
 * dW -- chunk c of the row-major gradient, as the ring reduce-scatter of the
 * flattened dW_r would leave on rank c.  scale = 1/K averages.
 * Requires F % K == 0, F % 64 == 0, D % 64 == 0, 16-byte-aligned base
 * pointers; outputs must not overlap the operands or each other.  T == 0
 * writes zeros.  Accuracy as for dp_allgather_matmul (fp32 accumulation, not
 * bit-defined).
 *
 * workspace (optional, NULL / 0 bytes: none): caller-owned device memory of
 * workspace_bytes, 16-byte aligned, not overlapping the operands or outputs,
 * any contents.  With at least dp_wgrad_workspace_size() bytes, the output
 * tiles of a last, less-than-half-full round of the persistent grid have
 * their token blocks split between several CTAs, which hand the fp32
 * accumulator on through the workspace, so that round takes a fraction of a
 * tile's time.  The accumulation order is unchanged: the result is bitwise
 * the same with or without a workspace (and under any CTA limit).  Calls
 * that may overlap on the GPU need separate workspaces.  Each call tags its
 * hand-off flags with a 64-bit value of its own and clears each flag once
 * it is read, so the workspace needs no clearing between calls.  A replay
 * of a captured call reuses the captured value: after a replay whose wait
 * expired (DP_ERR_TIMEOUT), zero the workspace before replaying again.
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA;
 * DP_ERR_TIMEOUT (from dp_get_device_error) if a hand-off waited > 2 s.
 */
DP_API dp_status_t dp_wgrad_reduce_scatter(const void* const* dy, const void* const* x, int K,
                                           int T, int F, int D, void* const* dw_shards,
                                           dp_dtype_t dw_dtype, float scale, void* workspace,
                                           size_t workspace_bytes, dp_stream_t stream);

/*
 * Workspace bytes with which dp_wgrad_reduce_scatter(K, T, F, D) splits its
 * last round on the current device under the current CTA limit
 * (dp_set_cta_limits); 0 when the shape has no such round.  A smaller
 * workspace is not an error: the call then runs without the split.
 * Errors: DP_ERR_INVALID_ARG (bytes NULL, K out of range, negative sizes),
 * DP_ERR_CUDA (no device).
 */
DP_API dp_status_t dp_wgrad_workspace_size(int K, int T, int F, int D, size_t* bytes);

/*
 * The paper has no counterpart to this call: it exists for callers that
 * cannot allocate device memory.  Frameworks whose memory pool owns the GPU
 * may forbid allocations outside the pool; a training step may not afford
 * the device-wide synchronisation that cudaMalloc / cudaFree can cause; a
 * deployment may fix its device-memory budget at start-up.  Such callers
 * cannot hand dp_wgrad_reduce_scatter a workspace, and would lose its split
 * of a part-full last round.
 *
 * dp_wgrad_reduce_scatter_noalloc computes exactly what dp_wgrad_reduce_scatter
 * does with a sufficient workspace (same arguments, same result bits), taking
 * the scratch from a file-scope device array of DP_WGRAD_NOALLOC_MAX_BYTES
 * (8 MiB) that every GPU which loads this library holds until the process
 * exits.  The call allocates nothing.  It rejects a shape whose split would
 * need more scratch than that (dp_wgrad_workspace_size() > the maximum) with
 * DP_ERR_UNSUPPORTED, without launching; shapes that need no scratch run
 * unsplit.  The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current); make that first call
 * before any stream capture.  Every call on a device shares the one array,
 * which keeps the previous call's contents; none of it needs clearing,
 * because each call tags its hand-off flags with a 64-bit value of its own
 * and reads a partial sum only after its flag carries that value.  Calls
 * that may overlap on the GPU race on the array and give wrong results.
 * Otherwise as dp_wgrad_reduce_scatter.
 * Errors: as dp_wgrad_reduce_scatter, plus DP_ERR_UNSUPPORTED when the
 * scratch needed exceeds DP_WGRAD_NOALLOC_MAX_BYTES.
 */
#define DP_WGRAD_NOALLOC_MAX_BYTES ((size_t)8 << 20)
DP_API dp_status_t dp_wgrad_reduce_scatter_noalloc(const void* const* dy, const void* const* x,
                                                   int K, int T, int F, int D,
                                                   void* const* dw_shards, dp_dtype_t dw_dtype,
                                                   float scale, dp_stream_t stream);

/*
 * One microbatch into a rank's fp32 gradient accumulator ("Using ODC to
 * Accelerate AMD SFT Training", section "From Per-iteration to Per-minibatch
 * Synchronization": microbatch gradients are accumulated locally and settled
 * once per minibatch; section "odc_pad vs odc_nopad", Figure 5: padding
 * buckets contribute no valid gradient).
 *
 * acc: device, N floats.  grad: device, N elements of grad_dtype, or NULL
 * for a padding bucket (gradient +0; the accumulator is still read and
 * rewritten, as a padded microbatch still costs its pass).
 *   acc[e] = (first ? +0 : acc[e]) + widen(grad[e]).
 * The accumulator starts at +0, so a padding bucket never changes its bits.
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA.
 */
DP_API dp_status_t dp_grad_accumulate(float* acc, const void* grad, size_t N, dp_dtype_t grad_dtype,
                               int first, dp_stream_t stream);

/*
 * The variable-length step's accumulate and settle in one pass ("Using ODC
 * to Accelerate AMD SFT Training", sections "From Per-iteration to
 * Per-minibatch Synchronization" and "odc_pad vs odc_nopad").
 *
 * grads: HOST table of K*Mmax device pointers, row-major by rank
 * (grads[r*Mmax + j] is microbatch j of rank r, N elements of grad_dtype,
 * or NULL for a padding bucket).  m: HOST array of K counts, 0 <= m[r] <=
 * Mmax <= DP_MAX_MICROBATCHES.  Rank r's gradient is the fp32 sum
 * (+0) + g_{r,0} + ... + g_{r,m[r]-1}, in that order; the K sums are then
 * ring-reduce-scattered exactly as dp_reduce_scatter_dual with in_dtype
 * DP_FP32 would do on K accumulators built by dp_grad_accumulate, without
 * writing the accumulators.  Requires N % K == 0.  out_f32 / out_bf16 as in
 * dp_reduce_scatter_dual.
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA.
 */
DP_API dp_status_t dp_odc_reduce_scatter(const void* const* grads, const int* m, int K, int Mmax,
                                  size_t N, dp_dtype_t grad_dtype, float* const* out_f32,
                                  void* const* out_bf16, float scale, dp_stream_t stream);

/*
 * All-reduce of one DDP gradient bucket, in place, without flattening it
 * ("CMU 11-868 L14-L15 ...", section "When to sync: gradient bucketing":
 * gradients are grouped into buckets and each bucket is all-reduced as one
 * message).
 *
 * The bucket is the concatenation, in the given order, of n tensors; tensor t
 * has numels[t] elements of dtype and its K rank copies are
 * grads[t*K + r] (HOST array of n*K device pointers).  The result equals a
 * ring all-reduce of the flat bucket of total = sum numels elements: chunk
 * length C = ceil(total/K), an element at bucket offset o is folded in the
 * order of chunk o / C, scaled, cast and written back into every rank's copy.
 * All n*K buffers must be pairwise disjoint.  Any alignment and any sizes
 * (16-byte-aligned tensors take the vector path); a tensor with numels[t] ==
 * 0 takes no part, and its pointers may be NULL (as frameworks give empty
 * tensors), every other pointer must not be.
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA.
 */
DP_API dp_status_t dp_bucket_allreduce(void* const* grads, const size_t* numels, int n, int K,
                                       dp_dtype_t dtype, float scale, dp_stream_t stream);

/*
 * One microbatch group's settle in a cross-iteration settle pipeline ("Using
 * ODC to Accelerate AMD SFT Training", section "Discussion: Settle Does Not
 * Yet Overlap with Backward": the previous microbatch group's settle runs on
 * a separate stream beside this group's backward compute, joined once per
 * minibatch; the settle itself as in "From Per-iteration to Per-minibatch
 * Synchronization").
 *
 * A minibatch's microbatches are split into groups, index ranges of j shared
 * by the ranks.  grads / m / Mmax describe this group only, as for
 * dp_odc_reduce_scatter: m[r] (0 allowed) of rank r's microbatches, in
 * order.  Each rank's group sum (+0) + g_{r,j} + ... is ring-folded over the
 * ranks exactly as dp_odc_reduce_scatter does, giving the settled chunk S_c
 * (not yet averaged).  owner_acc: HOST array of K device pointers, chunk c's
 * fp32 running sum (N/K floats each, caller-owned, 16-byte aligned for the
 * vector path).  phase (bits):
 *   DP_SETTLE_FIRST            owner_acc[c] = +0 + S_c    (outputs unused)
 *   0                          owner_acc[c] = owner_acc[c] + S_c
 *   DP_SETTLE_LAST             out[c] = cast((owner_acc[c] + S_c) * scale)
 *   DP_SETTLE_FIRST|LAST       out[c] = cast(S_c * scale) (= dp_odc_reduce_scatter;
 *                              owner_acc may be NULL)
 * so the owner adds the groups' settled chunks in the order of the calls and
 * averages once.  out_f32 / out_bf16 as in dp_reduce_scatter_dual (required
 * only with DP_SETTLE_LAST).  owner_acc must not overlap the gradients or
 * the outputs.  Requires N % K == 0.
 * Errors: DP_ERR_INVALID_ARG (also: phase outside the two bits, owner_acc
 * NULL when a phase needs it), DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA.
 */
#define DP_SETTLE_FIRST 1
#define DP_SETTLE_LAST 2
DP_API dp_status_t dp_odc_settle_group(const void* const* grads, const int* m, int K, int Mmax,
                                       size_t N, dp_dtype_t grad_dtype, float* const* owner_acc,
                                       int phase, float* const* out_f32, void* const* out_bf16,
                                       float scale, dp_stream_t stream);

/*
 * The cross-iteration settle pipeline: a side stream and events that run
 * each pushed group settle beside the caller's compute, and one join per
 * minibatch ("Using ODC to Accelerate AMD SFT Training", section
 * "Discussion: Settle Does Not Yet Overlap with Backward").
 *
 * dp_settle_pipe_create: a pipe on the current device, with its own
 *   non-blocking stream and two events (the library's only allocations here:
 *   CUDA stream and event objects, no device memory).  cta_limit > 0 caps
 *   the CTAs of the pipe's settle launches (so the compute keeps the other
 *   SMs), on top of the process-wide limit of dp_set_cta_limits; 0: that
 *   limit alone.
 * dp_settle_pipe_push: the group's gradients are complete in `stream`'s
 *   order at this point; the call records that point, makes the pipe's
 *   stream wait for it and enqueues dp_odc_settle_group (same arguments) on
 *   the pipe's stream, then returns; work enqueued afterwards on `stream`
 *   (the next group's backward) runs concurrently with the settle.  Settles
 *   run in push order.  The pushed gradient buffers are read until the
 *   settle finishes: do not overwrite them before a dp_settle_pipe_wait.
 *   Arguments are validated before anything is enqueued.
 * dp_settle_pipe_wait: `stream` waits for every settle pushed so far (the
 *   once-per-minibatch join; afterwards the outputs, the owners'
 *   accumulators and the pushed gradient buffers are free to use in
 *   `stream`'s order).  Under stream capture, join before ending the
 *   capture.
 * dp_settle_pipe_destroy: waits for the pipe's stream, then frees it.
 * Pushes and waits from several threads are serialised per pipe; the
 * current device must be the pipe's.
 * Errors: DP_ERR_INVALID_ARG (NULL pipe, another device), the errors of
 * dp_odc_settle_group, DP_ERR_CUDA.
 */
typedef struct dp_settle_pipe dp_settle_pipe_t;
DP_API dp_status_t dp_settle_pipe_create(int cta_limit, dp_settle_pipe_t** pipe);
DP_API dp_status_t dp_settle_pipe_push(dp_settle_pipe_t* pipe, const void* const* grads,
                                       const int* m, int K, int Mmax, size_t N,
                                       dp_dtype_t grad_dtype, float* const* owner_acc, int phase,
                                       float* const* out_f32, void* const* out_bf16, float scale,
                                       dp_stream_t stream);
DP_API dp_status_t dp_settle_pipe_wait(dp_settle_pipe_t* pipe, dp_stream_t stream);
DP_API dp_status_t dp_settle_pipe_destroy(dp_settle_pipe_t* pipe);

/*
 * The DDP gradient Reducer (same sections of "CMU 11-868 L14-L15 ...":
 * bucket_cap_mb, the fixed parameter-to-bucket map, reverse parameter order,
 * pending counts, buckets launched strictly in order, unused parameters).
 *
 * dp_reducer_create: P parameters of numels[p] elements of dtype, K ranks,
 *   bucket cap in bytes (25 MB = 25*1024*1024 in DDP's default), scale for
 *   every bucket's all-reduce (1/K averages).  Parameters are walked from
 *   P-1 down to 0 and appended to the open bucket, which is closed as soon as
 *   its size reaches the cap.  *out receives an opaque host object.
 * dp_reducer_mark_ready: parameter p's gradient is ready on all K ranks at
 *   grads[0..K-1] (HOST array of device pointers, read during the call;
 *   NULL is accepted only for a parameter of 0 elements).
 *   Decrements p's bucket's pending count; then every consecutive complete
 *   bucket from the next unlaunched one onward is all-reduced on `stream`
 *   (dp_bucket_allreduce over its parameters, in bucket layout order), and
 *   *launched (nullable) receives how many were launched by this call.
 *   Marking a parameter twice in one iteration is DP_ERR_INVALID_ARG.
 * dp_reducer_finish: ends the iteration.  DP_OK if every bucket was launched;
 *   otherwise DP_ERR_INVALID_ARG with *first_pending = the first bucket that
 *   never completed (a parameter that took no part -- where DDP would hang).
 *   Either way the reducer is reset for the next iteration.
 * dp_reducer_bucket_info / dp_reducer_param_slot: the layout (bucket sizes,
 *   parameter -> (bucket, element offset in the bucket)).
 * dp_reducer_set_dry_run: when on, buckets are recorded but not launched
 *   (lets the host logic be exercised without a GPU);
 *   dp_reducer_launch_log copies this iteration's launched bucket ids.
 * dp_reducer_set_overlap: on != 0 makes the reducer create (on the current
 *   device) two non-blocking streams of its own and three events; from then
 *   on bucket b is all-reduced on stream b % 2, after an event recorded in
 *   the mark_ready call's `stream` at the point where the bucket completed,
 *   so the caller's stream goes on with the backward of earlier layers while
 *   the bucket is reduced ("When to sync: gradient bucketing": the Reducer
 *   launches an asynchronous AllReduce while backward keeps computing), and
 *   consecutive buckets, whose data are disjoint, may run at the same time.
 *   on == 0 waits for and frees them.  mark_ready must then be called with
 *   that device current.
 * dp_reducer_wait: `stream` waits for every bucket launched so far (the
 *   join before the optimizer step reads the gradients); DP_OK and nothing
 *   to do without overlap.  In overlap mode the gradients of a launched
 *   bucket must not be written again before this join.
 * dp_reducer_destroy also waits for the reducer's streams.
 * A reducer is used by one iteration at a time; its calls are serialised by
 * an internal mutex.
 */
typedef struct dp_reducer dp_reducer_t;
DP_API dp_status_t dp_reducer_create(const size_t* numels, int P, dp_dtype_t dtype, int K,
                                     size_t bucket_cap_bytes, float scale, dp_reducer_t** out);
DP_API void dp_reducer_destroy(dp_reducer_t* r);
DP_API int dp_reducer_num_buckets(const dp_reducer_t* r);
DP_API dp_status_t dp_reducer_bucket_info(const dp_reducer_t* r, int b, int* num_params,
                                          size_t* numel);
DP_API dp_status_t dp_reducer_param_slot(const dp_reducer_t* r, int p, int* bucket,
                                         size_t* offset);
DP_API dp_status_t dp_reducer_mark_ready(dp_reducer_t* r, int p, void* const* grads,
                                         dp_stream_t stream, int* launched);
DP_API dp_status_t dp_reducer_finish(dp_reducer_t* r, int* first_pending);
DP_API dp_status_t dp_reducer_set_dry_run(dp_reducer_t* r, int on);
DP_API int dp_reducer_launch_log(dp_reducer_t* r, int* buckets, int cap);
DP_API dp_status_t dp_reducer_set_overlap(dp_reducer_t* r, int on);
DP_API dp_status_t dp_reducer_wait(dp_reducer_t* r, dp_stream_t stream);

/*
 * The global norm of a list of gradients and the coefficient that clips it:
 * the step between the gradient reduce-scatter and the optimizer ("CMU 11-868
 * L14-L15 ...", "Intuition: data parallelism has only one thing to
 * synchronize": the synchronised gradient then updates the parameters).
 *
 * grads: HOST array of n device pointers, numels[t] elements of grad_dtype
 * each (a tensor of 0 elements takes no part; its pointer may be NULL).
 *   norm = sqrt(sum over all elements of g^2)
 *   coef = min(1, max_norm / (norm + 1e-6)), or NaN when norm is not finite
 * norm and coef: one device float each; either may be NULL, not both.
 * max_norm > 0 (infinity: coef is 1).  An empty list has norm 0.
 * Squares are summed in fp32 over 32 elements, pairs of such sums are added
 * in fp32, and the rest is in double; the order is fixed by the sizes and
 * alignments, so a list gives the same bits under any CTA limit.  fp32 bounds
 * the squares: one element above 1.8e19, or 64 that are summed together above
 * 2.3e18, make the norm infinite (and coef NaN); below 1e-19 squares lose bits,
 * below 2.6e-23 they are 0.  In between the norm is within 17 * 2^-24 of itself.
 *
 * workspace: device memory of at least dp_grad_norm_workspace_size(n) bytes,
 * 16-byte aligned, overlapping nothing; its first 4 bytes are zero before
 * the first call, and every call leaves them zero.  Calls that may overlap
 * on the GPU need separate workspaces.
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA.
 */
DP_API dp_status_t dp_grad_norm(const void* const* grads, const size_t* numels, int n,
                                dp_dtype_t grad_dtype, float max_norm, float* norm, float* coef,
                                void* workspace, size_t workspace_bytes, dp_stream_t stream);
DP_API dp_status_t dp_grad_norm_workspace_size(int n, size_t* bytes);

/*
 * AdamW (decoupled weight decay) over a list of tensors in one launch per
 * 384 of them: the update of each rank's parameter shard from its reduced
 * gradient shard ("Sharding and Parallelism", section "FSDP and ZeRO": the
 * optimizer states b_o are sharded with the parameters and gradients).
 *
 * dp_adamw_create checks a list of tensors once and keeps it (host memory
 * only); the buffers stay the caller's and are read and written by every
 * step.  All pointers are device pointers:
 *   param       numel elements of param_dtype, updated in place
 *   grad        numel elements of grad_dtype
 *   copy        NULL, or numel bf16: the new parameter rounded to bf16
 *   exp_avg, exp_avg_sq
 *               DP_STATE_FP32: numel floats each, m and v
 *               DP_STATE_8BIT: numel bytes each, e4m3 codes of m and of
 *               sqrt(v); with exp_avg_scale / exp_avg_sq_scale, ceil(numel /
 *               DP_STATE_BLOCK) floats each: a value is its code times the
 *               scale of its block of DP_STATE_BLOCK consecutive elements
 *   weight_decay  this tensor's (0: none)
 * All-zero states are those of a run's start.  A tensor of 0 elements takes
 * no part.  Any element alignment; fastest where fp32 arrays are 32-byte,
 * bf16 arrays 16-byte and code arrays 8-byte aligned.  No buffer that is
 * written may overlap another buffer of the list.
 *
 * dp_adamw_step: step t >= 1, for every element, in fp32 with one rounding
 * per operation (with bf16 parameters or 8-bit states the root, of any v
 * above 0, and the quotient to 2^-22):
 *   g = grad * *grad_scale          (grad_scale NULL: 1)
 *   m = m * beta1 + g * (1 - beta1)
 *   v = v * beta2 + (g * g) * (1 - beta2)
 *   p = p * (1 - lr * weight_decay)
 *       - (lr / (1 - beta1^t)) * (m / (sqrt(v) * (1 / sqrt(1 - beta2^t)) + eps))
 * the factors in t, lr and the betas alone in double, rounded once.  8-bit
 * states: the step uses this step's unrounded m and v; then each block's m
 * and sqrt(v) are stored as codes nearest (ties to even) to value * (448 /
 * largest magnitude of the block), and a sqrt(v) above zero keeps at least
 * the smallest code (2^-9).  Of a block whose largest magnitude is below
 * 2^-110 m is dropped.
 * Half a code's step is 3 to 6 % of a root, and a stored root moves only in a
 * step that changes it by that much; smaller changes are rounded away each time,
 * and the root follows its block's scale.  At beta2 <= 0.95 roots follow v (the
 * middle nine tenths are within 0.9 to 1.25 times theirs).  Nearer to 1 they do
 * not follow a v that shrinks: where the gradients of half of each block fell to
 * a tenth, those roots were 3.4 times too large (median) 3000 steps later at
 * beta2 = 0.999, 13 times at 0.99, and the block's other roots 0.8 and 1.4 times
 * theirs.  32-bit states have none of this.
 * grad_scale: NULL or a device float (dp_grad_norm's coef).  A NaN there
 * leaves every buffer as it is: the step is left out.
 * schedule: NULL, or 3 device floats (lr, 1 - beta1^t, 1 - beta2^t) that are
 * read when the kernel runs in place of the call's values: a captured step
 * is replayed with new ones.
 * Requires 0 <= beta < 1, eps >= 2^-126, finite lr.  Steps of one object are
 * serialised on the host; the caller orders them on the GPU.
 *
 * dp_adamw_count_skips: skips is a device word (4-byte aligned, outside the
 * list's buffers) to which every later step that is left out adds 1 when it
 * runs, or NULL, as at creation.  A step with a word takes t = step - *skips in
 * its bias corrections (without schedule), so that steps left out, which the
 * host does not know of, do not count; where *skips > 0 the corrections are
 * formed in fp32, within 2^-21.  The caller zeroes it before the first step.
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA.
 */
#define DP_STATE_BLOCK 256
typedef struct {
  void* param;
  const void* grad;
  void* copy;
  void* exp_avg;
  void* exp_avg_sq;
  float* exp_avg_scale;
  float* exp_avg_sq_scale;
  size_t numel;
  double weight_decay;
} dp_adamw_tensor_t;
typedef struct dp_adamw dp_adamw_t;
DP_API dp_status_t dp_adamw_create(const dp_adamw_tensor_t* tensors, int n,
                                   dp_dtype_t param_dtype, dp_dtype_t grad_dtype,
                                   dp_state_t state, dp_adamw_t** out);
DP_API dp_status_t dp_adamw_step(dp_adamw_t* o, double lr, double beta1, double beta2, double eps,
                                 long long step, const float* grad_scale, const float* schedule,
                                 dp_stream_t stream);
DP_API dp_status_t dp_adamw_count_skips(dp_adamw_t* o, unsigned int* skips);
DP_API void dp_adamw_destroy(dp_adamw_t* o);

/*
 * Microscaled 4-bit matrices: the form in which a parameter shard is gathered
 * into the GEMM that uses it ("Sharding and Parallelism", section
 * "Communication predictions": a collective's bytes follow the element type).
 *
 * A matrix [rows, cols], cols a multiple of 32, both at most 2^31 - 2^16, has
 *   codes    rows x cols/2 bytes: e2m1 values (0 0.5 1 1.5 2 3 4 6, bit 3 the
 *            sign), two to a byte, the earlier column in the low half
 *   scales   one byte for each block of consecutive columns:
 *              DP_MXFP4  blocks of 32, 2^(byte - 127), 255 is NaN
 *              DP_NVFP4  blocks of 16, e4m3; values are also times the
 *                        tensor's fp32 scale (tensor_scale NULL: 1)
 *            in tiles of 128 rows x 4 blocks, 512 bytes each: row r, block b
 *            of a tile at (r % 32) * 16 + (r / 32) * 4 + b; the tiles of 128
 *            rows one after another along the columns; zero where the matrix
 *            has no row or block.  dp_mx4_scales_size gives the bytes.
 * Both device buffers are 16-byte aligned.
 *
 * dp_mx4_quantize: x is a HOST array of K device pointers to row shards
 * [rows, cols] of x_dtype, rows ld elements apart.  The matrix quantised is
 * their row concatenation [K*rows, cols], or with transpose != 0 its
 * transpose [cols, K*rows] (blocks along the concatenated rows: the operand
 * of the backward products, gathered and transposed in one pass).  The
 * blocked dimension must be a multiple of 32.  In fp32, with a the largest
 * magnitude of a block:
 *   DP_MXFP4  scale 2^(floor(log2 a) - 2), at least 2^-127; values x / scale
 *   DP_NVFP4  scale s = e4m3(a * (1/6) / t), t = *tensor_scale (or 1);
 *             values x / (s * t)
 * rounded to the nearest e2m1, ties to even, saturating at 6.  A block of
 * zeros has codes 0 and scale byte 0; a block with a NaN or an infinity has
 * codes 0 and a NaN scale, so that it is NaN when used.
 *
 * dp_mx4_tensor_scale: *scale = (largest magnitude of n tensors of numels[t]
 * elements) / 2688, the t that takes the largest block's scale to 448 and its
 * values to 6.  NaN or infinity if an element is.  workspace as for
 * dp_grad_norm (dp_grad_norm_workspace_size(n) bytes, zeroed once).
 *
 * dp_mx4_dequantize: out [rows, cols] of out_dtype, the values rounded once.
 *
 * dp_allgather_matmul_mx4: dp_allgather_matmul with both operands in 4 bits:
 *   y[m, f] = sum_d x[m, d] * w[f, d]
 * x [M, D] and K weight shards [F_shard, D]; block-scaled tensor-core
 * products accumulated in fp32, the sum times the tensors' scales (times their
 * fp32 product: two scales whose product is below 2^-126 lose bits, or are 0, and
 * above 2^128 infinite), one rounding to y_dtype.  y: row-major [M, K*F_shard].
 * Requires D % 32 == 0, F_shard % 16 == 0, 16-byte aligned buffers; y overlaps no
 * operand.  The summation order over d follows from the sizes; under a CTA limit
 * the result is the same.  D == 0 writes zeros.
 *
 * dp_allgather_linear_mx4: the same with x [M, D] of x_dtype, rows ld elements
 * apart, quantised on the way (dp_mx4_quantize with tensor scale x_scale) into
 * workspace: device memory of dp_allgather_linear_mx4_workspace_size(M, D)
 * bytes, 16-byte aligned, any contents, overlapping nothing else; free again
 * in stream order.  All arguments are checked before anything is enqueued.
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA;
 * DP_ERR_TIMEOUT later from dp_get_device_error if a pipeline wait expired.
 */
typedef struct {
  const void* codes;
  const void* scales;
  const float* tensor_scale;  /* device float or NULL; DP_NVFP4 only */
} dp_mx4_t;
DP_API dp_status_t dp_mx4_scales_size(int rows, int cols, dp_mx4_format_t format, size_t* bytes);
DP_API dp_status_t dp_mx4_quantize(const void* const* x, int K, int rows, int cols, long long ld,
                                   dp_dtype_t x_dtype, dp_mx4_format_t format, int transpose,
                                   const float* tensor_scale, void* codes, void* scales,
                                   dp_stream_t stream);
DP_API dp_status_t dp_mx4_tensor_scale(const void* const* x, const size_t* numels, int n,
                                       dp_dtype_t x_dtype, float* scale, void* workspace,
                                       size_t workspace_bytes, dp_stream_t stream);
DP_API dp_status_t dp_mx4_dequantize(const void* codes, const void* scales, int rows, int cols,
                                     dp_mx4_format_t format, const float* tensor_scale, void* out,
                                     dp_dtype_t out_dtype, dp_stream_t stream);
DP_API dp_status_t dp_allgather_matmul_mx4(const dp_mx4_t* x, int M, int D,
                                           const dp_mx4_t* w_shards, int K, int F_shard,
                                           dp_mx4_format_t format, void* y, dp_dtype_t y_dtype,
                                           dp_stream_t stream);
DP_API dp_status_t dp_allgather_linear_mx4(const void* x, int M, int D, long long ld,
                                           dp_dtype_t x_dtype, const float* x_scale,
                                           const dp_mx4_t* w_shards, int K, int F_shard,
                                           dp_mx4_format_t format, void* y, dp_dtype_t y_dtype,
                                           void* workspace, size_t workspace_bytes,
                                           dp_stream_t stream);
DP_API dp_status_t dp_allgather_linear_mx4_workspace_size(int M, int D, dp_mx4_format_t format,
                                                          size_t* bytes);

/*
 * A few tokens times 4-bit weight shards, the tokens as they are:
 *   y[m, f] = tw * sum_d x[m, d] * w[f, d]
 * x [M, D] bf16, rows ld elements apart, any alignment (fastest where rows start
 * on 16-byte boundaries); w_shards, K, F_shard, format and y as for
 * dp_allgather_matmul_mx4, y of any alignment.  For the single tokens of a model
 * that is served: it reads the weights once for each 32 tokens; for more tokens the
 * products of quantised x are faster.
 * Weights are decoded exactly, but for mxfp4 blocks whose scale is below 2^-27 of
 * the largest scale of their row of w: those within 2^-25 of that scale.  x is exact
 * down to 2^-27 of its row's largest magnitude, and below it within 2^-35 of that
 * magnitude.  Products are summed in fp32, in an order that follows from the sizes
 * alone, M among them: a token's last bits may differ between batches.  tw, the
 * shard's tensor scale, multiplies the sum.  x holding a NaN or an infinity gives that
 * token NaN or infinities.  D == 0 writes zeros.
 * Requires D % 32 == 0, D <= 2^30, F_shard % 16 == 0, M <= 524280.
 * workspace: device memory of dp_allgather_linear_w4_workspace_size(M, D) bytes
 * (none for M <= 8), 16-byte aligned, any contents, overlapping nothing else; free
 * again in stream order.
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA;
 * DP_ERR_TIMEOUT later from dp_get_device_error if the wait for a copy expired.
 */
DP_API dp_status_t dp_allgather_linear_w4_workspace_size(int M, int D, size_t* bytes);
DP_API dp_status_t dp_allgather_linear_w4(const void* x, int M, int D, long long ld,
                                          const dp_mx4_t* w_shards, int K, int F_shard,
                                          dp_mx4_format_t format, void* y, dp_dtype_t y_dtype,
                                          void* workspace, size_t workspace_bytes,
                                          dp_stream_t stream);

/*
 * The 8-bit microscaled form of activations (mxfp8), for products whose x keeps
 * more bits than the weights.  A matrix [rows, cols], cols a multiple of 32, has
 *   codes    rows x cols bytes: e4m3 values
 *   scales   one byte for each 32 consecutive columns, 2^(byte - 127), 255 is
 *            NaN, in the tiles of the 4-bit forms (dp_mx4_scales_size(rows,
 *            cols, DP_MXFP4) bytes)
 * Both device buffers are 16-byte aligned.
 *
 * dp_mx8_quantize: x [rows, cols] of x_dtype, rows ld elements apart.  With a
 * the largest magnitude of a block, its scale is the smallest 2^e, e >= -127,
 * with a <= 448 * 2^e, so no value saturates; codes are x / 2^e rounded to the
 * nearest e4m3, ties to even.  A block of zeros has scale byte 0, a block with a
 * NaN or an infinity codes 0 and a NaN scale.
 * dp_mx8_dequantize: out [rows, cols] of out_dtype, the values rounded once.
 *
 * dp_allgather_matmul_mx8: dp_allgather_matmul_mx4 with x [M, D] in this form
 * (tensor_scale NULL) and the weight shards in DP_MXFP4: the tensor cores multiply
 * e4m3 by e2m1 values with both blocks' scales exactly and accumulate in fp32.
 * Requirements, y and errors are that call's.
 * dp_allgather_linear_mx8: the same with x [M, D] of x_dtype, rows ld elements
 * apart, quantised on the way (dp_mx8_quantize) into workspace: device memory of
 * dp_allgather_linear_mx8_workspace_size(M, D) bytes, as for
 * dp_allgather_linear_mx4.
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA;
 * DP_ERR_TIMEOUT later from dp_get_device_error if a pipeline wait expired.
 */
DP_API dp_status_t dp_mx8_quantize(const void* x, int rows, int cols, long long ld,
                                   dp_dtype_t x_dtype, void* codes, void* scales,
                                   dp_stream_t stream);
DP_API dp_status_t dp_mx8_dequantize(const void* codes, const void* scales, int rows, int cols,
                                     void* out, dp_dtype_t out_dtype, dp_stream_t stream);
DP_API dp_status_t dp_allgather_matmul_mx8(const dp_mx4_t* x, int M, int D,
                                           const dp_mx4_t* w_shards, int K, int F_shard, void* y,
                                           dp_dtype_t y_dtype, dp_stream_t stream);
DP_API dp_status_t dp_allgather_linear_mx8(const void* x, int M, int D, long long ld,
                                           dp_dtype_t x_dtype, const dp_mx4_t* w_shards, int K,
                                           int F_shard, void* y, dp_dtype_t y_dtype,
                                           void* workspace, size_t workspace_bytes,
                                           dp_stream_t stream);
DP_API dp_status_t dp_allgather_linear_mx8_workspace_size(int M, int D, size_t* bytes);

/*
 * The root-mean-square norm of a layer's input, with the residual's addition and
 * the operand of the 4-bit products in the same pass:
 *   h = x + residual                       rounded to dtype
 *   rstd = 1 / sqrt(mean over D of h^2 + eps)
 *   y = h * rstd * weight
 * x, residual: [M, D] of dtype, rows ldx / ldr elements apart; weight: D of
 * weight_dtype.  Without a residual (NULL, and h NULL) h is x.  Any element
 * alignment; fastest where every row starts on a 32-byte boundary.
 * Outputs, contiguous: h and y [M, D] of dtype; rstd M floats, or NULL; with a
 * format, codes and scales of y as dp_mx4_quantize (tensor_scale: nvfp4's, or
 * NULL for 1) and dp_mx8_quantize define them, from the unrounded y.  y may then
 * be NULL; without a format codes and scales are.
 * Arithmetic in fp32: a thread sums 16 or 32 squares in four chains, the rest is
 * pairwise (the same bits for a row in any call with a format, and in any without one
 * where D is a multiple of 16 and the weight and every buffer's rows start on 32-byte
 * boundaries; other calls sum in another order).  That holds magnitudes up to 3.2e18;
 * where the sum passes fp32 the mean is infinite, rstd 0, and y 0, or NaN where
 * h * weight, which is formed first, is infinite; in other rows it has to stay within
 * fp32, too.  With an eps below 1e-30, rows below 5e-19 lose bits of rstd and rows
 * below 1e-23 count as zeros (rstd is then infinite if eps is 0).  A row with a NaN is
 * NaN throughout.
 * Requires D <= 32768, and D % 32 == 0 with a format; eps >= 0 and finite.
 * M == 0 or D == 0 writes nothing, rstd neither.
 *
 * dp_rms_norm_backward: from dy (the gradient of y) and dh (that which reaches h
 * past the norm, or NULL: none), both [M, D] of dtype,
 *   g = dy * weight,  xh = h * rstd
 *   dx = rstd * (g - xh * mean over D of (g * xh)) + dh      of dtype, contiguous
 *   dweight = sum over rows of dy * xh                       D floats
 * dx is the gradient of x and of the residual alike.  A quantised y's gradient
 * passes straight through.  dweight is summed in fp32 over at most 304 sets of
 * rows, then over those; the order follows from M and D, so a repeated call gives
 * the same bits under any CTA limit.  M == 0 writes zeros to dweight.
 * workspace: device memory of dp_rms_norm_backward_workspace_size(M, D) bytes,
 * 32-byte aligned, any contents; free again in stream order.
 * Nothing that is written may overlap anything else.
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA;
 * DP_ERR_TIMEOUT later from dp_get_device_error if the wait for a copy expired.
 */
DP_API dp_status_t dp_rms_norm(const void* x, long long ldx, const void* residual, long long ldr,
                               int M, int D, dp_dtype_t dtype, const void* weight,
                               dp_dtype_t weight_dtype, float eps, void* h, void* y, float* rstd,
                               dp_norm_format_t format, const float* tensor_scale, void* codes,
                               void* scales, dp_stream_t stream);
DP_API dp_status_t dp_rms_norm_backward(const void* dy, long long ldy, const void* h,
                                        long long ldh, const void* dh, long long ldd, int M, int D,
                                        dp_dtype_t dtype, const void* weight,
                                        dp_dtype_t weight_dtype, const float* rstd, void* dx,
                                        float* dweight, void* workspace, size_t workspace_bytes,
                                        dp_stream_t stream);
DP_API dp_status_t dp_rms_norm_backward_workspace_size(int M, int D, size_t* bytes);

/*
 * The parameter all-gather on the GPU's copy engines instead of its SMs
 * ("Optimizing ML Concurrent Computation and Communication with GPU DMA
 * Engines", Q2 "ConCCL (DMA Offload)": collectives that only move data can
 * run on DMA engines so that a concurrent GEMM keeps every compute unit).
 * Same arguments and result as dp_all_gather: K*K device-to-device
 * cudaMemcpyAsync copies (destination rank r, shard c), no kernel.  The
 * copies run on four internal streams of the library (created, with their
 * events, on the first call on each device: make that call before any stream
 * capture), forked from `stream` and joined back to it through events, so
 * several DMA engines work at once (issued shard by shard, each engine on
 * another destination of the same shard, so that repeated reads of a shard
 * hit L2) and the result is ordered on `stream` like any other call.  Calls
 * from several host
 * threads are serialised while they issue.  Bit-identical to dp_all_gather.
 * Errors: DP_ERR_INVALID_ARG, DP_ERR_UNSUPPORTED, DP_ERR_ALIAS, DP_ERR_CUDA.
 */
DP_API dp_status_t dp_all_gather_copy_engine(const void* const* shards, int K,
                                             size_t shard_elems, dp_dtype_t dtype,
                                             void* const* out, dp_stream_t stream);

/*
 * Which implementation dp_ring_allreduce and dp_all_gather use for aligned
 * buffers (process-wide, default 0):
 *   0  automatic: the bulk-copy kernels (the faster on GB300), except an
 *      all-reduce of at most 32 KiB per rank, which starts sooner on the
 *      register kernel;
 *   1  registers: every thread loads 16-byte vectors from the K ranks, folds
 *      them and stores the result to the K ranks;
 *   2  bulk copies: tiles cross shared memory by cp.async.bulk (TMA) -- K
 *      bulk loads, the fold in shared memory, K bulk stores issued by one
 *      thread per tile (the all-reduce "streamed through shared memory or
 *      TMA once" rather than in K-1 passes); the all-gather gives each CTA
 *      one destination rank (one load, one store per tile; the K ranks'
 *      CTAs read each tile together, so DRAM serves it once), or, under a
 *      stream CTA limit, one source shard (one load, K stores per tile).
 * The variants give identical bits.  Returns DP_ERR_INVALID_ARG for other
 * values.
 */
DP_API dp_status_t dp_set_collective_variant(int variant);
DP_API int dp_get_collective_variant(void);

/*
 * Process-wide upper bounds on the CTAs one launch may use: gemm_ctas for
 * the tensor-core kernels (dp_allgather_matmul, dp_matmul_*,
 * dp_wgrad_reduce_scatter*; the weight gradient's workspace size follows the
 * limit; dp_allgather_matmul_mx4, dp_allgather_linear_mx4 and their mx8 forms,
 * which where they split a tile over a cluster of 2, 4 or 8 CTAs use one cluster at least),
 * stream_ctas for the streaming collectives (reduce-scatter, all-gather,
 * all-reduce, accumulate, bucket and variable-length kernels), the gradient
 * norm, AdamW, the 4- and 8-bit quantisation and the RMS norm; neither is for
 * dp_allgather_linear_w4.  0 means no limit (the default: one resident grid over
 * every SM).  Lets a caller leave SMs free
 * for a kernel on another stream -- the resource-partitioning experiment of
 * "Optimizing ML Concurrent Computation and Communication with GPU DMA
 * Engines" (Q2, "Resource Partitioning").  Results do not depend on the
 * limits.  Applies to launches made after the call, from any thread.
 */
DP_API dp_status_t dp_set_cta_limits(int gemm_ctas, int stream_ctas);
DP_API dp_status_t dp_get_cta_limits(int* gemm_ctas, int* stream_ctas);

/*
 * Synchronises `stream`, then reports and clears the device error word of
 * the current device: DP_ERR_TIMEOUT if a bounded device-side wait expired
 * in any kernel since the last call, DP_ERR_CUDA if the stream reported a
 * CUDA error, DP_OK otherwise.
 */
DP_API dp_status_t dp_get_device_error(dp_stream_t stream);

/*
 * Diagnostic: launches one block that waits, with the library's bounded
 * wait, on a barrier that nothing completes, for at most timeout_us
 * microseconds, then records the expiry in the device error word and
 * returns.  dp_get_device_error then reports DP_ERR_TIMEOUT.  Lets a test
 * exercise the timeout path without touching any other kernel.
 * timeout_us must be in [1, 2000000].
 */
DP_API dp_status_t dp_selftest_bounded_wait(uint32_t timeout_us, dp_stream_t stream);

/* Static, human-readable name of a status. */
DP_API const char* dp_status_string(dp_status_t s);

/* Library version as 10000*major + 100*minor + patch. */
DP_API int dp_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DP_GB300_H */
