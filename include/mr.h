/*
 * mr.h -- C ABI of libmr: the W-way elementwise sum-reduce and the param-contiguous gather on one
 * MI355X (gfx950).
 *
 * Plain C. Only <stddef.h> and <stdint.h> are needed.  Every pointer argument marked "device" is GPU
 * memory (hipMalloc'd or torch-allocated) on the current HIP device; "host" pointers are CPU memory
 * read during the call only.  Streams are hipStream_t values (NULL = the default stream); the type
 * below is layout-compatible with hipStream_t, so HIP callers pass their stream directly.
 *
 * Semantics shared by every entry point:
 *  - Work is enqueued asynchronously on `stream`; no call synchronises the host except
 *    mr_workspace_check, mr_set_workspace when it frees library-owned buffers, and the copy-engine
 *    gather mr_allgather_param_contig_sdma (see there).  Kernel faults surface at the caller's next
 *    synchronisation (HIP convention).
 *  - Arguments are validated before any HIP call; an invalid call enqueues nothing.
 *  - The caller owns every buffer it passes and keeps it alive until the stream work completes (with
 *    a caching allocator and side streams, record the buffer on the stream).  The library never frees
 *    caller memory.
 *  - Return value: MR_OK (0) or a negative mr_status code; mr_status_string() names it and
 *    mr_last_hip_error() gives the hipError_t behind the calling thread's last MR_ERR_HIP.
 */
#ifndef MR_H_
#define MR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct ihipStream_t;
typedef struct ihipStream_t* mr_stream; /* == hipStream_t */

typedef int mr_status;
#define MR_OK 0
#define MR_ERR_INVALID_ARG (-1) /* null pointer, W/G/P out of range, size overflow */
#define MR_ERR_DTYPE (-2)       /* dtype not supported by this operation */
#define MR_ERR_ALIAS (-3)       /* output partially overlaps an input */
#define MR_ERR_WORKSPACE (-4)   /* two-shot workspace missing or too small (barrier errors: mr_workspace_check) */
#define MR_ERR_HIP (-5)         /* a HIP runtime call failed; see mr_last_hip_error() */
#define MR_ERR_ENGINE (-6)      /* SDMA copy engines unavailable or a copy failed; see mr_last_hip_error() */

typedef enum mr_dtype { MR_BF16 = 0, MR_FP16 = 1, MR_FP32 = 2, MR_INT32 = 3 } mr_dtype;
typedef enum mr_mode { MR_ONESHOT = 0, MR_TWOSHOT = 1 } mr_mode;

#define MR_MAX_W 16
#define MR_MAX_PARAMS_PER_LAUNCH 128
#define MR_MAX_TABLE_W 64 /* ranks in the shard-list gathers (pointer tables ride in the launch arguments) */

/* Human-readable name of a status code (static string, never NULL). */
const char* mr_status_string(mr_status status);

/* hipError_t value behind the calling thread's most recent MR_ERR_HIP, or for MR_ERR_ENGINE the HSA
 * runtime's hsa_status_t (or -1: an engine reported a failed copy); 0 if none. */
int mr_last_hip_error(void);

/*
 * mr_allreduce_sum -- one rank's result of a sum all-reduce over W rank buffers.
 *
 * Computes, for every element i < n,
 *     out[i] = narrow( (((widen(bufs[0][i]) + widen(bufs[1][i])) + ...) + widen(bufs[W-1][i])) )
 * with each term widened exactly to fp32, every add an fp32 round-to-nearest-even add in rank order
 * 0..W-1 (no reassociation, subnormals kept), and the sum rounded to nearest even into `dtype`.
 * That is the elementwise sum each block of a one-shot custom all-reduce forms after pulling its
 * chunk from every peer (page "Question and suggestions about custom allreduce", the quoted one-shot
 * block schedule), and the per-slice sum of two-shot (same page, reduce-scatter then gather; page
 * "triton_multimem_all_reduce.py", the per-rank slice of 128-bit packs).  The result is bit-identical
 * in both modes.
 *
 *  bufs   host array of W device pointers, each to n contiguous elements of `dtype` (read only).
 *         Pointers may repeat.  Any alignment is accepted.  When every pointer and out have the same
 *         address modulo 16 the kernels use aligned 16-byte loads and stores; when they are all
 *         multiples of the element size but their 16-byte phases differ, each input pack is realigned
 *         in registers from the two aligned packs it straddles (slightly slower: about 26.4 us
 *         instead of 24.5 us one-shot, 35 us instead of 31.5 us two-shot, for W=8 bf16 at 16 MiB); when some
 *         pointer is not a multiple of the element size, the call runs element by element with
 *         single-byte loads and stores only (much slower), never an unaligned multi-byte access.
 *  W      1 .. MR_MAX_W.
 *  n      elements per buffer; n == 0 is a successful no-op.
 *  dtype  MR_BF16, MR_FP16 or MR_FP32 (output has the same dtype); MR_INT32 -> MR_ERR_DTYPE.
 *  out    device pointer to n elements.  out == bufs[k] (exactly) is allowed (in place); any other
 *         overlap with an input -> MR_ERR_ALIAS.
 *  mode   MR_ONESHOT: one pass, W reads and one write per element.
 *         MR_TWOSHOT: phase 1 reduces the message into a stage buffer, share by share, an intra-GPU
 *         flag hand-off orders the phases, phase 2 copies the stage into out; the result is the
 *         same.  The shares are whole 16-byte packs of the aligned body (on out's 16-byte grid):
 *         W chunks of ceil(packs/W) packs each (the last ones may be short or empty), or, on the
 *         16-byte path with W <= 8 (the last arriver at any size, per-tile flags from 16 to
 *         64 MiB), one run of units per XCD (1, 4 or 16 KiB of output each, by size); the few
 *         elements before out's first 16-byte boundary and after its last whole pack are reduced
 *         with the first share.  (mr_reduce_scatter_sum's chunks, which are defined on element
 *         indices, coincide with the W chunks when n is a multiple of 16 bytes and out is 16-byte
 *         aligned.)  Needs a workspace (see below).
 *  stream hipStream_t to enqueue on.
 */
mr_status mr_allreduce_sum(const void* const* bufs, int W, size_t n, mr_dtype dtype, void* out,
                           mr_mode mode, mr_stream stream);

/*
 * mr_allgather_param_contig -- scatter a rank-major gathered buffer into [param][rank] order.
 *
 * src holds W rank shards of T = sum(splits) elements each, back to back ([W][T]).  Shard r is laid
 * out as P parameter pieces of splits[s] elements at offset O_s = splits[0] + ... + splits[s-1].
 * out receives, for every parameter s, the W pieces of s one after another:
 *     out[O_s*W + r*splits[s] + j] = src[r*T + O_s + j]
 * Ranks form W/G node-blocks of G ranks; the launch walks node-block m, then parameter s, then slot g
 * (rank r = m*G + g), placing node-block m of parameter s at O_s*W + m*G*splits[s] with slot stride
 * splits[s] (page "ccl: hierarchical cross-node AllGather (intra-node SDMA + inter-node RDMA) #441",
 * the commit adding enqueue_param_contiguous and the commit fusing the node-block x split loop into
 * one launch).  The output does not depend on G.  It is a pure bit copy: every dtype bit pattern,
 * NaN payloads included, is preserved; dtype only sets the element size.
 *
 *  src     device pointer, W*T elements (read only).
 *  W       1 .. 65535;  G >= 1 with W % G == 0 (G == W: one node-block).
 *  splits  host array of P element counts (splits[s] == 0 allowed).  Read during the call only.
 *  P       >= 1.  Up to MR_MAX_PARAMS_PER_LAUNCH parameters go in one kernel launch; more are split
 *          into independent launches of up to that many parameters each (all validated before the
 *          first is enqueued).
 *  dtype   any mr_dtype (element size 2 or 4 bytes).
 *  out     device pointer, W*T elements.  Any overlap with src -> MR_ERR_ALIAS.
 *  Any alignment of src and out is accepted: pieces whose source and destination share a 16-byte
 *  phase are copied as aligned 16-byte packs, others as destination-aligned packs realigned in
 *  registers, and pointers that are not multiples of the element size make the launch work in bytes
 *  (byte-granular edges).  All offsets are 64-bit; buffers beyond 2^31 bytes are supported.
 */
mr_status mr_allgather_param_contig(const void* src_rank_major, int W, int G, const uint64_t* splits,
                                    int P, mr_dtype dtype, void* out, mr_stream stream);

/*
 * mr_allgather_param_contig_sdma -- mr_allgather_param_contig's placement, copied by the GPU's SDMA
 * engines instead of its compute units.
 *
 * The mori page's hierarchical all-gather moves intra-node data on copy engines so that a concurrent
 * GEMM keeps the compute units (page "ccl: hierarchical cross-node AllGather (intra-node SDMA +
 * inter-node RDMA) #441", PR summary: copy engines against CU contention).  Here every (parameter,
 * rank) piece -- src[r*T + O_s .. + splits[s]) to out[O_s*W + r*splits[s] ..) -- is one 1-D engine copy
 * (pieces above 8 MiB are cut), spread over every SDMA engine the device reports.  An engine spends
 * about 15 microseconds on every copy beyond its bytes, so parameters whose pieces are smaller than
 * MR_OPT_SDMA_CU_BELOW bytes are copied instead by one launch of the param-contiguous kernel on
 * `stream`, which runs beside the engine copies (the same page later moves a copy step from the
 * engines to a compute-unit kernel).  Output bits are those of mr_allgather_param_contig.
 *
 * Arguments, limits and errors as mr_allgather_param_contig, plus MR_ERR_ENGINE.  Unlike every other
 * entry point this call is synchronous: it waits until `stream` has finished its earlier work (the
 * engines are not ordered by the stream), then copies (the kernel part, if any, enqueued on `stream`),
 * and returns once every copy is complete, the kernel part's included; work
 * enqueued on any stream afterwards sees the result.  Not capturable in a HIP graph.  The first call
 * on a device initialises the HSA runtime and creates one HSA signal that the library keeps for that
 * device until the process ends.
 *
 * mr_sdma_engines: number of SDMA engines the current device offers for its own memory; 0 if none or
 * the HSA runtime is unavailable, and then mr_last_hip_error() gives the HSA runtime's hsa_status_t.
 */
mr_status mr_allgather_param_contig_sdma(const void* src_rank_major, int W, int G, const uint64_t* splits, int P,
                                         mr_dtype dtype, void* out, mr_stream stream);
int mr_sdma_engines(void);

/*
 * mr_reduce_scatter_chunk / mr_reduce_scatter_sum -- one rank's share of a sum reduce-scatter.
 *
 * Two-shot's first phase hands chunk c of the message to owner c (page "Question and suggestions
 * about custom allreduce", the two-shot reduce-scatter; page "triton_multimem_all_reduce.py", each
 * rank's slice of cdiv(numel/8, W) 128-bit packs); it is also the gradient half of FSDP sharding.
 * Chunk c is elements [c*C, min((c+1)*C, n)) with C = ceil(n/W) rounded up to a whole 16 bytes
 * (8 bf16/fp16 or 4 fp32 elements), so trailing chunks may be short or empty.
 *
 * mr_reduce_scatter_chunk: host-only; writes chunk `rank`'s first element and length.
 * mr_reduce_scatter_sum:   out[j] = the mr_allreduce_sum formula at element offset+j, for j < count,
 *                          reading only that chunk of each rank buffer.  bufs/W/n/dtype as for
 *                          mr_allreduce_sum; 0 <= rank < W; out is a device buffer of `count`
 *                          elements; out may equal bufs[k] + offset exactly (in place), any other
 *                          overlap with a read chunk -> MR_ERR_ALIAS.  count == 0 is a no-op.
 */
mr_status mr_reduce_scatter_chunk(size_t n, int W, mr_dtype dtype, int rank, size_t* offset, size_t* count);
mr_status mr_reduce_scatter_sum(const void* const* bufs, int W, size_t n, mr_dtype dtype, int rank, void* out,
                                mr_stream stream);

/*
 * mr_allreduce_sum_noalloc -- mr_allreduce_sum that never allocates device memory, for callers that
 * cannot allocate: code under HIP graph capture, serving loops that must not allocate, harnesses that
 * forbid it.
 *
 * Same arguments, result bits and errors as mr_allreduce_sum, with these differences:
 *  - the two-shot workspace is a device array inside the library (MR_NOALLOC_MAX_BYTES of stage plus
 *    the barrier words, about 34 MiB per GPU), held by each GPU the library runs on until the process
 *    ends; the first call on a device looks its address up and clears it on `stream`;
 *  - a rank buffer larger than MR_NOALLOC_MAX_BYTES (n * element size) -> MR_ERR_WORKSPACE, nothing
 *    enqueued;
 *  - the two-shot hand-off is always the last arriver (on XCD-local units on the 16-byte path with
 *    W <= 8, else on chunk tiles), ignoring MR_OPT_TWOSHOT_SYNC and
 *    MR_OPT_TILE_SHAPE: no workgroup of it ever waits, so it never leaves a barrier word set after a
 *    launch and never produces an invalid output; there is no error word to check;
 *  - every call on one GPU shares that GPU's array: two-shot calls that overlap in time on one GPU (on
 *    two streams, or from two host threads) race and give undefined output.  One-shot calls use no
 *    workspace and never race.
 */
#define MR_NOALLOC_MAX_BYTES ((size_t)32 << 20)
mr_status mr_allreduce_sum_noalloc(const void* const* bufs, int W, size_t n, mr_dtype dtype, void* out,
                                   mr_mode mode, mr_stream stream);

/*
 * All-gathers from W separate rank shards (each a device buffer of T elements), one launch each.
 * Bit copies of any dtype; 1 <= W <= MR_MAX_TABLE_W; shards may not overlap any output (MR_ERR_ALIAS).
 * Shard and output pointers may have any alignment (as for mr_allgather_param_contig).
 *
 * mr_allgather_into_tensor:  rank-major gather (torch.distributed.all_gather_into_tensor's layout):
 *                            out[r*T + j] = shards[r][j]; out holds W*T elements.
 * mr_allgather_list:         list-output gather (torch.distributed.all_gather's layout, page "ccl:
 *                            hierarchical cross-node AllGather ...", the commit adding the list-output
 *                            all_gather): outs[r][j] = shards[r][j]; outs is a host array of W device
 *                            buffers of T elements that may not overlap one another.
 * mr_allgather_param_contig_shards: the param-contiguous placement of mr_allgather_param_contig
 *                            written straight from the W shards, with no rank-major intermediate (the
 *                            zero-copy push of enqueue_param_contiguous on the same page):
 *                            out[O_s*W + r*splits[s] + j] = shards[r][O_s + j].
 */
mr_status mr_allgather_into_tensor(const void* const* shards, int W, size_t T, mr_dtype dtype, void* out,
                                   mr_stream stream);
mr_status mr_allgather_list(const void* const* shards, int W, size_t T, mr_dtype dtype, void* const* outs,
                            mr_stream stream);
mr_status mr_allgather_param_contig_shards(const void* const* shards, int W, int G, const uint64_t* splits, int P,
                                           mr_dtype dtype, void* out, mr_stream stream);

/*
 * mr_layer_norm_forward -- layer norm of the sum of W rank buffers and a residual.
 *
 * For every row of `cols` elements, in fp32 and in this order,
 *     x = widen(bufs[0]) + widen(bufs[1]) + ... + widen(bufs[W-1]) + widen(residual)
 *     mean = avg(x),  var = avg((x - mean)^2),  rstd = 1 / sqrt(var + eps)
 *     y = narrow((x - mean) * rstd * gamma + beta)
 * W = 1 without a residual is a plain layer norm.  W > 1 is what follows a tensor-parallel all-reduce: the
 * one-shot sum of mr_allreduce_sum, the residual and the norm in one pass, x rounded once, when it is stored.
 *
 *  bufs      host array of W (1 .. MR_MAX_W) device pointers, each rows*cols elements of `dtype`.
 *  residual  device, rows*cols elements, or NULL.
 *  gamma, beta  device, cols elements of `wdtype`; NULL stands for ones / zeros.
 *  dtype     MR_BF16, MR_FP16 or MR_FP32; wdtype: dtype or MR_FP32.  Others -> MR_ERR_DTYPE.
 *  x_out     device, rows*cols elements: narrow(x), the residual stream and what the backward pass takes; or NULL.
 *  y         device, rows*cols elements.
 *  mean, rstd  device, rows floats each, for the backward pass; or NULL.
 *  x_out and y may each be one of the bufs or the residual exactly; any other overlap of an output with an
 *  input or another output -> MR_ERR_ALIAS.  Pointers are multiples of their element size (else
 *  MR_ERR_INVALID_ARG); rows need not start on any larger grid.  rows == 0 or cols == 0 is a no-op.
 *  cols < 2^31, eps >= 0 and within fp32's range (0, or 2^-149 to 2^128).  Infinities and NaN give what the formula gives, in their row only.
 */
mr_status mr_layer_norm_forward(const void* const* bufs, int W, const void* residual, const void* gamma, const void* beta,
                                size_t rows, size_t cols, mr_dtype dtype, mr_dtype wdtype, double eps, void* x_out, void* y,
                                float* mean, float* rstd, mr_stream stream);

/*
 * mr_layer_norm_backward -- the gradients of mr_layer_norm_forward.
 *
 * With xh = (x - mean) * rstd and gd = gamma * dy (rows as above, fp32),
 *     dx     = narrow(rstd * (gd - avg(gd) - xh * avg(gd * xh)) + dres)
 *     dgamma = sum over rows of dy * xh,   dbeta = sum over rows of dy      (rounded once, to wdtype)
 * dx is the gradient of every rank buffer and of the residual alike.  The weight gradients' sums are fp32 in an
 * order set by the shape alone: results are the same bits on every call.
 *
 *  dy, x     device, rows*cols elements of `dtype`; x is the forward pass's x_out (or its one buffer).
 *  gamma     as in the forward pass (NULL: ones);  mean, rstd: rows floats from the forward pass.
 *  dres      device, rows*cols elements: the gradient that reaches x beside the norm; or NULL.
 *  dx        device, rows*cols elements, or NULL; may be dy, x or dres exactly.
 *  dgamma, dbeta  device, cols elements of `wdtype`, or NULL.  With rows == 0 they become zeros.
 *  Other overlaps, types and alignments as above.  The weight gradients' partial sums take up to 2 KiB a column of the
 *  stream's library workspace (see mr_set_workspace); one that the caller binds is large enough for any number of rows
 *  with mr_workspace_bytes(1, 512 * max(cols, 32), MR_FP32) bytes.
 */
mr_status mr_layer_norm_backward(const void* dy, const void* x, const void* gamma, const float* mean, const float* rstd,
                                 const void* dres, size_t rows, size_t cols, mr_dtype dtype, mr_dtype wdtype, void* dx,
                                 void* dgamma, void* dbeta, mr_stream stream);

/*
 * mr_grad_norm -- the 2-norm of a list of gradients and the factor that clips it.
 *
 *     out[0] = N = scale * sqrt(sum over all tensors of g^2)
 *     out[1] = scale * min(1, max_norm / (N + 1e-6))     (scale alone where max_norm <= 0)
 *     out[2] = 1 if every element is finite, else 0      (out[1] is then 0)
 * The sum is fp64 and in an order set by the sizes alone.  mr_adamw_step takes `out` as its `clip`, so a
 * step reads the factor on the device and is left out where a gradient is not finite, with no host round trip.
 *
 *  grads   host array of P device pointers, counts[i] elements of `dtype` (MR_BF16, MR_FP16, MR_FP32) each,
 *          multiples of the element size; counts[i] == 0 allowed (its pointer is not read), and P == 0.
 *  scale   finite and > 0: e.g. 1 / the loss scale.  max_norm: finite.
 *  out     device, 3 floats; overlap with a gradient -> MR_ERR_ALIAS.
 *  Takes 4 KiB of the stream's library workspace for every 128 tensors; one that the caller binds is large enough with
 *  mr_workspace_bytes(1, 8 * P + 1024, MR_FP32) bytes.
 */
mr_status mr_grad_norm(const void* const* grads, const uint64_t* counts, int P, mr_dtype dtype, double scale,
                       double max_norm, float* out, mr_stream stream);

/*
 * mr_adamw_step -- one AdamW step over a list of tensors.
 *
 * For every element, in fp32, with step t and f = clip[1] (1 without clip),
 *     g = f * grad,  m' = beta1*m + (1-beta1)*g,  v' = beta2*v + (1-beta2)*g^2
 *     p' = (1 - lr*weight_decay)*p - lr/(1-beta1^t) * m' / (sqrt(v')/sqrt(1-beta2^t) + eps)
 *
 * The optimizer state is flat: tensor i's part starts at the sum of the earlier counts, each rounded up to a
 * multiple of 32, and mr_adamw_state_elems gives its total length.  Elements between tensors are kept at 0.
 *
 * MR_STATE_FP32:  m and v are floats.  m_scale and v_scale are NULL.
 * MR_STATE_MXFP8: m and v are bytes, E4M3 numbers in blocks of 32 that share a scale 2^(b-127), b the block's
 *     byte in m_scale / v_scale (the OCP microscaling format MXFP8).  v holds the square root of the second
 *     moment.  The scale is the smallest that brings the block's largest magnitude to 448 or less (b = 255: not
 *     finite, the whole block reads as NaN).  Values are rounded to one of their two neighbours, up with
 *     probability (distance to the lower) / (spacing), by 16 bits of a hash of (seed, t, element): calls with the same
 *     arguments give the same bits.  A second moment whose root is 2^-149 or more is never rounded to zero.  A state of zero
 *     bytes is the start.  The step itself uses m' and v' before they are rounded.  Gradients (times f) below 2^47 in magnitude; the
 *     block of a larger one becomes not finite.
 * master: floats, or NULL.  With it, p is read from master and written to both; `params` is not read (and may be NULL
 *     if params_out is given).  Only for 16-bit parameters.
 *
 *  params, grads  host arrays of P device pointers, counts[i] elements each, of dtype and grad_dtype (MR_FP32, or
 *           MR_BF16/MR_FP16 with grad_dtype the same or MR_FP32), multiples of their element size.
 *  state    host struct of device pointers, 256-byte aligned (scales: any).
 *  params_out, state_out  where results go; NULL: in place.  Each output may be its own input exactly; any
 *           other overlap -> MR_ERR_ALIAS.
 *  hyper    host struct; beta1, beta2 in [0, 1), eps 0 or at least 2^-126, lr, weight_decay and eps finite, t >= 1.
 *  clip     device, mr_grad_norm's 3 floats, or NULL.  Where clip[2] is 0 the step is not taken: outputs
 *           are the inputs (params_out the rounded master, with one).
 *  Up to 80 tensors go in one launch; counts[i] == 0 is allowed, counts[i] <= 2^33.
 *  hyper is read on the host: a HIP graph that captured the call repeats the same lr, t and seed at every replay, so its
 *  bias corrections stand still and 8-bit moments meet the same random bits, whose roundings then no longer average out.
 */
typedef enum mr_state_format { MR_STATE_FP32 = 0, MR_STATE_MXFP8 = 1 } mr_state_format;
typedef struct mr_adamw_state {
  void* m;
  void* v;
  uint8_t* m_scale;
  uint8_t* v_scale;
  float* master;
} mr_adamw_state;
typedef struct mr_adamw_hyper {
  double lr, beta1, beta2, eps, weight_decay;
  uint64_t step; /* t, from 1 */
  uint64_t seed;
} mr_adamw_hyper;
mr_status mr_adamw_state_elems(const uint64_t* counts, int P, uint64_t* elems);
mr_status mr_adamw_step(const void* const* params, const void* const* grads, const uint64_t* counts, int P, mr_dtype dtype,
                        mr_dtype grad_dtype, mr_state_format format, const mr_adamw_state* state, void* const* params_out,
                        const mr_adamw_state* state_out, const mr_adamw_hyper* hyper, const float* clip, mr_stream stream);

/*
 * mr_muon_step -- one Muon step over a list of matrices: momentum, orthogonalisation by Newton-Schulz products, update.
 *
 * For every matrix of rows[i] x cols[i], with f = clip[1] (1 without clip),
 *     g = f * grad,   m' = momentum*m + (1-momentum)*g,   u = momentum*m' + (1-momentum)*g (nesterov) or m'
 *     X = u / max(|u|, eps)  (Frobenius norm),  steps times:  X = (a I + b X X^T + c (X X^T)^2) X
 *     p' = (1 - lr*weight_decay)*p - lr*s*X,   s = sqrt(max(1, rows/cols)) (MR_MUON_RATIO) or 0.2 sqrt(max(rows, cols)) (MR_MUON_RMS)
 *
 *  params, grads  host arrays of P device pointers to row-major matrices, as for mr_adamw_step (types, alignment, NULL params
 *           with a master copy and params_out).  rows[i], cols[i] <= 65536, either may be 0.
 *  state    momentum and master: floats, laid out as mr_adamw_state_elems says (counts rows[i]*cols[i]), 256-byte aligned;
 *           elements between matrices become 0.  master NULL: none; with it, p is read from master and written to both.
 *  params_out, state_out  where results go; NULL: in place.  Each output may be its own input exactly; any other overlap
 *           -> MR_ERR_ALIAS.
 *  hyper    momentum in [0, 1), eps from 2^-114, lr, weight_decay and eps finite.  steps 1 to 16.  coefficients: host array of
 *           {a, b, c} for every step; NULL: 3.4445, -4.775, 2.0315.  Polynomials that take a singular value of X past 3.8, or P = a I
 *           + b A + c A^2 past 15, -> MR_ERR_INVALID_ARG.
 *           products = 16: operands of the products rounded to fp16 (held times 2^12, sums fp32); X is then off by 1e-3 to 2e-2
 *           of its norm, the more the lower its rank; 32: operands in two fp16 pieces, three products for one; off as fp32 is.
 *  clip     device, mr_grad_norm's 3 floats, or NULL.  Where clip[2] is 0 the step is not taken: outputs are the inputs.
 *  A gradient or momentum that is not finite gives NaN in its own matrix only.
 *  Matrices are worked off up to 32 at a time, in the stream's library workspace (see mr_set_workspace), about six to ten bytes
 *  an element for products = 16 and twice that for 32, with sides rounded up to multiples of 96 (a matrix of few rows or columns takes
 *  more: 65536 x 1 25 MB), up to 2 GiB or what the largest matrix takes.  The library's own is kept, as for the other calls, until
 *  mr_set_workspace replaces it.  mr_muon_workspace_bytes: bytes that one bound by the caller needs for a list (0: invalid
 *  arguments).  hyper is read on the host: a graph repeats its lr.
 */
typedef enum mr_muon_adjust { MR_MUON_RATIO = 0, MR_MUON_RMS = 1 } mr_muon_adjust;
typedef struct mr_muon_state {
  float* momentum;
  float* master;
} mr_muon_state;
typedef struct mr_muon_hyper {
  double lr, momentum, weight_decay, eps;
  const double* coefficients; /* host, 3 * steps, or NULL */
  int steps, nesterov, products;
  mr_muon_adjust adjust;
} mr_muon_hyper;
size_t mr_muon_workspace_bytes(const uint64_t* rows, const uint64_t* cols, int P, int products);
mr_status mr_muon_step(const void* const* params, const void* const* grads, const uint64_t* rows, const uint64_t* cols, int P,
                       mr_dtype dtype, mr_dtype grad_dtype, const mr_muon_state* state, void* const* params_out,
                       const mr_muon_state* state_out, const mr_muon_hyper* hyper, const float* clip, mr_stream stream);

/*
 * Losses on logits: log-probabilities of target tokens with their gradient, a clipped policy loss and a preference loss.
 *
 * Logits are `rows` rows (tokens, of any number of packed sequences) of `cols` elements (the vocabulary) of `dtype` (MR_BF16,
 * MR_FP16, MR_FP32), `stride` >= cols elements apart, so that a padded vocabulary's last columns may be left out; rows and
 * pointers lie anywhere on the element grid.  In fp32, with T the temperature (> 0, log2(e)/T a normal fp32 number),
 *     m = max_j z_j,   S = sum_j exp((z_j - m) / T),   logp = (z_t - m) / T - ln S
 * A row whose target lies outside [0, cols) (-100, say: prompts and padding), or, in the policy loss, whose weight is 0, carries
 * no loss: it is not read, its logp and statistics are 0 and its gradient is zeros.  Logits of -inf have probability 0; other
 * infinities and NaN give what the formulas give, in their row and in the sums over rows.
 *
 * mr_token_logprob_forward:   logp (rows floats, or NULL) and stats (rows pairs of floats {m, S} for the backward pass, or NULL).
 * mr_token_logprob_backward:  dlogits[i][j] = narrow(dlogp_i / T * ([j = t_i] - exp((z_ij - m_i) / T) / S_i))
 * mr_policy_loss:  for each row, with r = exp(logp - old_logp) and d = ref_logp - logp,
 *         loss_i = max(-A r, -A min(max(r, 1 - clip_low), 1 + clip_high)) + kl_coef * (exp(d) - d - 1)
 *     record[0..3] = sums over the rows of  w loss_i,  w (exp(d) - d - 1),  w [the clipped term is the larger],  w
 *     (fp64 sums in an order set by the sizes and the rows' alignment), and with dlogits the gradient of grad_scale * record[0], from the same
 *     pass over the logits where a row fits a workgroup's registers: 131072 16-bit or 65536 fp32 columns on the 16-byte grid, 131065
 *     or 65533 where rows start off it.  Longer rows, fewer than 32 rows of more than three quarters of that, and rows of less
 *     than 16 bytes are read twice.  A term that is clipped, and only that, passes no gradient.
 *       old_logp  of the policy that sampled the tokens; NULL: of this one (r = 1).  ref_logp: NULL without a KL term (d = 0); with
 *       kl_coef 0 the term is reported in record[1] and left out of the loss and the gradient.  exp is finite up to fp64's range.
 *       advantages  rows floats;  weights: rows floats (a mask over its sum, say), or NULL: ones.
 *       logp, dlogits  or NULL.
 * mr_preference_loss:  rows hold 2 * pairs sequences, sequence k in [offsets[k], offsets[k+1]): pair p's chosen one is 2p, its
 *     rejected one 2p+1.  With s_k the sum of logp - ref_logp over a sequence and h_p = beta * (s_2p - s_2p+1),
 *         loss_p = -(1 - smoothing) ln sigmoid(h_p) - smoothing ln sigmoid(-h_p)
 *     record[0..2] = loss_scale * sum of loss_p,  the share of h_p > 0,  the mean of h_p;  margins[p] = h_p, or NULL;
 *     dlogp: the gradient of grad_scale * record[0] by each row's logp, zeros in rows of no sequence, or NULL; may be logp
 *     exactly.  offsets (device) do not decrease; they are held to [0, rows], and others give undefined values.
 *
 *  targets  device, rows int64.  dlogits: rows `dstride` elements apart, only their `cols` elements written; it may be the logits
 *           exactly, with their stride.  Other overlaps -> MR_ERR_ALIAS; the rest is checked as above.  rows == 0 is a no-op,
 *           but for the records, which become zeros.
 *  The losses and a forward pass of few rows keep partial sums in the stream's library workspace; one that the caller binds
 *  is large enough with mr_workspace_bytes(1, 256 * rows + 65536, MR_FP32) bytes.
 */
typedef struct mr_policy_hyper {
  double temperature, clip_low, clip_high, kl_coef, grad_scale; /* clip_low in [0, 1], clip_high >= 0, grad_scale > 0 */
} mr_policy_hyper;
typedef struct mr_preference_hyper {
  double beta, smoothing, loss_scale, grad_scale; /* smoothing in [0, 0.5], grad_scale > 0 */
} mr_preference_hyper;
mr_status mr_token_logprob_forward(const void* logits, size_t rows, size_t cols, size_t stride, mr_dtype dtype, const int64_t* targets,
                                   double temperature, float* logp, float* stats, mr_stream stream);
mr_status mr_token_logprob_backward(const void* logits, size_t rows, size_t cols, size_t stride, mr_dtype dtype, const int64_t* targets,
                                    double temperature, const float* stats, const float* dlogp, void* dlogits, size_t dstride,
                                    mr_stream stream);
mr_status mr_policy_loss(const void* logits, size_t rows, size_t cols, size_t stride, mr_dtype dtype, const int64_t* targets,
                         const float* old_logp, const float* ref_logp, const float* advantages, const float* weights,
                         const mr_policy_hyper* hyper, float* record, float* logp, void* dlogits, size_t dstride, mr_stream stream);
mr_status mr_preference_loss(const float* logp, const float* ref_logp, size_t rows, const int64_t* offsets, size_t pairs,
                             const mr_preference_hyper* hyper, float* record, float* margins, float* dlogp, mr_stream stream);

/*
 * Two-shot workspace.
 *
 * By default the library allocates, on first two-shot use of a (device, stream) pair, a grow-only
 * workspace of at least mr_workspace_bytes() bytes holding the stage buffer and the barrier words.
 * Growth at least doubles the size and keeps the replaced buffer alive, so launches in flight and HIP
 * graphs that captured a two-shot call on the stream stay valid; replaced buffers are freed only by
 * mr_set_workspace on that stream.  One workspace per (device, stream): eager two-shot calls on
 * different streams never share barrier words.  The layer norm's backward pass, the gradient norm and the losses keep
 * their partial sums there too, mr_muon_step its matrices.  Calls on one stream from several host threads are safe: each enqueues its kernels together.
 * (hipStreamPerThread is one handle and a stream of each thread: make such calls on it from one thread only.)
 *
 * A two-shot call made while its stream is being captured into a HIP graph uses a library-owned
 * workspace of that capture (device, stream, capture id), allocated during the capture with this
 * thread's capture mode relaxed for the allocation and cleared by a kernel recorded into the graph.  So
 * graphs captured one after another on one stream -- torch.cuda.graph captures every graph on one
 * shared stream -- never share barrier words, and may be replayed at the same time on different
 * streams.  Two replays of the same graph that overlap in time do share its workspace and race.  These
 * workspaces live until mr_set_workspace is called on the capture stream (destroy the graphs first).
 * Caller-owned memory bound with mr_set_workspace is used for captured calls too.
 *
 * Every launch returns its barrier words and flags to zero before it ends, also when a bounded wait
 * gave up (the call that timed out has invalid output; later calls are unaffected).
 *
 * mr_workspace_bytes: bytes a caller-owned workspace needs for a two-shot call of this shape (and, as described there,
 *                     for mr_layer_norm_backward, mr_grad_norm and the losses).
 * mr_set_workspace:   bind caller-owned device memory (256-byte aligned) as the workspace of `stream`
 *                     on the current device, replacing any library-owned one; the barrier words and
 *                     flags are cleared on `stream` here.  Memory too small to hold them plus some
 *                     stage -> MR_ERR_INVALID_ARG; a bound workspace too small for a later call makes
 *                     that call return MR_ERR_WORKSPACE.  dev_ptr == NULL unbinds (the library
 *                     allocates again on next use).  Either way it synchronises `stream` and frees
 *                     every library-owned workspace buffer of the stream (its captures' included), so
 *                     a graph that captured a two-shot call on it must not be replayed afterwards.
 *                     If a free fails, the call returns MR_ERR_HIP and leaves the stream with no
 *                     workspace bound.  Not thread-safe against concurrent calls on that stream.
 * mr_workspace_check: synchronises `stream`, then reads and clears the barrier error words of its
 *                     workspaces (its own and those of graphs captured on it).  *flags receives their
 *                     OR: 0 = no error; bit 0 = a phase-2 workgroup gave up waiting for phase 1, so
 *                     that call's output is not valid; bits 1 and 2 = the XCD-local two-shot
 *                     recomputed units from the rank buffers (after a wait gave up / because a
 *                     unit's producer ran on another XCD than the workgroup that copies it), output
 *                     valid.  Returns MR_ERR_WORKSPACE if
 *                     there is no workspace for the stream.
 */
size_t mr_workspace_bytes(int W, size_t n, mr_dtype dtype);
mr_status mr_set_workspace(mr_stream stream, void* dev_ptr, size_t bytes);
mr_status mr_workspace_check(mr_stream stream, uint32_t* flags);

/*
 * Process-wide options (thread-safe; they apply to calls made after the change).
 *
 * MR_OPT_TWOSHOT_SYNC  how a two-shot phase-2 tile waits for phase 1 (all give identical results):
 *   MR_TWOSHOT_SYNC_AUTO  (default) LAST up to 32 MiB per rank buffer, TILE above;
 *   MR_TWOSHOT_SYNC_TILE  per-tile producer flags: a phase-2 tile waits only for the
 *                         phase-1 tiles it copies (the per-block flag hand-off of the custom
 *                         allreduce page's block_barrier, applied to the two phases);
 *   MR_TWOSHOT_SYNC_CHUNK per-chunk barrier: waits for every phase-1 tile of its 1/W chunk;
 *   MR_TWOSHOT_SYNC_GRID  grid barrier: waits for every phase-1 tile of every chunk;
 *   MR_TWOSHOT_SYNC_LAST  no waiting: each group of phase-1 tiles counts its releases, and the
 *                         workgroup whose release completes the group copies it.
 *   Under TILE (16 to 64 MiB per rank buffer) and LAST (any size) the 16-byte path with W <= 8 runs
 *   on XCD-local units (16 KiB of output each from 8 MiB per rank buffer, 4 or 1 KiB below; one run
 *   per XCD) unless MR_OPT_TILE_SHAPE forces a tile shape; otherwise on W chunks.
 * MR_OPT_SPIN_LIMIT    polls a waiting workgroup makes before it gives up and sets the workspace error
 *                      word (see mr_workspace_check); default 2^22.  A value of 0 makes every wait
 *                      that is not already satisfied give up at once (for testing error handling).
 * MR_OPT_TILE_SHAPE    tile shape of the sum-reduce kernels (results are identical for every shape):
 *   MR_TILE_AUTO   (default) chosen from the message size and dtype: narrow below 64 Ki packs
 *                  of 16 B, medium below 256 Ki (fp32) or 512 Ki (16-bit types) packs,
 *                  MR_TILE_WIDE_PAIR from 1 Mi to 4 Mi packs (16 to 64 MiB per rank buffer) when
 *                  W <= 8, wide otherwise; two-shot: 64-pack tiles below 8 Ki packs, 256 below 128 Ki, 1024 above;
 *   MR_TILE_WIDE   one-shot 256 lanes x 4 packs of 16 B (256 x 1 for W > 8), two-shot phase-1
 *                  tiles of 1024 packs;
 *   MR_TILE_MEDIUM one-shot 256 x 1, two-shot 256-pack tiles;
 *   MR_TILE_NARROW one-shot 64 x 1, two-shot 64-pack tiles;
 *   MR_TILE_WIDE_PAIR  one-shot: wide tiles pipelined on a persistent grid of resident workgroups,
 *                  each storing one tile's sums while the next tile's loads are in flight (W <= 8;
 *                  wide for W > 8); two-shot under TILE or LAST: XCD-local units at any size
 *                  (W <= 8, 16-byte path), otherwise as MR_TILE_WIDE.
 * MR_OPT_SDMA_CU_BELOW mr_allgather_param_contig_sdma: a parameter whose per-rank piece is smaller than
 *                      this many bytes is copied by the compute-unit kernel, the others by the engines;
 *                      0 puts every piece on the engines.  0 .. 2^32-1, default 1048576 (1 MiB).  The
 *                      kernel part needs free compute units: beside a kernel that holds them all, the
 *                      call returns only after that kernel has made room, so a caller that must not
 *                      wait on other work sets 0.
 * Unknown options or out-of-range values -> MR_ERR_INVALID_ARG.  Environment variables
 * MR_TWOSHOT_SYNC, MR_SPIN_LIMIT, MR_TILE_SHAPE and MR_SDMA_CU_BELOW set the initial values when the
 * library loads; a value that is not a whole number in the option's range is ignored.  MR_TRACE=1 makes
 * every launch print its plan (path, shape, grid) to stderr.
 */
typedef enum mr_option {
  MR_OPT_TWOSHOT_SYNC = 0,
  MR_OPT_SPIN_LIMIT = 1,
  MR_OPT_TILE_SHAPE = 2,
  MR_OPT_SDMA_CU_BELOW = 3
} mr_option;
#define MR_TWOSHOT_SYNC_TILE 0
#define MR_TWOSHOT_SYNC_CHUNK 1
#define MR_TWOSHOT_SYNC_GRID 2
#define MR_TWOSHOT_SYNC_LAST 3
#define MR_TWOSHOT_SYNC_AUTO 4
#define MR_TILE_AUTO 0
#define MR_TILE_WIDE 1
#define MR_TILE_MEDIUM 2
#define MR_TILE_NARROW 3
#define MR_TILE_WIDE_PAIR 4
mr_status mr_set_option(mr_option opt, int64_t value);
mr_status mr_get_option(mr_option opt, int64_t* value);

/* Library ABI version (major*100 + minor).  1.01 added MR_OPT_TILE_SHAPE, MR_TWOSHOT_SYNC_LAST and
 * MR_TWOSHOT_SYNC_AUTO (the new default hand-off); 1.02 added MR_TILE_WIDE_PAIR; 1.03 added
 * mr_allgather_param_contig_sdma, mr_sdma_engines and MR_ERR_ENGINE; 1.04 added
 * mr_allreduce_sum_noalloc and the last-arriver hand-off on XCD-local units (the default up to 32 MiB
 * per rank buffer); 1.05 added MR_OPT_SDMA_CU_BELOW (small parameters of the SDMA gather on the
 * compute units).  The training-step entry points (mr_layer_norm_forward and those after it) came later
 * under the same number: they add symbols and change none. */
int mr_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MR_H_ */
