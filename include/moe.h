/*
 * moe.h -- C ABI of the GB300 (sm_103a) sparse Mixture-of-Experts block
 * (Qwen3-MoE style: router, softmax over the E experts, top-k, renormalised
 * weights, grouped SwiGLU experts, weighted combine back to token order).
 *
 * The op sequence is the one the unsloth commit page 80aaf1121b
 * ("Qwen3-30B-A3B decode ... CUDA-graph capture", paragraph on the grouped_mm
 * backend) names for the MoE block: expert histogram (bincount, replaced by a
 * capture-safe scatter_add_), cumsum, argsort, torch._grouped_mm, index_add_.
 * Here each op is a hand-written CUDA kernel; the whole block runs without a
 * host synchronisation, so moe_route, moe_permute, moe_grouped_swiglu,
 * moe_unpermute and the moe_forward* calls that take a caller workspace can be
 * captured in a CUDA graph (the capture failure that page describes came from
 * a host round trip inside bincount).
 *
 * Notation: T tokens, H hidden size, E experts, k experts per token, I expert
 * intermediate size, A = T*k assignments.  Assignment a = t*k + j is token t's
 * j-th choice (j = 0 is the largest router logit).  All arrays are row-major
 * and C-contiguous.
 *
 * Conventions shared by every entry point:
 *  - Every data pointer is a DEVICE pointer owned by the caller; the library
 *    never allocates, frees or copies to the host, and never synchronises the
 *    stream (moe_read_device_error excepted).  Work is enqueued on `stream`
 *    (NULL = the legacy default stream) in stream order; outputs are ready
 *    when the stream reaches that point.
 *  - Device pointers must be 16-byte aligned (MOE_ERR_ALIGN otherwise).
 *  - Arguments are validated on the host before anything is launched; on any
 *    error nothing is enqueued and the error code is returned.
 *  - Calls on different streams are independent if they use different
 *    workspaces and outputs; two calls in flight must not share a workspace.
 *  - Inconsistent device data (an expert id outside [0, E) given to
 *    moe_permute) is not trapped: the kernel records MOE_ERR_DEVICE in the
 *    workspace's error word, skips the bad element and returns.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream. */
typedef struct CUstream_st *moe_stream_t;

enum moe_status {
    MOE_OK = 0,
    MOE_ERR_NULLPTR = -1,    /* a required pointer is NULL */
    MOE_ERR_SHAPE = -2,      /* sizes outside the supported range (see moe_shape) */
    MOE_ERR_DTYPE = -3,      /* unsupported activation / weight dtype combination */
    MOE_ERR_WORKSPACE = -4,  /* workspace NULL or smaller than moe_workspace_size() */
    MOE_ERR_ALIGN = -5,      /* a device pointer is not 16-byte aligned */
    MOE_ERR_LAUNCH = -6,     /* the CUDA runtime rejected a launch */
    MOE_ERR_DEVICE = -7      /* recorded on the device: inconsistent input data */
};

enum moe_dtype {
    MOE_DT_F32 = 0,   /* IEEE fp32 */
    MOE_DT_BF16 = 1,  /* bfloat16 (stored as 16-bit patterns) */
    MOE_DT_Q4 = 2     /* 4-bit codebook codes + bf16 block scales (expert weights only) */
};

/*
 * Problem sizes and formats.
 *   1 <= E <= 256, 1 <= k <= min(E, 32), 0 <= T <= 2^18, T*k < 2^30,
 *   H and I positive multiples of 8.
 * Supported (act_dtype, w_dtype): (F32, F32), (BF16, BF16), (BF16, Q4).
 *   act_dtype is the dtype of x, the router weight and the output.
 *   Q4 needs q_block even, dividing both H and I.
 * norm_topk != 0 renormalises the k selected softmax probabilities to sum to 1
 * (Qwen3-30B-A3B's norm_topk_prob); 0 keeps the softmax probabilities.
 */
typedef struct {
    int32_t T, H, E, k, I;
    int32_t act_dtype;
    int32_t w_dtype;
    int32_t norm_topk;
    int32_t q_block;
} moe_shape;

/*
 * 4-bit expert weights.  With w_dtype == MOE_DT_Q4, the w_gate / w_up / w_down
 * arguments point to packed codes: row-major [E][rows][in/2] bytes where
 * element 2i of a row sits in the low nibble of byte i and element 2i+1 in the
 * high nibble ("in" is the input dim: H for gate/up, I for down; rows is I for
 * gate/up and H for down).  Element value = codebook[code] * scale, with one
 * bf16 scale per q_block consecutive input-dim elements of a row:
 * scales are row-major [E][rows][in/q_block] bf16 DEVICE arrays.  The
 * codebook is given by value (host memory) and travels in the kernel
 * parameters.
 */
typedef struct {
    const void *gate_scales;
    const void *up_scales;
    const void *down_scales;
    float codebook[16];
} moe_q4;

/*
 * LoRA adapters on the experts (moe_forward_lora): rank r in [1, 16], fp32,
 * one (A, B) pair per expert and projection, so that each projection becomes
 *   z = x . W^T + scale * (x . A^T) . B^T,
 * the "fp32 LoRA injection" on top of bf16 or 4-bit expert weights that the
 * unsloth commit page 4f2bfe7f69 names for its rank-16 LoRA runs.
 *   a_gate, a_up [E][r][H]     b_gate, b_up [E][I][r]
 *   a_down       [E][r][I]     b_down       [E][H][r]
 * Device pointers, row-major, 16-byte aligned.
 *
 * packed: NULL, or the output of moe_lora_pack for these adapters and this
 * shape (device, 256-byte aligned).  With a pack, the bf16 tensor-core path runs
 * the adapter products on the tensor cores.  Each fp32 operand (the adapters, and
 * scale * x . A^T) is split as hi = bf16(v), lo = bf16(v - hi), and the products
 * are hi.hi + hi.lo + lo.hi with fp32 accumulation (x is bf16 already, so
 * x . A^T takes x.hi + x.lo): close to fp32 accuracy.  The 4-bit tensor-core
 * path does the same: the A-side products in launches of their own, the B side
 * as one more MMA stage of each tile.  Without a pack, and on every other path,
 * the products run in fp32 on CUDA cores.
 */
typedef struct {
    int32_t rank;
    float scale;   /* lora_alpha / rank */
    const float *a_gate, *b_gate;
    const float *a_up, *b_up;
    const float *a_down, *b_down;
    const void *packed;
} moe_lora;

/*
 * Workspace bytes the entry points below need for this shape (host only, no
 * CUDA call).  The same workspace serves every entry point; it must be
 * 256-byte aligned.  Its first 2048 bytes hold the device error word and
 * scheduling counters and must be zeroed once before first use; the kernels
 * leave the counters at zero again (moe_read_device_error clears the error
 * word).  Returns MOE_ERR_NULLPTR / MOE_ERR_SHAPE / MOE_ERR_DTYPE on bad
 * arguments.
 */
MOE_API int moe_workspace_size(const moe_shape *shape, size_t *bytes);

/*
 * Router GEMM, softmax, top-k and renormalisation (steps A-B).  Defined by
 * the Qwen3-MoE gate whose "router pointwise ops" the unsloth commit page
 * a1bc5cbd73 (compile_walker paragraph) fuses; the tie rule below answers the
 * "tie-break logit boundary" that page 80aaf1121b (flex_moe_parity paragraph)
 * names as its only divergence.
 *   x           [T][H]   act dtype
 *   w_router    [E][H]   act dtype
 *   b_router    [E] fp32 or NULL (added to the logits before softmax/top-k)
 *   expert_ids  [T][k]   int32 out: chosen experts, largest logit first;
 *                         equal fp32 logits: lower expert index first
 *   weights     [T][k]   fp32 out: softmax probabilities of the chosen experts,
 *                         divided by their sum when norm_topk
 *   tie_margin  [T]      fp32 out or NULL: logit of the k-th choice minus the
 *                         (k+1)-th largest logit (+inf when k == E)
 *   logits      [T][E]   fp32 out or NULL: router logits (bias included)
 * Logits accumulate in fp32; softmax is max-subtracted in fp32.
 */
MOE_API int moe_route(const moe_shape *shape, const void *x, const void *w_router, const float *b_router,
              int32_t *expert_ids, float *weights, float *tie_margin, float *logits,
              void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * Expert histogram, exclusive scan and stable permutation (steps C-D): the
 * bincount (capture-safe scatter_add_) + cumsum + argsort of the grouped_mm
 * path on the unsloth commit page 80aaf1121b (grouped_mm paragraph and the
 * closing paragraph on the capture-safe histogram).
 *   expert_ids [A] int32 in
 *   counts     [E] int32 out: assignments per expert
 *   offsets    [E+1] int32 out: offsets[0] = 0, offsets[e+1] = offsets[e] + counts[e]
 *   order      [A] int32 out: order[p] = assignment at permuted row p; rows of
 *              expert e are [offsets[e], offsets[e+1]) in ascending a (stable)
 *   pos        [A] int32 out: inverse of order
 * Integer-exact and deterministic.  An id outside [0, E) sets MOE_ERR_DEVICE.
 */
MOE_API int moe_permute(const moe_shape *shape, const int32_t *expert_ids, int32_t *counts, int32_t *offsets,
                int32_t *order, int32_t *pos, void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * Grouped SwiGLU experts (steps E-F) over the permuted rows: the
 * torch._grouped_mm step of the grouped_mm path on the unsloth commit page
 * 80aaf1121b (grouped_mm paragraph), with the Qwen3-MoE SwiGLU expert MLP.
 * For permuted row
 * p of expert e (offsets[e] <= p < offsets[e+1]) and source token
 * t = order[p] / k:
 *   h = SiLU(x[t] . W_gate[e]^T) * (x[t] . W_up[e]^T),  SiLU(z) = z / (1 + e^-z)
 *   y[p] = h . W_down[e]^T
 *   x       [T][H] act dtype
 *   offsets, order: as produced by moe_permute
 *   w_gate, w_up [E][I][H], w_down [E][H][I]: F32 / BF16 elements, or Q4 codes
 *   q4      scales + codebook when w_dtype == MOE_DT_Q4, else ignored (may be NULL)
 *   y       [A][H] out: fp32 when act dtype is F32, bf16 when BF16
 * Accumulation is fp32; with bf16 activations h is rounded to bf16 before the
 * down projection.
 */
MOE_API int moe_grouped_swiglu(const moe_shape *shape, const void *x, const int32_t *offsets, const int32_t *order,
                       const void *w_gate, const void *w_up, const void *w_down, const moe_q4 *q4,
                       void *y, void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * Weighted un-permute (step G), the index_add_ step of the grouped_mm path on
 * the unsloth commit page 80aaf1121b (grouped_mm paragraph), done as a gather:
 * out[t] = sum_{j<k} weights[t][j] * y[pos[t*k+j]],
 * summed in j order in fp32 and rounded once to the act dtype.  No atomics;
 * bitwise deterministic.
 *   y [A][H] (dtype as produced by moe_grouped_swiglu), weights [T][k] fp32,
 *   pos [A] int32, out [T][H] act dtype.
 */
MOE_API int moe_unpermute(const moe_shape *shape, const void *y, const float *weights, const int32_t *pos,
                  void *out, moe_stream_t stream);

/*
 * The whole block (steps A-G) in one call, intermediates in the workspace: the
 * sparse MoE block that the unsloth commit page 80aaf1121b captures per batch
 * bucket (capture_decode_cudagraph and grouped_mm paragraphs).
 *   out            [T][H] act dtype
 *   expert_ids_out [T][k] int32 or NULL, weights_out [T][k] fp32 or NULL:
 *                  optional copies of the routing decision.
 * Other arguments as in the calls above.
 */
MOE_API int moe_forward(const moe_shape *shape, const void *x, const void *w_router, const float *b_router,
                const void *w_gate, const void *w_up, const void *w_down, const moe_q4 *q4,
                void *out, int32_t *expert_ids_out, float *weights_out,
                void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * The MoE block with the pre-router RMSNorm and the residual add of the Qwen3
 * decoder layer fused in: the "layernorm + residual + router pointwise ops"
 * that the unsloth commit page a1bc5cbd73 (compile_walker paragraph) reports
 * Inductor fusing for about 2x decode throughput.
 *   xn  = RMSNorm(hs) * gamma = (hs / sqrt(mean_h hs^2 + eps)) * gamma, in fp32,
 *         rounded once to the activation dtype; the router and the experts
 *         read xn
 *   out = hs + MoE(xn) when add_residual, else MoE(xn)
 * For T <= 64 the norm runs inside the router launch (the expert-block-0
 * column of the router grid writes xn); larger batches take one extra launch.
 *   hs [T][H], gamma [H]: activation dtype.  eps: finite, >= 0 (else
 *                  MOE_ERR_SHAPE).
 *   x_norm_out     [T][H] activation dtype, or NULL: where xn is written (the
 *                  workspace otherwise).
 * Other arguments, the workspace size and the errors are those of moe_forward.
 */
MOE_API int moe_forward_rmsnorm(const moe_shape *shape, const void *hs, const void *gamma, float eps,
                                int add_residual, const void *w_router, const float *b_router, const void *w_gate,
                                const void *w_up, const void *w_down, const moe_q4 *q4, void *out,
                                void *x_norm_out, int32_t *expert_ids_out, float *weights_out, void *workspace,
                                size_t workspace_bytes, moe_stream_t stream);

/*
 * moe_forward with LoRA adapters on the three expert projections (see
 * moe_lora).  The rank-r products x . A^T and h . A_down^T are computed by
 * separate launches and the B side is added before SiLU (gate/up) and before y
 * is rounded (down): in fp32 on CUDA cores, or, with a pack on the bf16
 * tensor-core path, as tensor-core tiles and one more MMA stage per tile.  Same arguments, results,
 * workspace and errors as moe_forward, plus MOE_ERR_NULLPTR for a NULL lora or
 * adapter pointer and MOE_ERR_SHAPE for a rank outside [1, 16] or a non-finite
 * scale.
 */
MOE_API int moe_forward_lora(const moe_shape *shape, const void *x, const void *w_router, const float *b_router,
                             const void *w_gate, const void *w_up, const void *w_down, const moe_q4 *q4,
                             const moe_lora *lora, void *out, int32_t *expert_ids_out, float *weights_out,
                             void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * Bytes of the adapter pack for this shape (host only, no CUDA call): the four
 * bf16 arrays the tensor-core LoRA path reads, zero-padded, each 256-byte aligned
 * (hi = bf16(v), lo = bf16(v - hi); rank rows or columns past r are zero):
 *   [E][64][H]   A_gate hi, A_up hi, A_gate lo, A_up lo  (16 rows each)
 *   [E][32][I]   A_down hi, A_down lo                    (16 rows each)
 *   [E*I][128]   B_gate then B_up, each as 64 columns (hi, hi, lo, 0) x 16
 *   [E*H][64]    B_down as (hi, hi, lo, 0) x 16 columns
 * With 4-bit weights (shape->w_dtype MOE_DT_Q4) the A columns of every
 * 8-column group are stored in the order (0,4,1,5,2,6,3,7), the order in which
 * the 4-bit path keeps its token rows and h; a pack is therefore specific to the
 * weight type of the shape it was written for.
 */
MOE_API int moe_lora_pack_size(const moe_shape *shape, size_t *bytes);

/*
 * Writes that pack from the fp32 adapters (lora->packed is ignored) into
 * `packed` (device, 256-byte aligned, at least moe_lora_pack_size bytes), on
 * `stream`.  Adapters are static across calls, so a caller packs once and
 * passes the pack in moe_lora.packed; after changing the adapters it packs
 * again.  Errors: MOE_ERR_NULLPTR, MOE_ERR_SHAPE (rank, scale or shape),
 * MOE_ERR_ALIGN, MOE_ERR_WORKSPACE (packed_bytes too small), MOE_ERR_LAUNCH.
 */
MOE_API int moe_lora_pack(const moe_shape *shape, const moe_lora *lora, void *packed, size_t packed_bytes,
                          moe_stream_t stream);

/* Size of the library's fixed device scratch array used by moe_forward_static_scratch. */
#define MOE_STATIC_SCRATCH_BYTES (32u << 20)

/*
 * moe_forward without a caller workspace, for callers that cannot allocate
 * device memory: code running while another thread captures a CUDA graph in
 * global mode (cudaMalloc is illegal then), plugins whose host framework owns
 * the whole device-memory budget, latency-critical paths that cannot afford
 * cudaMalloc's implicit synchronisation.  The pages have no counterpart: this
 * is a deployment convenience, not a step of the method.
 *
 * Same arguments and results as moe_forward, minus the workspace.  The scratch
 * is one fixed MOE_STATIC_SCRATCH_BYTES (32 MiB) array in the library's device
 * image; every GPU that loads the library holds it until the process exits.
 *   - Calls no allocating routine.  The array's module is loaded lazily: the
 *     first call on each device looks up the array's device address (with that
 *     device current), and that lookup is when the driver reserves the 32 MiB
 *     on the device and may synchronise.  Make that first call where a
 *     synchronisation is harmless.
 *   - Shapes whose moe_workspace_size() exceeds 32 MiB are rejected with
 *     MOE_ERR_WORKSPACE before anything is enqueued (the decode shapes fit:
 *     the Qwen3-30B-A3B layer up to a few hundred tokens).  Every other argument
 *     error is also returned before anything is enqueued.
 *   - Every call shares the one array and leaves its contents behind; each call
 *     clears the array's scheduling counters itself.  Calls whose executions
 *     overlap on the GPU (different streams, or concurrent replays) race on the
 *     array: serialise them.
 *   - A device-detected error (MOE_ERR_DEVICE) is recorded in the array's error
 *     word and stays there, across later calls, until
 *     moe_static_scratch_read_error reads and clears it.
 */
MOE_API int moe_forward_static_scratch(const moe_shape *shape, const void *x, const void *w_router,
                                       const float *b_router, const void *w_gate, const void *w_up,
                                       const void *w_down, const moe_q4 *q4, void *out,
                                       int32_t *expert_ids_out, float *weights_out, moe_stream_t stream);

/*
 * moe_read_device_error for the static scratch array of the current device:
 * reads and clears its error word after the work enqueued on `stream`.
 * Synchronises `stream`.  *code receives MOE_OK or MOE_ERR_DEVICE.  Returns
 * MOE_ERR_NULLPTR for a NULL code, MOE_ERR_LAUNCH if the copy failed.
 */
MOE_API int moe_static_scratch_read_error(int32_t *code, moe_stream_t stream);

/*
 * Number of kernel launches one moe_forward call with this shape enqueues
 * (host only, no CUDA call).  Lets callers account for the kernels they run.
 */
MOE_API int moe_forward_launches(const moe_shape *shape, int32_t *launches);

/*
 * Reads and clears the device error word of a workspace.  Synchronises
 * `stream` (use outside graph capture).  *code receives MOE_OK or
 * MOE_ERR_DEVICE.  Returns MOE_OK or MOE_ERR_LAUNCH if the copy failed.
 */
MOE_API int moe_read_device_error(void *workspace, int32_t *code, moe_stream_t stream);

/*
 * Failure-path test hook (process-wide; not for production use).  Every wait
 * inside the tensor-core expert kernels (a pipeline barrier, or a down tile
 * waiting for its expert's h) is bounded: after limit_ns of wall time
 * (default 2e9 = 2 s) it records MOE_ERR_DEVICE in the error word, and the CTA
 * stops starting new work, waits for the copies and MMAs it already issued,
 * frees its tensor memory and exits.  extra_need > 0 raises the count every
 * down tile waits for by that much, so those waits can never be met and must
 * run out: a test sets a short limit and extra_need, checks that the call
 * returns with MOE_ERR_DEVICE recorded, restores (2e9, 0), and checks that the
 * next ordinary call is correct.  Read at each launch; calls already enqueued
 * keep their values.  MOE_ERR_SHAPE for limit_ns == 0 or extra_need < 0.
 */
MOE_API int moe_debug_set_waits(uint64_t limit_ns, int32_t extra_need);

/* ------------------------------------------------------------------------
 * Bucketed CUDA-graph decode (the capture pattern of the unsloth commit page
 * 80aaf1121b, paragraph on FlexMoEInference.capture_decode_cudagraph): one
 * graph of moe_forward per batch-size bucket [1, 2, 4, 8] + 16, 32, ... up to
 * the first multiple of 16 >= max_bs, static input / output buffers and one
 * device arena shared by every bucket.
 *
 * A step with T live tokens replays the smallest bucket B >= T: the static
 * input rows [T, B) are zeroed, the T live rows copied in, the graph replayed
 * and the first T output rows (and expert ids) copied out.  Padded rows are
 * routed like any token and their results discarded, so the live rows equal
 * those of moe_forward on the zero-padded batch of B tokens.
 */
typedef struct moe_graphs moe_graphs;

/*
 * The bucket list for max_bs (host only): writes n <= cap sizes to buckets.
 * MOE_ERR_SHAPE if max_bs is outside [1, 2^18] or the list needs more than cap
 * (or 64) entries.
 */
MOE_API int moe_graph_buckets(int max_bs, int32_t *buckets, int cap, int32_t *n);

/*
 * Device arena bytes a graph set for this shape and max_bs needs (host only):
 * static x, out and expert ids for the largest bucket and one workspace that
 * every bucket's moe_workspace_size() fits in.  shape->T is ignored.
 */
MOE_API int moe_graphs_arena_size(const moe_shape *shape, int max_bs, size_t *bytes);

/*
 * Captures the bucket graphs on `stream` (a non-default stream; thread-local
 * capture mode) after one eager moe_forward per bucket (outside capture).
 * Each bucket gets two graphs: the forward alone, and the forward between a
 * copy-in kernel (the step's rows, then zero padding rows, into the arena) and
 * a copy-out kernel.  Should the second one fail to capture, that bucket's
 * steps take the first route of moe_graphs_run (nothing is reported).
 *   arena          caller-owned device memory of moe_graphs_arena_size() bytes,
 *                  256-byte aligned; the graphs own it until moe_graphs_destroy.
 *   weights, q4    captured by address (their contents may change between
 *                  replays, their addresses may not); the 4-bit codebook values
 *                  are captured by value.
 *   *graphs        receives a host handle (heap memory of the library).
 * Returns MOE_ERR_WORKSPACE if arena_bytes is too small, the moe_forward
 * validation errors for the bucket shapes, MOE_ERR_LAUNCH if a capture or
 * instantiation fails (nothing is kept then).
 */
MOE_API int moe_graphs_create(const moe_shape *shape, int max_bs, const void *w_router, const float *b_router,
                              const void *w_gate, const void *w_up, const void *w_down, const moe_q4 *q4,
                              void *arena, size_t arena_bytes, moe_stream_t stream, moe_graphs **graphs);

/* The bucket a step of T tokens replays (host only); MOE_ERR_SHAPE if none. */
MOE_API int moe_graphs_bucket(const moe_graphs *graphs, int T, int32_t *bucket);

/*
 * One decode step of T tokens (1 <= T <= largest bucket), enqueued on `stream`.
 *   x    [T][H] activations, device or host memory (cudaMemcpyDefault).
 *   out  [T][H] output, device or host memory.
 *   expert_ids_out [T][k] int32 or NULL.
 * When x and out are both device-addressable (device memory, or pinned or
 * registered host memory through its device address) at 16-byte aligned
 * addresses, the step is one launch of the bucket's copy graph, its copy nodes
 * pointed at x and out first; otherwise a zero-fill of the padding rows, a
 * copy of x, the forward graph and a copy of out are enqueued one by one.
 * Both routes give the same bits.  expert_ids_out is copied after either.
 * Steps on different streams must be serialised: the graphs share one arena.
 */
MOE_API int moe_graphs_run(moe_graphs *graphs, int T, const void *x, void *out, int32_t *expert_ids_out,
                           moe_stream_t stream);

/* Frees the graph executables and the handle (not the arena). */
MOE_API int moe_graphs_destroy(moe_graphs *graphs);

/* ------------------------------------------------------------------------
 * The attention half of a decoder layer, for callers that run a whole layer
 * around the MoE block: projections with 4-bit weights, rotary positions with
 * the write into a paged key/value cache, and attention of the new tokens over
 * that cache.  The conventions at the top of this file hold for these calls
 * too (device pointers, 16-byte alignment, host-side validation before any
 * launch, no allocation or synchronisation, graph capturable).
 *
 * A batch is n_seqs sequences.  Sequence b brings a chunk of new tokens, rows
 * [cu_q[b], cu_q[b+1]) of q, k, v and out, and holds kv_len[b] keys, its new
 * tokens' own among them (they are its last ones): new token j of a chunk of n
 * has the place kv_len[b] - n + j in its sequence.  Place p is slot p mod
 * page_size of page block_table[b][p / page_size].  Rows from cu_q[n_seqs] on
 * (padding of a graph's batch) may hold anything and are not written.
 *
 * Sizes: 0 <= n_tokens <= 2^20, 0 <= n_seqs <= 2^16, n_kv_heads divides
 * n_heads <= 1024, head_dim a multiple of 8 up to 256, max_pages * page_size
 * and n_pages below 2^31.  max_q bounds the longest chunk (0 <= max_q <=
 * n_tokens): the host knows it, and the kernel that suits it is chosen from it.
 * dtype: MOE_DT_F32 or MOE_DT_BF16, for q, k, v, out and the cache.
 *
 * Device data is checked on the device: a page number outside [0, n_pages)
 * among those a sequence uses, a chunk longer than max_q, a kv_len outside
 * [0, max_pages * page_size] or a cu_q that falls or leaves [0, n_tokens]
 * records MOE_ERR_DEVICE in the workspace's error word (moe_read_device_error).
 * Nothing outside the arrays is touched then; that sequence's results (with a
 * wrong cu_q, the whole call's) are unspecified.
 */
typedef struct {
    int32_t n_tokens, n_seqs;
    int32_t n_heads, n_kv_heads, head_dim;
    int32_t page_size, n_pages, max_pages;
    int32_t max_q;
    int32_t dtype;
} moe_attn_shape;

/* The sequences of a batch (device arrays): cu_q [n_seqs + 1], kv_len [n_seqs],
 * block_table [n_seqs][max_pages] (entries past a sequence's last page are not
 * read).  These need only their natural 4-byte alignment. */
typedef struct {
    const int32_t *cu_q;
    const int32_t *kv_len;
    const int32_t *block_table;
} moe_attn_batch;

/* The paged cache: slot s of head h of page p starts at element
 * p * page_stride + h * head_stride + s * token_stride of k and of v, head_dim
 * consecutive elements.  Strides are in elements, each a multiple of 16 bytes,
 * so [pages][heads][slots][dim] and [pages][slots][heads][dim] both fit. */
typedef struct {
    void *k, *v;
    int64_t page_stride, head_stride, token_stride;
} moe_kv_cache;

/*
 * Workspace bytes of moe_rope_append and moe_paged_attention for this shape
 * (host only, no CUDA call): 256-byte aligned, its first 2048 bytes (error word
 * and counters) zeroed once before first use.  moe_rope_append needs those 2048
 * bytes only.
 */
MOE_API int moe_attn_workspace_size(const moe_attn_shape *shape, size_t *bytes);

/* Scaling of the rotation rates f_i = base^(-2i / rot_dim) for contexts longer
 * than the trained ones, by `factor`:
 *   LINEAR  f_i / factor
 *   NTK     base * factor^(rot_dim / (rot_dim - 2)) in the place of base
 *   YARN    pairs that turn more than 32 times within trained_len positions keep
 *           f_i, pairs that turn less than once take f_i / factor, the others a
 *           linear ramp over i between; the rotated part is multiplied by
 *           1 + 0.1 ln(factor) */
enum moe_rope_scaling { MOE_ROPE_NONE = 0, MOE_ROPE_LINEAR = 1, MOE_ROPE_NTK = 2, MOE_ROPE_YARN = 3 };

/*
 * The rotation table (host only, no CUDA call): turns[i], i < rot_dim / 2, is
 * the part of a full turn that pair i advances by each position, in units of
 * 2^-64 turn, and *mscale the factor on the rotated part.  The kernel multiplies
 * turns[i] by the position modulo 2^64, so that the angle's fraction of a turn
 * is as exact at position 10^6 as at 1.  Copy turns to the device once.
 * rot_dim: a multiple of 16 up to 256.  base > 1, factor >= 1 and, for YARN,
 * trained_len > 0, else MOE_ERR_SHAPE.
 */
MOE_API int moe_rope_turns(int32_t rot_dim, int32_t scaling, double base, double factor, int32_t trained_len,
                           uint64_t *turns, float *mscale);

/*
 * Rotary positions: the first rot_dim elements of a head (a multiple of 16, at
 * most head_dim) are rotated in pairs, the others pass through.  Pair i is
 * elements (2i, 2i+1) when interleaved, else (i, i + rot_dim/2):
 *   (a, b) -> mscale * (a cos t - b sin t, b cos t + a sin t), t = position * f_i
 * turns: DEVICE copy of moe_rope_turns' table.  q_gamma / k_gamma: NULL, or the
 * weights [head_dim] (dtype of the shape) of an RMS norm of each q / k head
 * before the rotation: x / sqrt(mean x^2 + eps) * gamma.
 */
typedef struct {
    int32_t rot_dim;
    int32_t interleaved;
    float mscale;
    float eps;
    const uint64_t *turns;
    const void *q_gamma, *k_gamma;
} moe_rope;

/*
 * Normalises (if asked), rotates and stores the new tokens: q_out = rotated q,
 * the rotated k and the plain v go to the cache slots of the tokens' places.
 * Computed in fp32, rounded once.
 *   q [n_tokens][n_heads][head_dim], k, v [n_tokens][n_kv_heads][head_dim]:
 *     token rows q_stride / k_stride / v_stride elements apart (multiples of 16
 *     bytes below 2^31 elements: slices of one projection's output), heads
 *     contiguous in a row
 *   positions [n_tokens] int32 or NULL: the position of each token's rotation
 *     (NULL: its place in the sequence)
 *   q_out [n_tokens][n_heads][head_dim], rows q_out_stride apart; may be q itself
 * A token whose place is negative (kv_len shorter than the chunk) is rotated but
 * not stored.
 */
MOE_API int moe_rope_append(const moe_attn_shape *shape, const moe_rope *rope, const void *q, int64_t q_stride,
                            const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                            const moe_kv_cache *cache, const moe_attn_batch *batch, const int32_t *positions,
                            void *q_out, int64_t q_out_stride, void *workspace, size_t workspace_bytes,
                            moe_stream_t stream);

/*
 * Attention of the new tokens over the cache, causal, with grouped heads (query
 * head i reads key head i / (n_heads / n_kv_heads)): new token j of a chunk of n
 * sees the keys at places 0 .. kv_len - n + j,
 *   out = sum_p softmax_p(scale * q . k_p) v_p.
 * A token that sees no key gets out = 0 and lse = -inf.  Slots at or past kv_len
 * may hold anything (NaN included); a k that is not finite reaches the tokens that
 * see it, a v also those of the same chunk before it (as 0 * NaN in the formula).  Scores, the softmax's maximum and sum and
 * the output accumulate in fp32; with bf16 the probabilities are rounded to bf16
 * for the product with v.  Results do not depend on timing (bitwise
 * deterministic).
 *   q, out [n_tokens][n_heads][head_dim], token rows q_stride / out_stride
 *     elements apart (multiples of 16 bytes below 2^31 elements)
 *   lse [n_tokens][n_heads] fp32 or NULL: natural log of the sum of
 *     exp(scale * q . k_p)
 *   scale: finite, else MOE_ERR_SHAPE
 */
MOE_API int moe_paged_attention(const moe_attn_shape *shape, const void *q, int64_t q_stride,
                                const moe_kv_cache *cache, const moe_attn_batch *batch, float scale, void *out,
                                int64_t out_stride, float *lse, void *workspace, size_t workspace_bytes,
                                moe_stream_t stream);

/* Sizes of moe_q4_linear: T rows of x, K inputs, N outputs; 0 <= T <= 2^18,
 * K a multiple of 8, N >= 1, K and N at most 2^22, q_block even and dividing K.
 * x and the residual are bf16; out_dtype MOE_DT_BF16 or MOE_DT_F32. */
typedef struct {
    int32_t T, K, N;
    int32_t out_dtype;
    int32_t q_block;
} moe_q4_linear_shape;

/* One weight matrix [N][K] in the 4-bit format of moe_q4: codes [N][K/2] bytes,
 * scales [N][K/q_block] bf16 (device), the codebook by value. */
typedef struct {
    const void *codes;
    const void *scales;
    float codebook[16];
} moe_q4_weight;

/*
 * out = x . W^T (+ residual) with a 4-bit W, for decode batches.  A pass over the
 * weights takes 16, 32 or 64 rows with a uniform codebook, q_block of 64 and up and
 * large weights, else 8 or 16, and 8 where q_block is neither 32 nor 64 times a power
 * of two; more rows repeat it.
 *   out[t][n] = sum_k codebook[code[n][k]] * scale[n][k / q_block] * x[t][k]
 *               (+ residual[t][n]),
 * accumulated in fp32, rounded once.  The codebook's values are kept to 24 bits for
 * fp32 results and to 16 (2^-17 of a value) for bf16 ones; a codebook within 2^-20
 * (fp32) or 2^-17 (bf16) of each value from a uniform one is taken as uniform.
 * q_block that is neither 32 nor 64 times a power of two keeps the fp32 values.
 * Infinite, NaN and very large x give what the formula gives (a row of x that holds
 * an infinity, or a value past 2^116, takes many times as long).
 *   x [T][K] bf16, rows x_stride elements apart (a multiple of 8)
 *   residual [T][N] bf16, rows residual_stride apart, or NULL; out [T][N], rows
 *     out_stride apart (any stride >= N); residual may be out itself
 */
MOE_API int moe_q4_linear(const moe_q4_linear_shape *shape, const void *x, int64_t x_stride,
                          const moe_q4_weight *weight, const void *residual, int64_t residual_stride, void *out,
                          int64_t out_stride, moe_stream_t stream);

/*
 * Reads and clears the error word of moe_q4_linear on the current device
 * (MOE_ERR_DEVICE if a bounded wait of its tensor-core kernel ran out, which no
 * healthy call does; that call's results are unspecified).  The call has no
 * workspace: the word is one for all its calls on the device, whatever their
 * stream, so whoever reads it learns of (and clears) the errors of every stream's
 * calls that have ended.  Synchronises `stream`.  Returns MOE_ERR_NULLPTR for a
 * NULL code, MOE_ERR_LAUNCH if the copy failed.
 */
MOE_API int moe_q4_linear_read_error(int32_t *code, moe_stream_t stream);

/* Static, human-readable name of a status code. */
MOE_API const char *moe_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
