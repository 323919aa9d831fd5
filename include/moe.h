/*
 * moe.h -- C ABI of libmoe_gb300.so: the single-GPU forward of one
 * Mixture-of-Experts FFN layer on GB300 (sm_103a), and (at the end) the
 * operators that train its routed experts in 8 bits, run them in 4 bits and
 * move tokens with gradients.
 *
 * The layer, as the page "MOE推理流程解析" (ffner.com) lays it out:
 *   section 三: the router scores every eligible expert; top-k keeps the
 *     chosen experts' indices and weights; a permutation reads the token
 *     vectors, writes them in expert order and records an inverse map; a
 *     grouped GEMM runs all expert matrices (of different row counts) in
 *     one launch; each expert applies its activation and output projection;
 *     the inverse map restores token order, the routing weight is applied
 *     and the contributions of the same token are summed.
 *   section 二: assignments (token vector, expert, weight) are grouped by
 *     expert into contiguous matrices, each row keeping its source token id;
 *     an expert batch counts assignments, not unique tokens (top-2 gives two
 *     rows per token).
 *   section 一: shared experts process every token whatever the router
 *     scores.
 * Precision ("MoE 推理部署", zzmblog.top, section 专家量化): quantisation
 * scales are per expert; the router and shared experts stay at higher
 * precision than quantised routed experts.
 *
 * Conventions (all entry points)
 *   - Every pointer named as a tensor is a DEVICE pointer of the current CUDA
 *     device, row-major, densely packed, 16-byte aligned.  The caller owns
 *     every buffer and the stream; the library allocates no device memory.
 *   - Weights are [out, in] (the reduction index is contiguous):
 *       w_router [E, d]; w_gate, w_up [E, ffn, d]; w_down [E, d, ffn];
 *       shared expert: w_shared_gate, w_shared_up [ffn_shared, d],
 *       w_shared_down [d, ffn_shared].
 *   - Experts are numbered from 0.  R = T * k assignment rows.
 *   - Calls are asynchronous on `stream` (NULL = the legacy default stream).
 *     Argument errors are detected on the host and returned before anything
 *     is enqueued; launch failures return MOE_ERR_CUDA.  Errors found by a
 *     kernel (an expired bounded wait, an out-of-range index) are recorded in
 *     a per-device status word read by moe_read_device_status().
 *   - Unsupported combinations of sizes or dtypes return MOE_ERR_UNSUPPORTED;
 *     there is no fallback path.
 *   - T == 0 is valid: nothing is enqueued and MOE_OK is returned.
 *
 * Supported storage:  act_dtype / w_dtype
 *   MOE_F32  / MOE_F32          fp32 CUDA-core path (fp32 accumulation)
 *   MOE_BF16 / MOE_BF16         tcgen05 tensor-core path (fp32 accumulation)
 *   MOE_BF16 / MOE_FP8_E4M3     as above, FP8 weights (OCP E4M3) with fp32
 *                               per-expert, per-output-channel scales;
 *                               the router and shared expert stay bf16.
 *                               The bf16 rows (tokens, then h) enter the
 *                               FP8 x FP8 tensor-core instructions as two
 *                               E4M3 rows each (moe_split_rows_e4m3x2),
 *                               the bf16 values themselves for elements
 *                               within 2^9 of their row's maximum:
 *                               g[r,o] = s_gate[e,o] * s_x[r] *
 *                                 sum_i (hi[r,i] + lo[r,i]) code_gate[e][o,i]
 *                               (likewise u); h = SiLU(g) * u held in bf16,
 *                               split the same way before the down product.
 *                               Any finite bf16 magnitude is accepted.
 *   MOE_BF16 / MOE_FP8_E4M3_ACT8
 *                               FP8 weights as above; both routed GEMMs
 *                               multiply them with E4M3 activation rows
 *                               (per-row scales, moe_quantize_rows_e4m3):
 *                               g[r,o] = s_x[r] * s_gate[e,o] *
 *                                        sum_i q_x[r,i] * code_gate[e][o,i]
 *                               (likewise u), h = SiLU(g) * u held in f16
 *                               and quantised per row the same way, then
 *                               y[r,o] = s_h[r] * s_down[e,o] *
 *                                        sum_j q_h[r,j] * code_down[e][o,j].
 *                               Router and shared expert stay bf16.
 *   MOE_BF16 / MOE_MXFP4        OCP Microscaling FP4 weights ("MoE 推理部署",
 *                               section 专家量化: MXFP4 block-scaled 4-bit
 *                               experts): W[o,i] = E2M1(code[o,i]) *
 *                               2^(s[i/32,o] - 127).  w_gate / w_up
 *                               [E, ffn, d/2] and w_down [E, d, ffn/2] bytes,
 *                               two codes per byte (element 2i in the low
 *                               nibble of byte i); s_gate / s_up [E, d/32,
 *                               ffn] and s_down [E, ffn/32, d] UE8M0 bytes,
 *                               reduction-block-major (a k-block's scales of
 *                               all output channels contiguous), passed
 *                               through the float* scale parameters.  The
 *                               kernels convert to f16 operands, exactly for
 *                               block scales 2^-23 .. 2^13 (UE8M0 104..140);
 *                               larger scales overflow f16 and are not
 *                               supported.  Router and shared expert bf16.
 * Size limits: 1 <= k <= min(E, 32), E <= 1024, T * k <= 2^24,
 * d % 8 == 0, ffn % 8 == 0; the tensor-core path further needs
 * d % 128 == 0, ffn % 128 == 0 and ffn_shared % 128 == 0.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ABI_VERSION 5

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

/* A cudaStream_t. */
typedef struct CUstream_st *moe_stream_t;

typedef enum moe_dtype {
  MOE_F32 = 0,
  MOE_BF16 = 1,
  MOE_FP8_E4M3 = 2,
  /* w_dtype only: FP8 weights as MOE_FP8_E4M3, and both routed expert
   * products take activations quantised per row to E4M3
   * (moe_quantize_rows_e4m3) on FP8 x FP8 tensor-core instructions */
  MOE_FP8_E4M3_ACT8 = 3,
  /* w_dtype only: OCP MXFP4 routed expert weights (see "Supported storage") */
  MOE_MXFP4 = 4
} moe_dtype;

typedef enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1,    /* null pointer, bad size, k > E, ...        */
  MOE_ERR_UNSUPPORTED = -2,    /* valid but not implemented combination     */
  MOE_ERR_WORKSPACE = -3,      /* workspace missing or too small            */
  MOE_ERR_CUDA = -4,           /* a CUDA runtime / driver call failed       */
  MOE_ERR_DEVICE_TIMEOUT = -5, /* a kernel's bounded wait expired           */
  MOE_ERR_DEVICE_BOUNDS = -6   /* a kernel met an out-of-range index/offset */
} moe_status;

/* The problem statement shared by every entry point. */
typedef struct moe_problem {
  int32_t T;          /* tokens in the batch                                */
  int32_t d;          /* hidden size                                        */
  int32_t ffn;        /* routed expert intermediate size                    */
  int32_t E;          /* routed experts                                     */
  int32_t k;          /* experts chosen per token                           */
  int32_t ffn_shared; /* shared expert intermediate size; 0 = none          */
  int32_t act_dtype;  /* moe_dtype of x, w_router, shared expert, outputs   */
  int32_t w_dtype;    /* moe_dtype of the routed expert weights             */
} moe_problem;

/*
 * moe_router_topk -- router scores, softmax, top-k, renormalised weights.
 * Page "MOE推理流程解析", section 三 (the router scores each eligible expert;
 * top-k keeps the chosen indices and weights) and section 九 (the kept
 * weights are re-normalised).
 *
 *   l[t,e]   = sum_i x[t,i] * w_router[e,i] (+ router_bias[e]), fp32 accumulate
 *   p        = softmax(l[t,:]) over all E experts
 *   S_t      = the k experts with the largest l (ties: lower expert index)
 *   w[t,j]   = p[S_t,j] / sum_{e in S_t} p[e]   (== softmax over S_t only)
 * Slots j are in descending weight.  Non-finite logits: infinities order as
 * numbers, -0 ties +0, and NaN logits rank after every number (among
 * themselves by expert index).
 *
 *   x            [T, d] act_dtype
 *   w_router     [E, d] act_dtype
 *   router_bias  [E] fp32 or NULL
 *   logits_in    [T, E] fp32 or NULL: when given, used as l directly (no
 *                matmul; router_bias must then be NULL; x, w_router unused)
 *   logits_out   [T, E] fp32 or NULL: receives l (including the bias)
 *   topk_idx     [T, k] int32 out      topk_w  [T, k] fp32 out
 */
MOE_API moe_status moe_router_topk(const moe_problem *p, const void *x, const void *w_router,
                           const float *router_bias, const float *logits_in,
                           float *logits_out, int32_t *topk_idx, float *topk_w,
                           moe_stream_t stream);

/*
 * moe_permute -- group the T*k assignments by expert and move token rows.
 * Page "MOE推理流程解析", section 二 (grouping by expert into contiguous
 * matrices, the source token id kept beside each row) and section 三 (the
 * permutation writes token vectors in expert order and records an inverse
 * map for the combine).
 *
 *   counts[e]       = #{(t,j) : topk_idx[t,j] == e}                [E] int32 out
 *   offsets[e]      = sum_{e'<e} counts[e'], offsets[E] = T*k     [E+1] int32 out
 *   perm_token[r]   = source token of row r                       [T*k] int32 out
 *   inv_row[t*k+j]  = row holding assignment (t, j)               [T*k] int32 out
 *   x_perm[r, :]    = x[perm_token[r], :]      [T*k, d] act_dtype out, or NULL
 * Rows inside an expert's range are in ascending token order (deterministic,
 * bit-exact).  x may be NULL only when x_perm is NULL.  topk_idx entries
 * outside [0, E) are skipped and flag MOE_ERR_DEVICE_BOUNDS.
 * workspace: at least moe_workspace_size() bytes, device memory.
 */
MOE_API moe_status moe_permute(const moe_problem *p, const int32_t *topk_idx, const void *x,
                       int32_t *counts, int32_t *offsets, int32_t *perm_token,
                       int32_t *inv_row, void *x_perm, void *workspace,
                       size_t workspace_bytes, moe_stream_t stream);

/*
 * moe_permute_static_scratch -- moe_permute without a workspace argument.
 * No counterpart on the pages: it exists for callers that cannot allocate
 * device memory -- code hosted by another framework whose memory manager
 * must own every allocation, or latency-critical loops that cannot afford a
 * cudaMalloc (which may synchronise the device).  Arguments and results are
 * those of moe_permute; the caller still passes every input and output.
 *
 * The scratch moe_permute takes from the workspace (per-chunk expert counts,
 * ceil(T*k/256) * E int32 values) lives instead in a 1 MiB array compiled
 * into the library and held by every GPU that loads it until the process
 * exits.  Problems needing more (ceil(T*k/256) * E > 262144) are rejected
 * with MOE_ERR_WORKSPACE.  The first call on each device looks up the
 * array's device address with that device current; make that first call
 * before any stream capture.  That cached address (like the library's other
 * per-device state) does not survive a device reset (cudaDeviceReset) in
 * the same process.  The problem is checked exactly as moe_permute checks
 * it, then against the array's size.  All calls share the array and it keeps the
 * last call's contents (every entry read is first rewritten, so nothing has
 * to be cleared); calls that overlap on the GPU race on it.  Allocates
 * nothing.
 */
MOE_API moe_status moe_permute_static_scratch(const moe_problem *p, const int32_t *topk_idx,
                                              const void *x, int32_t *counts, int32_t *offsets,
                                              int32_t *perm_token, int32_t *inv_row,
                                              void *x_perm, moe_stream_t stream);

/*
 * moe_grouped_swiglu -- all expert matrices in one grouped computation.
 * Page "MOE推理流程解析", section 三 (a grouped GEMM runs several expert
 * matrices with different row counts in one launch; each expert applies its
 * activation and output projection) and section 二 (variable-row expert
 * matrices, no padding in the result).
 *
 * For every expert e and every row r in [offsets[e], offsets[e+1]):
 *   h[r,:]      = SiLU(x_perm[r,:] W_g[e]^T) * (x_perm[r,:] W_u[e]^T)
 *   y_perm[r,:] = h[r,:] W_d[e]^T
 * with FP8 weights W[e][o,:] = code[e][o,:] * scale[e][o] (s_gate, s_up
 * [E, ffn]; s_down [E, d]; NULL unless the weights are quantised: FP8, or
 * MXFP4 with the block-scale arrays described above).  With
 * MOE_FP8_E4M3_ACT8 the rows of x_perm and of h enter their products
 * quantised per row (moe_quantize_rows_e4m3, into the workspace).
 *
 *   x_perm   [T*k, d] act_dtype      offsets [E+1] int32 (device)
 *   y_perm   [T*k, d] act_dtype out
 * h is kept in workspace in act_dtype (bf16 for the tensor-core path).
 * Offsets must be non-decreasing with offsets[E] <= T*k; rows outside every
 * expert's range are left untouched.
 */
MOE_API moe_status moe_grouped_swiglu(const moe_problem *p, const void *x_perm, const int32_t *offsets,
                              const void *w_gate, const void *w_up, const void *w_down,
                              const float *s_gate, const float *s_up, const float *s_down,
                              void *y_perm, void *workspace, size_t workspace_bytes,
                              moe_stream_t stream);

/*
 * moe_quantize_rows_e4m3 -- per-row FP8 quantisation of activation rows.
 * Page "MOE推理流程解析", section 三 (activations may be quantised before
 * dispatch, so that the permuted rows move fewer bytes, or dispatched at
 * higher precision and quantised just before the experts) and page
 * "MoE 推理部署", section 专家量化 (FP8 inference).  The layer forward with
 * w_dtype MOE_FP8_E4M3_ACT8 quantises x before dispatch with this
 * operation, moe_grouped_swiglu quantises x_perm (after dispatch), and both
 * quantise the rows of h (held in f16) before the down product.
 *
 *   s[r]      = max_i |x[r,i]| / 448, or 1 when row r is all zero
 *   code[r,i] = E4M3(x[r,i] / s[r]): nearest E4M3 value, ties to the even
 *               code, magnitudes above 448 saturated to 448, sign kept
 *               (-0 -> 0x80)
 * Both divisions are correctly rounded fp32 operations, so the codes and
 * scales are exact functions of the inputs (bit-reproducible).
 *
 *   x       [rows, cols] bf16, device, 16-byte aligned
 *   codes   [rows, cols] uint8 out (OCP E4M3 bit patterns), 16-byte aligned
 *   scales  [rows] fp32 out
 * rows >= 0 (0: nothing is enqueued); cols > 0 and cols % 8 == 0, else
 * MOE_ERR_UNSUPPORTED.  Null pointers with rows > 0: MOE_ERR_INVALID_ARG.
 */
MOE_API moe_status moe_quantize_rows_e4m3(int32_t rows, int32_t cols, const void *x, uint8_t *codes,
                                          float *scales, moe_stream_t stream);

/*
 * moe_split_rows_e4m3x2 -- bf16 rows as two E4M3 rows each, exactly.
 * Page "MoE 推理部署", section 专家量化 (FP8 expert weights, the
 * activations kept at higher precision): the FP8-weight mode
 * (MOE_FP8_E4M3) multiplies its E4M3 weights with bf16 activation rows on
 * FP8 x FP8 tensor-core instructions by handing them each row in this
 * form; the layer forward applies it to x (before dispatch) and to h.
 *
 *   s[r]         = 2^p, p the integer with max_i |x[r,i]| / 2^p in
 *                  (224, 448]; 1 when row r is all zero
 *   hi[r,i]      = E4M3(x[r,i] / s[r])
 *   lo[r,i]      = E4M3(x[r,i] / s[r] - hi[r,i])
 * (nearest E4M3 value, ties to the even code).  Then
 *   x[r,i] = s[r] * (hi[r,i] + lo[r,i])
 * exactly for every element with |x[r,i]| >= max_i |x[r,i]| * 2^-9, and
 * within s[r] * 2^-10 for smaller ones: a bf16 value has 8 significant
 * bits, hi holds the top four (rounded) and lo the signed remainder, which
 * E4M3 holds exactly down to its smallest step.  An FP8 x FP8 product on
 * hi plus one on lo, accumulated together, multiplies by the bf16 row.
 *
 *   x       [rows, cols] bf16, device, 16-byte aligned
 *   codes   [2, rows, cols] uint8 out: every row's hi codes, then every
 *           row's lo codes (row r's lo codes are row rows + r of a
 *           [2*rows, cols] matrix), 16-byte aligned
 *   scales  [rows] fp32 out (powers of two)
 * rows >= 0 (0: nothing is enqueued); cols > 0 and cols % 8 == 0, else
 * MOE_ERR_UNSUPPORTED.  Null pointers with rows > 0: MOE_ERR_INVALID_ARG.
 */
MOE_API moe_status moe_split_rows_e4m3x2(int32_t rows, int32_t cols, const void *x, uint8_t *codes,
                                         float *scales, moe_stream_t stream);

/*
 * moe_combine -- restore token order, apply routing weights, sum.
 * Page "MOE推理流程解析", section 三 (the inverse map restores token order,
 * the routing weight is applied, contributions with the same token id are
 * summed) and section 二 (T1's output is 0.7 * E1(T1) + 0.3 * E3(T1)).
 *
 *   out[t,:] = sum_{j<k} topk_w[t,j] * y_perm[inv_row[t*k+j], :] (+ shared_out[t,:])
 * accumulated in fp32 in slot order j = 0..k-1, rounded once to act_dtype.
 *   y_perm [T*k, d]  inv_row [T*k] int32  topk_w [T, k] fp32
 *   shared_out [T, d] act_dtype or NULL      out [T, d] act_dtype
 */
MOE_API moe_status moe_combine(const moe_problem *p, const void *y_perm, const int32_t *inv_row,
                       const float *topk_w, const void *shared_out, void *out,
                       moe_stream_t stream);

/*
 * moe_layer_forward -- the whole layer: router top-k, permutation, grouped
 * SwiGLU experts, optional shared expert, combine (page "MOE推理流程解析",
 * sections 一, 二, 三; section 十一 lists the step: routing, token
 * permutation, grouped expert compute, combine, unpermutation).
 *
 *   out[t,:] = sum_{e in S_t} w[t,e] * FFN_e(x[t,:]) + FFN_shared(x[t,:])
 *
 * Shared expert weights are all NULL when p->ffn_shared == 0, all non-NULL
 * otherwise.  topk_idx_out [T,k], topk_w_out [T,k] and counts_out [E] are
 * optional copies of the routing decision (NULL = not wanted).
 * The whole sequence is enqueued on `stream` without any host
 * synchronisation, so it can be captured into a CUDA graph by the caller.
 */
MOE_API moe_status moe_layer_forward(const moe_problem *p, const void *x, const void *w_router,
                             const float *router_bias, const void *w_gate, const void *w_up,
                             const void *w_down, const float *s_gate, const float *s_up,
                             const float *s_down, const void *w_shared_gate,
                             const void *w_shared_up, const void *w_shared_down, void *out,
                             int32_t *topk_idx_out, float *topk_w_out, int32_t *counts_out,
                             void *workspace, size_t workspace_bytes, moe_stream_t stream);

/*
 * Per-stage timing of the layer forward (page "MOE推理流程解析", section 三:
 * measure routing, permutation, expert GEMM and combine separately; one
 * merged MoE timer cannot say which stage is slow).
 *
 * A stage timer holds CUDA events for one call of moe_layer_forward_timed();
 * reading it waits for that call's last event.  Stage indices:
 */
enum {
  MOE_STAGE_ROUTER = 0,   /* logits, softmax, top-k                        */
  MOE_STAGE_PERMUTE = 1,  /* counts, offsets, maps, row moves              */
  MOE_STAGE_GATE_UP = 2,  /* grouped gate/up GEMM + SiLU*mul               */
  MOE_STAGE_DOWN = 3,     /* grouped down GEMM                             */
  MOE_STAGE_SHARED = 4,   /* shared expert (0 when absent)                 */
  MOE_STAGE_COMBINE = 5,  /* unpermute, weights, sum                       */
  MOE_NUM_STAGES = 6
};
typedef struct moe_stage_timer moe_stage_timer;

/* Create / destroy a timer (host object owning CUDA events; no device memory). */
MOE_API moe_status moe_stage_timer_create(moe_stage_timer **timer);
MOE_API moe_status moe_stage_timer_destroy(moe_stage_timer *timer);
/* Wait for the timed call to finish; ms[MOE_NUM_STAGES] receives each stage's
 * device time in milliseconds. */
MOE_API moe_status moe_stage_timer_read(moe_stage_timer *timer, float *ms);

/* moe_layer_forward with CUDA events recorded on `stream` between stages. */
MOE_API moe_status moe_layer_forward_timed(
    const moe_problem *p, const void *x, const void *w_router, const float *router_bias,
    const void *w_gate, const void *w_up, const void *w_down, const float *s_gate,
    const float *s_up, const float *s_down, const void *w_shared_gate, const void *w_shared_up,
    const void *w_shared_down, void *out, int32_t *topk_idx_out, float *topk_w_out,
    int32_t *counts_out, void *workspace, size_t workspace_bytes, moe_stream_t stream,
    moe_stage_timer *timer);

/* Number of kernels one moe_layer_forward() call launches for problem *p on
 * the current device (written to *launches). */
MOE_API moe_status moe_layer_launch_count(const moe_problem *p, int32_t *launches);

/*
 * moe_plan_info -- the tiling the library chose for problem *p on the
 * current device (no page counterpart; for benchmarks and tests):
 * info[0] rows per tile of the gate/up GEMM, info[1] rows per tile of the
 * down GEMM, info[2] reduction splits of the down GEMM, info[3] persistent
 * CTAs per GEMM launch, info[4] reduction splits of the gate/up GEMM,
 * info[5] bit 0 / bit 1: the gate/up / down GEMM runs on CTA pairs
 * (256 output channels per tile).  `info` holds 6 entries.  All zero for
 * the fp32 CUDA-core path.
 */
MOE_API moe_status moe_plan_info(const moe_problem *p, int32_t *info);

/*
 * moe_plan_info_for, moe_layer_launch_count_for, moe_workspace_size_for --
 * the same answers as moe_plan_info, moe_layer_launch_count and
 * moe_workspace_size for a device with `num_sms` multiprocessors, computed
 * on the host alone: they touch no device and need none (planning ahead of
 * time, and tests of the tiling rules on machines without a GPU).  The
 * device entry points are these with the current device's SM count.
 * Returns MOE_ERR_INVALID_ARG for a null output or num_sms outside
 * [1, 4096], and MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED for problems the
 * library rejects.
 */
MOE_API moe_status moe_plan_info_for(const moe_problem *p, int32_t num_sms, int32_t *info);
MOE_API moe_status moe_layer_launch_count_for(const moe_problem *p, int32_t num_sms, int32_t *launches);
MOE_API moe_status moe_workspace_size_for(const moe_problem *p, int32_t num_sms, size_t *bytes);

/*
 * moe_workspace_size -- device workspace (bytes) sufficient for every entry
 * point above with problem *p on the current device.  Returns
 * MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED for problems the library rejects.
 */
MOE_API moe_status moe_workspace_size(const moe_problem *p, size_t *bytes);

/*
 * moe_read_device_status -- synchronise `stream`, then read and clear the
 * current device's kernel status word.  *status receives MOE_OK or the first
 * error a kernel recorded since the last read (MOE_ERR_DEVICE_TIMEOUT,
 * MOE_ERR_DEVICE_BOUNDS).  Returns MOE_ERR_CUDA if synchronisation fails.
 */
MOE_API moe_status moe_read_device_status(moe_stream_t stream, int32_t *status);

/* Human-readable name of a status code (static storage). */
MOE_API const char *moe_status_string(int32_t status);

/* The last CUDA error text recorded by a call that returned MOE_ERR_CUDA on
 * this host thread (static thread-local storage; "" if none). */
MOE_API const char *moe_last_cuda_error(void);

/* MOE_ABI_VERSION of the loaded library. */
MOE_API int32_t moe_abi_version(void);

/*
 * moe_selftest_bounded_wait -- failure-detection self test (no page
 * counterpart).  Launches the tensor-core kernel's wait machinery on a
 * barrier that nothing arrives at, with a wait limit of timeout_ns
 * nanoseconds.  No copy or MMA is issued, so the wait expiring leaves no
 * work in flight; the kernel records MOE_ERR_DEVICE_TIMEOUT in the status
 * word, frees its tensor memory and returns.  Read the outcome with
 * moe_read_device_status().
 */
MOE_API moe_status moe_selftest_bounded_wait(int64_t timeout_ns, moe_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Training the routed experts in 8 bits.  No page counterpart: the pages
 * describe inference; these entry points are the products, checkpoints and
 * gradients that fine-tuning the same layer needs next to it.
 *
 * Rows are grouped by expert as moe_permute leaves them: rows
 * offsets[e] .. offsets[e+1] - 1 belong to expert e, offsets [E+1] int32 on
 * the device.  Offsets outside [0, R], or decreasing ones, are clamped and
 * flag MOE_ERR_DEVICE_BOUNDS.  A block is 128 consecutive columns of a row
 * (rows x: one fp32 scale per block, scales [rows, ceil(cols/128)]) or 128 x
 * 128 of a weight matrix; the last block of a row or matrix may be shorter.
 * Limits: E <= 1024, R <= 2^24.
 * ---------------------------------------------------------------------------
 */
typedef enum moe_scale_kind {
  MOE_SCALE_AMAX = 0, /* s = a / 448, correctly rounded                       */
  MOE_SCALE_POW2 = 1  /* s = 2^p with a / 2^p in (224, 448]                   */
} moe_scale_kind;

/*
 * moe_quantize_blocks_e4m3 -- rows as E4M3 codes with a scale per block.
 *
 *   a         = largest finite |x| of the block, at least 2^-100
 *               (s = 1 when every finite value of the block is zero)
 *   code[r,i] = E4M3(x[r,i] * t): nearest E4M3 value, ties to the even code;
 *               t = 448 / a correctly rounded (MOE_SCALE_AMAX), t = 1 / s
 *               exactly (MOE_SCALE_POW2)
 * Infinities and NaN become the NaN code and do not enter the scale.  Codes
 * and scales are exact functions of the inputs (bit-reproducible).  With
 * MOE_SCALE_POW2 code * s is exactly a bf16 value: the form to keep rows in
 * for moe_grouped_wgrad.
 *
 *   x       [rows, cols] x_dtype (MOE_BF16 or MOE_F32), row pitch ld_x
 *           elements (>= cols; rows 16-byte aligned)
 *   codes   [rows, cols] uint8 out      scales [rows, ceil(cols/128)] fp32 out
 * cols % 8 == 0, else MOE_ERR_UNSUPPORTED.  rows == 0: nothing is enqueued.
 */
MOE_API moe_status moe_quantize_blocks_e4m3(int32_t rows, int32_t cols, int32_t x_dtype, int32_t scale_kind,
                                            const void *x, int64_t ld_x, uint8_t *codes, float *scales,
                                            moe_stream_t stream);

/*
 * moe_grouped_block_gemm -- E4M3 rows times E4M3 weights, both with scales
 * per block of 128 along the reduction.  For every row r of expert e:
 *
 *   out[r,n] = sum_kb a_scales[r,kb] * w_scales[e,n/128,kb] *
 *              sum_{i in block kb} a[r,i] * w[e,n,i]
 *
 * products exact, sums and scales in fp32, rounded once to out_dtype.
 *   a_codes [R, K]   a_scales [R, ceil(K/128)]
 *   transposed == 0: w_codes [E, N, K], w_scales [E, ceil(N/128), ceil(K/128)]
 *   transposed != 0: w_codes [E, K, N], w_scales [E, ceil(K/128), ceil(N/128)]
 *     -- the data gradient of the product above on the same arrays: call with
 *     K the forward's output channels and N its input channels
 *   out [R, N] MOE_BF16 or MOE_F32
 * Any fp32 scales are accepted.  K % 16 == 0 and N % 16 == 0, else
 * MOE_ERR_UNSUPPORTED.  Rows outside every expert's range are left untouched;
 * R == 0: nothing is enqueued.
 */
MOE_API moe_status moe_grouped_block_gemm(int32_t R, int32_t K, int32_t N, int32_t E, int32_t transposed,
                                          int32_t out_dtype, const uint8_t *a_codes, const float *a_scales,
                                          const int32_t *offsets, const uint8_t *w_codes,
                                          const float *w_scales, void *out, moe_stream_t stream);

/*
 * moe_swiglu_save_e4m3 -- h = SiLU(g) * u, keeping g and u in 8 bits.
 *
 *   g, u          [R, ffn] bf16, row pitch ld elements each (the halves of one
 *                 [R, 2 ffn] product: u = g + ffn, ld = 2 ffn)
 *   h             [R, ffn] bf16 out, or NULL
 *   h_codes       [R, ffn], h_scales [R, ceil(ffn/128)] out, or both NULL: h
 *                 in blocks with MOE_SCALE_AMAX, from h in fp32
 *   saved_codes   [2, R, ffn], saved_scales [2, R, ceil(ffn/128)] out: g, then
 *                 u, as moe_quantize_blocks_e4m3 with MOE_SCALE_POW2
 * ffn % 16 == 0, else MOE_ERR_UNSUPPORTED.
 */
MOE_API moe_status moe_swiglu_save_e4m3(int32_t R, int32_t ffn, const void *g, const void *u, int64_t ld,
                                        void *h, uint8_t *h_codes, float *h_scales, uint8_t *saved_codes,
                                        float *saved_scales, moe_stream_t stream);

/*
 * moe_swiglu_backward_e4m3 -- the gradient of h = SiLU(g) * u from the kept
 * codes: with g, u the values they stand for and s = sigmoid(g),
 *
 *   dg = dh * u * s * (1 + g * (1 - s)),   du = dh * g * s,   h = g * s * u
 *
 *   dh            [R, ffn] bf16
 *   dg, du        [R, ffn] bf16 out, row pitch ld elements each
 *   h             [R, ffn] bf16 out, or NULL (for the down projection's
 *                 weight gradient, without having kept it)
 *   d_codes       [R, 2 ffn], d_scales [R, 2 ffn/128] out, or both NULL: dg,
 *                 then du of each row in blocks with MOE_SCALE_AMAX, from fp32
 *                 (the rows of the data gradient); needs ffn % 128 == 0
 * ffn % 16 == 0, else MOE_ERR_UNSUPPORTED.
 */
MOE_API moe_status moe_swiglu_backward_e4m3(int32_t R, int32_t ffn, const uint8_t *saved_codes,
                                            const float *saved_scales, const void *dh, void *dg, void *du,
                                            int64_t ld, void *h, uint8_t *d_codes, float *d_scales,
                                            moe_stream_t stream);

/*
 * moe_grouped_wgrad -- the weight gradient of a grouped product.  For every
 * expert e:
 *
 *   dw[e,n,k] = sum_{r of e} dy[r,n] * x[r,k]   (accumulate == 0; zeros for an
 *                                               expert without rows)
 *   dw[e,n,k] += the same                       (accumulate != 0)
 * summed in fp32, rounded once to dw_dtype (and once more by the addition).
 *
 *   dy   [R, N] bf16, row pitch ld_dy elements
 *   x    x_dtype MOE_BF16: [R, K], x_scales NULL; MOE_FP8_E4M3: codes [R, K]
 *        with x_scales [R, ceil(K/128)], x = code * scale: exact when the
 *        scales are powers of two, else rounded to bf16
 *   dw   [E, N, K] MOE_F32 or MOE_BF16, in and out
 * N % 16 == 0 and K % 16 == 0, else MOE_ERR_UNSUPPORTED.
 */
MOE_API moe_status moe_grouped_wgrad(int32_t R, int32_t N, int32_t K, int32_t E, int32_t x_dtype,
                                     int32_t dw_dtype, int32_t accumulate, const void *dy, int64_t ld_dy,
                                     const void *x, const float *x_scales, const int32_t *offsets, void *dw,
                                     moe_stream_t stream);

/*
 * moe_router_losses -- load-balance and z losses of a batch's router logits.
 * With p = softmax(logits[t,:]), lse[t] its log-sum-exp, n the tokens whose
 * mask is nonzero (all of them when mask is NULL) and c_e the assignments of
 * those tokens to expert e:
 *
 *   loss[0] = balance_coef * E * sum_e (c_e / (n k)) * (mean over them of p[t,e])
 *   loss[1] = z_coef * mean over them of lse[t]^2          (both 0 when n == 0)
 *
 *   logits   [T, E] fp32      topk_idx [T, k] int32      mask [T] bytes or NULL
 *   loss     [2] fp32 out
 *   counts   [E+1] int32 out: c_e, then n
 *   lse      [T] fp32 out
 *   workspace: moe_router_losses_workspace_size() bytes
 * A row whose logits are all -inf has no probabilities: it adds nothing to
 * the means' sums.  Indices outside [0, E) are skipped and flag
 * MOE_ERR_DEVICE_BOUNDS.  Bit-reproducible.
 */
MOE_API moe_status moe_router_losses(int32_t T, int32_t E, int32_t k, const float *logits,
                                     const int32_t *topk_idx, const uint8_t *mask, float balance_coef,
                                     float z_coef, float *loss, int32_t *counts, float *lse, void *workspace,
                                     size_t workspace_bytes, moe_stream_t stream);
MOE_API moe_status moe_router_losses_workspace_size(int32_t T, int32_t E, size_t *bytes);
MOE_API moe_status moe_router_losses_workspace_size_for(int32_t T, int32_t E, int32_t num_sms, size_t *bytes);

/*
 * moe_router_losses_backward -- the gradient of the router's logits: of
 * *grad_loss * (loss[0] + loss[1]) with the counts held constant (grad_loss
 * NULL: 1), and, when topk_w [T, k] (moe_router_topk's) and its gradient
 * d_topk_w are given, of the renormalised weights:
 *
 *   d_logits[t,e] = *grad_loss * mask_t / n * p[t,e] *
 *                     (balance_coef * E * (f_e - sum_j f_j p[t,j]) + 2 z_coef lse[t])
 *                 + (e == topk_idx[t,j]) * w_tj * (dw_tj - sum_i w_ti dw_ti)
 * with f_e = c_e / (n k).  Masked tokens keep the second part.  A row whose
 * logits are all -inf gets no gradient from the losses.
 *   d_logits [T, E] fp32 out
 */
MOE_API moe_status moe_router_losses_backward(int32_t T, int32_t E, int32_t k, const float *logits,
                                              const int32_t *topk_idx, const uint8_t *mask,
                                              float balance_coef, float z_coef, const int32_t *counts,
                                              const float *lse, const float *grad_loss, const float *topk_w,
                                              const float *d_topk_w, float *d_logits, moe_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * The experts in 4 bits, and the gradients of the token movement.  No page
 * counterpart beyond the MXFP4 storage above: the rows that a layer's tokens
 * become (moe_dispatch, moe_combine_rows), as they are or in MXFP4, products
 * of MXFP4 rows with MXFP4 weights, and what training needs of the movement.
 *
 * MXFP4 rows [rows, cols]: codes [rows, cols/2], two E2M1 codes a byte
 * (element 2i in the low half of byte i), and scales [rows, cols/32]: byte b
 * stands for 2^(b - 127), 255 for NaN; a value is E2M1(code) * scale.  MXFP4
 * weights [E, N, K] have codes [E, N, K/2] and scales [E, K/32, N], as the
 * layer's MOE_MXFP4 weights.
 * Assignments whose expert index is negative are dropped: padding tokens, or
 * an expert's capacity.  They take no row and add nothing; inv_row is -1 there.
 * Limits: E <= 1024, k <= 32, T * k <= 2^24, rows <= 2^24.
 * ---------------------------------------------------------------------------
 */
typedef enum moe_mx_scale {
  MOE_MX_FLOOR = 0, /* 2^(floor(log2 a) - 2), the OCP MX rule: the largest
                       magnitudes of a block, above 6 scales, become 6        */
  MOE_MX_FIT = 1    /* the least 2^p with a / 2^p <= 6: nothing is clipped    */
} moe_mx_scale;

/*
 * moe_dispatch -- tokens to rows grouped by expert.
 *
 *   topk_idx  [T, k] int32: expert of each assignment, negative: dropped.
 *             Values from E on are dropped too and flag MOE_ERR_DEVICE_BOUNDS
 *   counts    [E] out: assignments of each expert
 *   offsets   [E+1] out: offsets[e] = sum of counts before e
 *   row_token [T*k] out: token of each row; -1 from row offsets[E] on
 *   inv_row   [T, k] out: row of each assignment, or -1
 *   rows      out, or NULL (maps alone; x is not read then):
 *             rows_dtype x_dtype: rows[r,:] = x[row_token[r],:], [T*k, d]
 *             rows_dtype MOE_MXFP4 (d % 32 == 0): codes [T*k, d/2] of them with
 *             row_scales [T*k, d/32], as moe_quantize_mxfp4 with scale_kind
 *   x         [T, d] MOE_BF16 or MOE_F32, row pitch ld_x elements
 * Rows of an expert are in assignment order (bit-exact).  Rows from
 * offsets[E] on are left as they are.  d % 8 == 0, else MOE_ERR_UNSUPPORTED.
 * T == 0: counts and offsets are set to zero.
 *   workspace: moe_dispatch_workspace_size() bytes (the same on every device;
 *              0: may be NULL).  Calls that overlap on the GPU need one each.
 */
MOE_API moe_status moe_dispatch(int32_t T, int32_t d, int32_t E, int32_t k, int32_t x_dtype, int32_t rows_dtype,
                                int32_t scale_kind, const void *x, int64_t ld_x, const int32_t *topk_idx,
                                int32_t *counts, int32_t *offsets, int32_t *row_token, int32_t *inv_row,
                                void *rows, uint8_t *row_scales, void *workspace, size_t workspace_bytes,
                                moe_stream_t stream);
MOE_API moe_status moe_dispatch_workspace_size(int32_t T, int32_t E, int32_t k, size_t *bytes);

/*
 * moe_combine_rows -- rows back to tokens: as moe_combine, with dropped
 * assignments and, without weights, the gradient of moe_dispatch.
 *
 *   out[t,:] = sum_j topk_w[t,j] * rows[inv_row[t,j],:] (+ add[t,:])
 *
 * over the assignments with inv_row >= 0, in fp32 in slot order, then add,
 * rounded once to dtype.
 *   rows     [R, d] MOE_BF16 or MOE_F32     inv_row [T, k] int32
 *   topk_w   [T, k] fp32, or NULL: weights of 1 (d_x of moe_dispatch from the
 *            rows' gradients, MXFP4's rounding passed through; add: what
 *            reaches x another way)
 *   add      [T, d] dtype or NULL           out [T, d] dtype (may be add)
 * inv_row values from R on are skipped and flag MOE_ERR_DEVICE_BOUNDS.
 * d % 8 == 0, else MOE_ERR_UNSUPPORTED.  T == 0: nothing is enqueued.
 */
MOE_API moe_status moe_combine_rows(int32_t T, int32_t d, int32_t k, int32_t R, int32_t dtype, const void *rows,
                                    const int32_t *inv_row, const float *topk_w, const void *add, void *out,
                                    moe_stream_t stream);

/*
 * moe_combine_rows_backward -- the gradients of moe_combine_rows:
 *
 *   d_rows[inv_row[t,j],:] = topk_w[t,j] * d_out[t,:]
 *   d_topk_w[t,j]          = sum_i d_out[t,i] * rows[inv_row[t,j],i]
 *
 * (0 where the assignment is dropped; the gradient of add is d_out).  Sums in
 * fp32 in a fixed order.  d_rows [R, d] dtype out, or NULL; d_topk_w [T, k]
 * fp32 out, or NULL (rows is not read then).  topk_w NULL: weights of 1.
 * Rows that no assignment has are left as they are.  inv_row holds each row at
 * most once.
 */
MOE_API moe_status moe_combine_rows_backward(int32_t T, int32_t d, int32_t k, int32_t R, int32_t dtype,
                                             const void *d_out, const void *rows, const int32_t *inv_row,
                                             const float *topk_w, void *d_rows, float *d_topk_w,
                                             moe_stream_t stream);

/*
 * moe_quantize_mxfp4 -- MXFP4 codes and scales of rows or weights.
 *
 *   a     = largest magnitude of the block of 32 columns
 *   scale = 2^p, p by scale_kind within [-127, 127]; 1 when a == 0
 *   code  = E2M1(x / 2^p): nearest value, ties to the even code, magnitudes
 *           above 6 saturated to 6, sign kept
 * A block with an infinity or a NaN gets scale 255 and codes 0: all of its
 * values are NaN.  Codes and scales are exact functions of the inputs.
 *
 *   x       [rows, cols] MOE_BF16 or MOE_F32, row pitch ld_x elements
 *   codes   [rows, cols/2] out
 *   scales  matrix_rows == 0: [rows, cols/32] out; else x is rows/matrix_rows
 *           weight matrices of matrix_rows rows, scales
 *           [rows/matrix_rows, cols/32, matrix_rows] out
 * cols % 32 == 0, else MOE_ERR_UNSUPPORTED.  rows == 0: nothing is enqueued.
 */
MOE_API moe_status moe_quantize_mxfp4(int32_t rows, int32_t cols, int32_t x_dtype, int32_t scale_kind,
                                      int32_t matrix_rows, const void *x, int64_t ld_x, uint8_t *codes,
                                      uint8_t *scales, moe_stream_t stream);

/*
 * moe_mxfp4_values -- the values that MXFP4 codes stand for, rounded to dtype
 * (exact but where it over- or underflows); sizes and layouts as
 * moe_quantize_mxfp4.   out [rows, cols] MOE_BF16 or MOE_F32
 */
MOE_API moe_status moe_mxfp4_values(int32_t rows, int32_t cols, int32_t dtype, int32_t matrix_rows,
                                    const uint8_t *codes, const uint8_t *scales, void *out, moe_stream_t stream);

/*
 * moe_swiglu_mxfp4 -- h = SiLU(g) * u in fp32 as MXFP4 rows.
 *
 *   g, u     [R, ffn] bf16, row pitch ld elements each (the halves of one
 *            [R, 2 ffn] product: u = g + ffn, ld = 2 ffn)
 *   codes    [R, ffn/2] out      scales [R, ffn/32] out
 *   h        [R, ffn] bf16 out, or NULL
 * ffn % 32 == 0, else MOE_ERR_UNSUPPORTED.  R == 0: nothing is enqueued.
 */
MOE_API moe_status moe_swiglu_mxfp4(int32_t R, int32_t ffn, int32_t scale_kind, const void *g, const void *u,
                                    int64_t ld, uint8_t *codes, uint8_t *scales, void *h, moe_stream_t stream);

/*
 * moe_grouped_mxfp4_gemm -- MXFP4 rows times MXFP4 weights.  For every row r
 * of expert e (offsets [E+1] int32 on the device):
 *
 *   out[r,n] = sum_b 2^(sa[r,b] - 127) * 2^(sw[e,b,n] - 127) *
 *              sum_{i in block b} a[r,i] * w[e,n,i]
 *
 * products exact down to 2^-149, fp32's least step (below it each may lose up to
 * one), sums in fp32 on the tensor cores (a partial sum past its range makes the
 * result infinite), rounded once to out_dtype.
 *   a_codes [R, K/2]      a_scales [R, K/32]
 *   w_codes [E, N, K/2]   w_scales [E, K/32, N]
 *   out     [R, N] MOE_BF16 or MOE_F32, row pitch ld_out elements
 * A scale of 255 makes every result that it enters NaN.  The gradient of the
 * rows is the same product with the weights quantised along N (the codes of
 * each matrix's transpose).  Offsets outside [0, R], or decreasing ones, are
 * clamped and flag MOE_ERR_DEVICE_BOUNDS.  Rows outside every expert's range
 * are left untouched.  K % 32 == 0 and N % 16 == 0, else MOE_ERR_UNSUPPORTED;
 * R == 0: nothing is enqueued.
 */
MOE_API moe_status moe_grouped_mxfp4_gemm(int32_t R, int32_t K, int32_t N, int32_t E, int32_t out_dtype,
                                          const uint8_t *a_codes, const uint8_t *a_scales, const int32_t *offsets,
                                          const uint8_t *w_codes, const uint8_t *w_scales, void *out,
                                          int64_t ld_out, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
