/*
 * tb.h -- C ABI of the GB300 (sm_103a) memory-bound training-step library.
 *
 * The library implements the memory-bound half of an LLM training step as
 * hand-written CUDA kernels:
 *   - a fused, multi-tensor, mixed-precision AdamW update;
 *   - the row-wise softmax backward;
 *   - the LayerNorm backward (dX, dgamma, dbeta);
 *   - rotary positions and the per-head RMS norm of queries and keys, with their
 *     gradients;
 *   - causal attention over whole prompts, with its gradient;
 *   - the gated projections of a feed-forward block, with their gradients;
 *   - the softmax cross entropy of a linear output layer, with its gradients.
 *
 * Sources (web pages on the subject; cited by page title and section):
 *   [GPU-Opt-P2]  "GPU 优化实战 Part 2：用 CUDA/ROCm 实现 LLM 反向传播与训练循环"
 *   [Mastering]   "Mastering LLM Training with CUDA and ROCm: The Backpropagation
 *                  and Optimization Workflow"
 *
 * Conventions for every entry point
 *   - Buffers are device-accessible memory owned by the caller, row-major and
 *     contiguous (queries, keys and values are strided: see tb_heads).  The library
 *     keeps no pointer after a call returns, except the AdamW plan's copy of
 *     the tensor table (see tb_adamw_plan_create).
 *   - `stream` is a cudaStream_t passed as void*; NULL is the legacy default
 *     stream.  Work is enqueued on it and the call returns without waiting: a
 *     fault inside a kernel surfaces at the caller's next synchronisation.
 *   - Argument errors are reported synchronously, before anything is enqueued,
 *     as a tb_status.  A failed launch reports TB_ERR_CUDA.
 *   - The softmax, LayerNorm, RMSNorm, rotary, attention, gated and output-layer
 *     kernels are launched as programmatic
 *     dependents of the work before them on `stream`: their blocks may start
 *     while the previous kernel drains, set up shared memory and (LayerNorm,
 *     RMSNorm) prefetch their first rows into L2, but they load and store no
 *     global memory before every earlier kernel on the stream has completed and
 *     its writes are visible.  Stream order is kept exactly.
 *   - fp32 pointers must be 4-byte aligned, 16-bit pointers 2-byte aligned and
 *     64-bit ones 8-byte aligned (TB_ERR_MISALIGNED otherwise).  Any larger
 *     alignment is optional: 16-byte aligned buffers take the vectorised path,
 *     others a scalar one.  Exceptions: workspaces are 16-byte aligned, and
 *     so are attention's heads, the gated projections' matrices, and the output
 *     layer's H and W where D is a multiple of 8.
 *   - The calls are not thread-safe against tb_adamw_plan_destroy of the plan
 *     they use; otherwise they may be called from several host threads.
 */
#ifndef TB_H_
#define TB_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum tb_status {
    TB_OK = 0,
    TB_ERR_INVALID_VALUE = 1,     /* null pointer, negative size, step < 1, ... */
    TB_ERR_UNSUPPORTED_DTYPE = 2, /* dtype not accepted by this entry point     */
    TB_ERR_MISALIGNED = 3,        /* pointer not aligned to its element size    */
    TB_ERR_ALIAS = 4,             /* an output overlaps an input or another output */
    TB_ERR_WORKSPACE = 5,         /* workspace missing or smaller than required */
    TB_ERR_OOM = 6,               /* the library's own small allocation failed  */
    TB_ERR_CUDA = 7,              /* a CUDA runtime call or launch failed        */
    TB_ERR_DEVICE = 8,            /* plan used with another device current       */
    TB_ERR_TIMEOUT = 9            /* a kernel's bounded wait gave up (see tb_device_error) */
} tb_status;

typedef enum tb_dtype {
    TB_F32 = 0,   /* IEEE binary32 */
    TB_F16 = 1,   /* IEEE binary16 */
    TB_BF16 = 2   /* bfloat16 */
} tb_dtype;

/* Human-readable name of a status code (static storage; never NULL). */
const char* tb_status_string(tb_status status);

/* Library version as 10000*major + 100*minor + patch. */
int tb_version(void);

/*
 * tb_device_error -- read (and optionally clear) the device-side error word of
 * the current device.  Kernels that wait on an mbarrier for their own bulk
 * copies (and, in attention, the gated projections and the output layer's loss,
 * tensor-core instructions) give up
 * after about one second; they then set this word to
 * TB_ERR_TIMEOUT, drain what they issued and return early (their outputs are
 * then undefined).  tb_adamw_step_device sets it to TB_ERR_INVALID_VALUE when
 * the step counter it reads is below 1, tb_linear_xent when a target is
 * neither in the vocabulary nor ignore_index, and the attention calls when offsets
 * do not count up within the row.  This call synchronises the
 * current device.
 *   code   out: 0 when no kernel gave up since the last reset
 *   reset  nonzero: clear the word after reading it
 * Returns TB_OK, TB_ERR_INVALID_VALUE (code == NULL) or TB_ERR_CUDA.
 */
tb_status tb_device_error(int* code, int reset);

/*
 * tb_layernorm_bwd_selftest_timeout -- exercises that failure path without a
 * GPU fault.  It runs the LayerNorm backward's two bulk-copy ring kernels on
 * small internal problems (4 x 256 bf16 on one CTA per row block, then 4 x
 * 16,384 bf16 split over a four-CTA cluster; zeroed buffers the call allocates
 * and frees) with their copies withheld, so that every wait on them runs out after
 * wait_limit_ns nanoseconds; each kernel then sets the device error word to
 * TB_ERR_TIMEOUT, waits (bounded as well) for the copies it would have issued,
 * and returns -- the CTAs of a cluster together, after telling each other of the
 * failure.  Nothing is in flight when it returns, so the context stays usable.
 * The call synchronises `stream`; afterwards tb_device_error reports
 * TB_ERR_TIMEOUT.
 *   wait_limit_ns  1,000 .. 1,000,000,000
 * Returns TB_OK once the kernel has finished, TB_ERR_INVALID_VALUE (limit out of
 * range), TB_ERR_OOM or TB_ERR_CUDA.
 */
tb_status tb_layernorm_bwd_selftest_timeout(int64_t wait_limit_ns, void* stream);

/*
 * tb_linear_xent_selftest_timeout -- the same for the output layer's products,
 * whose waits stand between two CTAs: their bulk copies, their tensor-core
 * instructions and the accumulators that they hand over.  It runs the loss's
 * product on one pair of CTAs over three small internal problems (zeroed
 * buffers the call allocates and frees), TB_LINEAR_XENT_SELFTEST_LAUNCHES
 * launches in all, each with one thing withheld: the copies of one of the two
 * CTAs, the word that an accumulator is complete, or the word that it is free
 * again.  Every launch sets the device error word to TB_ERR_TIMEOUT, waits
 * (bounded as well) for all copies and tensor-core instructions that either CTA
 * had started, and returns.  The call synchronises
 * `stream` and resets the device error word before each launch; afterwards the
 * word is the last launch's, TB_ERR_TIMEOUT.
 *   wait_limit_ns  1,000 .. 1,000,000,000
 *   launches       out: launches whose waits gave up
 * Returns TB_OK once the kernels have finished, TB_ERR_INVALID_VALUE (limit out
 * of range, launches == NULL), TB_ERR_OOM or TB_ERR_CUDA.
 */
#define TB_LINEAR_XENT_SELFTEST_LAUNCHES 11

tb_status tb_linear_xent_selftest_timeout(int64_t wait_limit_ns, int* launches, void* stream);

/*
 * tb_attention_selftest_timeout, tb_gated_linear_selftest_timeout -- the same for
 * the kernels of attention (forward, the gradient of keys and values, that of
 * queries; heads of 64 and 128) and for the two products of the gated projections:
 * TB_ATTENTION_SELFTEST_LAUNCHES and TB_GATED_LINEAR_SELFTEST_LAUNCHES launches on
 * small internal problems, each with the loads of one of the two CTAs withheld, or
 * a word by which the warps hand over what lies in tensor memory.
 */
#define TB_ATTENTION_SELFTEST_LAUNCHES 30
#define TB_GATED_LINEAR_SELFTEST_LAUNCHES 8

tb_status tb_attention_selftest_timeout(int64_t wait_limit_ns, int* launches, void* stream);

tb_status tb_gated_linear_selftest_timeout(int64_t wait_limit_ns, int* launches, void* stream);

/* ======================================================================== */
/* Fused mixed-precision AdamW (multi-tensor)                               */
/* ======================================================================== */
/*
 * One pass over every element of every tensor computes, per element
 * ([Mastering] §"AdamW Algorithm" update rule; [GPU-Opt-P2] §"AdamW 优化器——
 * 融合内核" and §"混合精度训练（FP16 / BF16）"):
 *     g      = float(grad) * inv_loss_scale            (unscale)
 *     m      = beta1*m + (1-beta1)*g
 *     v      = beta2*v + (1-beta2)*g*g
 *     m_hat  = m / (1 - beta1^t),  v_hat = v / (1 - beta2^t)
 *     param  = param - lr*(m_hat/(sqrt(v_hat)+eps) + weight_decay*param_t)
 *     copy   = round-to-nearest-even(param) in copy_dtype
 *     grad   = +0
 * with decoupled weight decay taken on the pre-update parameter param_t.
 * The bias corrections and (1-beta) are formed once per call on the host.
 */
typedef struct tb_tensor_desc {
    float* param;   /* fp32 master weights [n], read and written in place        */
    float* m;       /* fp32 first moment   [n], read and written in place        */
    float* v;       /* fp32 second moment  [n], read and written in place        */
    void* grad;     /* loss-scaled gradient [n] in grad_dtype, read then zeroed  */
    void* copy;     /* working copy [n] in copy_dtype, written; NULL: none       */
    int64_t n;      /* element count (>= 0; 0 skips the tensor)                  */
} tb_tensor_desc;

typedef struct tb_adamw_hparams {
    float lr;            /* learning rate eta                         */
    float beta1;         /* first-moment decay, in [0, 1)             */
    float beta2;         /* second-moment decay, in [0, 1)            */
    float eps;           /* added to sqrt(v_hat), >= 0                */
    float weight_decay;  /* decoupled decay lambda, >= 0              */
} tb_adamw_hparams;

typedef struct tb_adamw_plan tb_adamw_plan;   /* opaque */

/*
 * tb_adamw_plan_create -- validate a table of parameter tensors and copy it to
 * the current device once, so that every later step is a single launch.
 *   tensors     host array of n_tensors descriptors (read during the call only)
 *   n_tensors   >= 1
 *   grad_dtype  TB_F16, TB_BF16 or TB_F32
 *   copy_dtype  TB_BF16 or TB_F16 (unused when the tensors have no copy)
 *               Either every tensor with n > 0 has a working copy, or none has
 *               (copy == NULL: the step writes no copy).
 *   out         receives the plan; the caller owns it and frees it with
 *               tb_adamw_plan_destroy.  The plan owns a device copy of the table
 *               (64 bytes per tensor) followed by the step kernel's 16-byte tile
 *               counter, and remembers the current device.
 *               Every call that takes a plan first looks it up among the plans
 *               created and not yet destroyed; any other pointer (a destroyed
 *               plan included) is rejected with TB_ERR_INVALID_VALUE without
 *               being dereferenced.
 * Errors: TB_ERR_INVALID_VALUE (null param/m/v/grad with n > 0, copies given for
 * some tensors only, n < 0, n_tensors < 1,
 * out == NULL), TB_ERR_UNSUPPORTED_DTYPE, TB_ERR_MISALIGNED, TB_ERR_ALIAS (any
 * two of the 5*n_tensors buffers overlap), TB_ERR_OOM, TB_ERR_CUDA.
 */
tb_status tb_adamw_plan_create(const tb_tensor_desc* tensors, int n_tensors,
                               tb_dtype grad_dtype, tb_dtype copy_dtype,
                               tb_adamw_plan** out);

/*
 * tb_adamw_step -- enqueue one fused AdamW step over every tensor of the plan.
 *   step            global step t >= 1 (the first update is t = 1)
 *   hp              hyperparameters (read during the call only)
 *   inv_loss_scale  1/loss_scale (exact for a power-of-two scale); > 0
 *   stream          cudaStream_t or NULL
 * The kernel's CTAs claim tiles of the flat parameter space from a counter kept
 * in the plan's device memory (so CTAs on faster SMs take more tiles).  Each call
 * enqueues a 16-byte cudaMemsetAsync of that counter on `stream` before the
 * launch, so every launch starts from zero whatever an earlier launch left
 * there.  Steps of one plan (plain, clipped or device) must run one after
 * another: on one stream, or ordered by events.  They update the same tensors
 * and share the counter, so they must be ordered in any case.
 * Errors: TB_ERR_INVALID_VALUE (plan/hp NULL, step < 1, beta outside [0,1),
 * eps, lr or weight_decay negative or not finite, inv_loss_scale <= 0),
 * TB_ERR_DEVICE (another device is current), TB_ERR_CUDA.
 */
tb_status tb_adamw_step(const tb_adamw_plan* plan, int64_t step,
                        const tb_adamw_hparams* hp, float inv_loss_scale,
                        void* stream);

/*
 * Global gradient-norm clipping with a non-finite check, fused into the step
 * without a host synchronisation ([GPU-Opt-P2] §"完整训练循环（整合一切）", its
 * gradient-clipping step: the L2 norm of the unscaled gradient over all
 * parameters; when it exceeds max_norm the gradients are scaled by
 * max_norm / norm before the optimizer).
 *
 * tb_adamw_grad_norm reads every gradient of the plan once (2 bytes per
 * parameter) and writes three floats to device memory `out`:
 *     out[0] = norm   = sqrt(sum_i (float(grad_i) * inv_loss_scale)^2)
 *     out[1] = factor = max_norm / norm if max_norm > 0 and norm > max_norm, else 1
 *     out[2] = 1 if any gradient element is NaN or infinite, else 0
 * Each thread adds its squares in fp32 in rounds of at most 32, adds the round
 * sums of one tile (at most 256 squares) in fp32 and the tile sums in fp64; each
 * CTA adds a fixed set of tiles (consecutive chunks of 262,144 elements on large
 * tables, tiles dealt round-robin on small ones) into one partial, and the
 * partials are added in a fixed order, so the result is reproducible.
 *   workspace  device scratch of tb_adamw_grad_norm_workspace_size() bytes,
 *              8-byte aligned (one fp64 partial and one flag per CTA)
 * Errors: TB_ERR_INVALID_VALUE, TB_ERR_MISALIGNED, TB_ERR_WORKSPACE, TB_ERR_ALIAS,
 * TB_ERR_DEVICE, TB_ERR_CUDA.
 *
 * tb_adamw_step_clipped is tb_adamw_step with the unscaled gradient multiplied by
 * clip[1] (clip = the `out` of tb_adamw_grad_norm, read on the device).  When
 * clip[2] != 0 the step does not happen: parameters, moments and the working copy
 * are left as they are and only the gradient is reset to zero.  Whether the
 * caller then advances its step counter is its choice (clip[2] can be read back
 * later).  Errors as tb_adamw_step, plus TB_ERR_INVALID_VALUE for clip == NULL.
 */
tb_status tb_adamw_grad_norm_workspace_size(const tb_adamw_plan* plan, size_t* bytes);

tb_status tb_adamw_grad_norm(const tb_adamw_plan* plan, float inv_loss_scale, float max_norm,
                             float* out, void* workspace, size_t workspace_bytes, void* stream);

tb_status tb_adamw_step_clipped(const tb_adamw_plan* plan, int64_t step,
                                const tb_adamw_hparams* hp, float inv_loss_scale,
                                const float* clip, void* stream);

/*
 * tb_adamw_step_device -- tb_adamw_step (clip == NULL) or tb_adamw_step_clipped
 * (clip != NULL) with the step counter in device memory: the kernel reads t from
 * `step` when it runs and forms the bias corrections 1 - beta^t itself (in
 * double, rounded to fp32, as the host does for the other entry points).  With
 * every per-step input on the device, a whole optimizer step -- counter
 * increment, gradient norm, update -- can be captured once in a CUDA graph and
 * replayed every iteration.  The counter is only read: the caller advances it.
 *   step   device int64, 8-byte aligned; a value below 1 makes the kernel set the
 *          device error word to TB_ERR_INVALID_VALUE and update nothing
 *   clip   NULL, or the device output of tb_adamw_grad_norm
 * Errors: as tb_adamw_step, plus TB_ERR_INVALID_VALUE (step == NULL) and
 * TB_ERR_MISALIGNED.
 */
tb_status tb_adamw_step_device(const tb_adamw_plan* plan, const int64_t* step,
                               const tb_adamw_hparams* hp, float inv_loss_scale,
                               const float* clip, void* stream);

/*
 * tb_adamw_selftest_stale_counter -- test hook for the tile counter above.  It
 * waits for `stream`, then writes `next` into the plan's tile counter (and a
 * nonzero value into the counter's second word) with a synchronous cudaMemcpy,
 * as a launch that stopped part-way would leave them.  The next step of the
 * plan must still update and zero every element.  Not for use in training.
 * Errors: TB_ERR_INVALID_VALUE (not a live plan), TB_ERR_DEVICE, TB_ERR_CUDA.
 */
tb_status tb_adamw_selftest_stale_counter(const tb_adamw_plan* plan, uint64_t next,
                                          void* stream);

/* Free a plan (NULL is accepted; a pointer that is not a live plan, e.g. one
 * destroyed already, returns TB_ERR_INVALID_VALUE).  Synchronises nothing: the
 * caller must not destroy a plan while a step that uses it may still be running. */
tb_status tb_adamw_plan_destroy(tb_adamw_plan* plan);

/* ======================================================================== */
/* Stand-alone casts                                                         */
/* ======================================================================== */
/*
 * The two casts of the pages' mixed-precision loop that the fused step does
 * internally ([GPU-Opt-P2] §"混合精度训练（FP16 / BF16）", §"完整训练循环（整合一切）"
 * its unscale cast and its copy-back cast), for callers that keep the optimizer
 * steps apart:
 *   tb_cast_to_f32   : dst[i] = float(src[i]) * scale (one fp32 rounding),
 *                      src in src_dtype (TB_F16, TB_BF16 or TB_F32), dst fp32
 *   tb_cast_from_f32 : dst[i] = round-to-nearest-even(src[i]) in dst_dtype
 *                      (TB_F16 or TB_BF16)
 *   0 <= n <= INT64_MAX / 8 elements (0: nothing is enqueued); src and dst must not
 *   overlap.
 * Errors: TB_ERR_INVALID_VALUE, TB_ERR_UNSUPPORTED_DTYPE, TB_ERR_MISALIGNED,
 * TB_ERR_ALIAS, TB_ERR_CUDA.
 */
tb_status tb_cast_to_f32(const void* src, tb_dtype src_dtype, float scale, float* dst,
                         int64_t n, void* stream);

tb_status tb_cast_from_f32(const float* src, void* dst, tb_dtype dst_dtype, int64_t n,
                           void* stream);

/* ======================================================================== */
/* Softmax backward                                                          */
/* ======================================================================== */
/*
 * tb_softmax_bwd -- for every row r of a [rows, cols] matrix
 *     dX[r,i] = P[r,i] * (dY[r,i] - sum_j P[r,j]*dY[r,j])
 * ([GPU-Opt-P2] §2.1 "Softmax 反向内核"), P being the forward softmax output.
 * The dot product is accumulated in fp32 whatever the I/O dtype.
 *   dY, P   inputs [rows, cols] in dtype
 *   dX      output [rows, cols] in dtype; must not overlap dY or P
 *   rows, cols  >= 0 (either 0: nothing is enqueued)
 *   dtype   TB_F32, TB_BF16 or TB_F16
 * Each element of dY and P is read from HBM once when a row fits on chip
 * (cols <= 8192 fp32 / 16384 16-bit, 16-byte aligned rows); longer or
 * unaligned rows are read twice.
 * Errors: TB_ERR_INVALID_VALUE, TB_ERR_UNSUPPORTED_DTYPE, TB_ERR_MISALIGNED,
 * TB_ERR_ALIAS, TB_ERR_CUDA.
 */
tb_status tb_softmax_bwd(const void* dY, const void* P, void* dX,
                         int64_t rows, int64_t cols, tb_dtype dtype, void* stream);

/*
 * tb_softmax_bwd_causal -- tb_softmax_bwd for the rows of causally masked
 * attention, reading only the part of each row the mask left open.
 * Row r can be nonzero only on its first
 *     valid(r) = min(cols, (r mod period) + 1 + offset)
 * columns: `period` is the query length S_q of one (batch, head) block whose
 * rows are stacked, `offset` = S_k - S_q (0 for square self-attention).  P must
 * be exactly 0 on every other column, as a masked forward softmax leaves it; the
 * kernel never reads those columns of P or dY and writes +0 to dX there.  On
 * such inputs the result equals tb_softmax_bwd's (masked entries are +-0 there)
 * bit for bit for rows of up to 2,048 16-bit / 1,024 fp32 columns; longer rows
 * sum the same dot-product terms in another grouping and agree within its fp32
 * rounding.  Every call on the same inputs returns the same bits.  When a
 * causal block fits in `rows` (period <= rows), rows q and period-1-q of a block
 * are processed together, so the work per warp or CTA does not depend on q.
 * HBM traffic per row: reads of the valid columns (rounded up to 16-byte
 * vectors) plus the full row of dX written.
 *   period >= 1, offset >= 0; other arguments and errors as tb_softmax_bwd.
 */
tb_status tb_softmax_bwd_causal(const void* dY, const void* P, void* dX, int64_t rows,
                                int64_t cols, int64_t period, int64_t offset,
                                tb_dtype dtype, void* stream);

/* ======================================================================== */
/* LayerNorm backward                                                        */
/* ======================================================================== */
/*
 * Forward being y = gamma * xhat + beta with xhat = (x - mean) * inv_std over
 * the D features of each row, the backward computes ([GPU-Opt-P2] §2.2
 * "LayerNorm 反向"; [Mastering] §"Layer Normalization Backpropagation"):
 *     dxhat   = dY * gamma
 *     dX      = inv_std * (dxhat - mean_D(dxhat) - xhat * mean_D(dxhat*xhat))
 *     dgamma  = sum over rows of dY * xhat     (per column)
 *     dbeta   = sum over rows of dY            (per column)
 * dgamma and dbeta are OVERWRITTEN (not accumulated).  They are reduced in two
 * stages -- per-CTA partial sums into the workspace, then a second kernel that
 * adds them in a fixed order -- so results are bitwise reproducible run to run
 * on the same device model.  Rows longer than 16 KB (more than 8,192 16-bit or
 * 4,096 fp32 columns; 16-byte aligned buffers, D a multiple of 2..8 times the
 * 16-byte vector) are split by columns over the CTAs of a thread-block cluster,
 * which exchange their shares of the row sums through distributed shared memory
 * and write one partial row per cluster; all CTAs of a cluster use bitwise the
 * same row sums.
 */

/*
 * tb_layernorm_bwd_workspace_size -- bytes of workspace tb_layernorm_bwd needs
 * for this shape on the current device (it depends on the SM count).
 * Errors: TB_ERR_INVALID_VALUE (bytes NULL, rows or D negative),
 * TB_ERR_UNSUPPORTED_DTYPE, TB_ERR_CUDA.
 */
tb_status tb_layernorm_bwd_workspace_size(int64_t rows, int64_t D, tb_dtype io_dtype,
                                          size_t* bytes);

/*
 * tb_layernorm_bwd
 *   dY, x      inputs [rows, D] in io_dtype (TB_F32, TB_BF16 or TB_F16)
 *   mean       fp32 [rows], the forward's saved row means
 *   inv_std    fp32 [rows], the forward's saved 1/sqrt(var + eps)
 *   gamma      fp32 [D]
 *   dX         output [rows, D] in io_dtype
 *   dgamma     output fp32 [D]
 *   dbeta      output fp32 [D]
 *   workspace  device scratch of at least tb_layernorm_bwd_workspace_size()
 *              bytes, 16-byte aligned; contents on entry are ignored
 *   stream     cudaStream_t or NULL
 * rows == 0 writes zeros to dgamma and dbeta; D == 0 enqueues nothing.
 * Outputs must not overlap any input, each other or the workspace.
 * Errors: TB_ERR_INVALID_VALUE, TB_ERR_UNSUPPORTED_DTYPE, TB_ERR_MISALIGNED,
 * TB_ERR_ALIAS, TB_ERR_WORKSPACE, TB_ERR_CUDA.
 */
tb_status tb_layernorm_bwd(const void* dY, const void* x, const float* mean,
                           const float* inv_std, const float* gamma,
                           void* dX, float* dgamma, float* dbeta,
                           int64_t rows, int64_t D, tb_dtype io_dtype,
                           void* workspace, size_t workspace_bytes, void* stream);

/* ======================================================================== */
/* RMSNorm backward                                                          */
/* ======================================================================== */
/*
 * The LayerNorm above without the mean subtraction and without beta (the norm
 * layers of Llama-style models): forward y = gamma * x * inv_rms with
 * inv_rms = 1/sqrt(mean_D(x^2) + eps).  Backward, per row and per column:
 *     dxhat  = dY * gamma,  xhat = x * inv_rms
 *     dX     = inv_rms * (dxhat - xhat * mean_D(dxhat * xhat))
 *     dgamma = sum over rows of dY * xhat      (overwritten, two-stage, deterministic)
 * Same kernels, layouts, alignment rules and errors as tb_layernorm_bwd, with
 * inv_rms in place of mean/inv_std and no dbeta.  The workspace is half the
 * LayerNorm one (one partial row of D floats per CTA).
 */
tb_status tb_rmsnorm_bwd_workspace_size(int64_t rows, int64_t D, tb_dtype io_dtype,
                                        size_t* bytes);

tb_status tb_rmsnorm_bwd(const void* dY, const void* x, const float* inv_rms,
                         const float* gamma, void* dX, float* dgamma,
                         int64_t rows, int64_t D, tb_dtype io_dtype,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * tb_layernorm_bwd_noalloc -- the same LayerNorm backward as tb_layernorm_bwd,
 * for callers that cannot allocate device memory when they run it.  (The pages
 * have no counterpart: this is a convenience of this library.)
 *
 * Who needs it: code that runs where a cudaMalloc is not an option -- inside a
 * framework that hands out every byte of device memory from its own pool (a
 * stray allocation there fails or fragments the pool), or a step loop that must
 * not call cudaMalloc/cudaFree because they can synchronise with the device.
 * Such callers have no buffer to pass as `workspace`, so this entry point keeps
 * its scratch (the per-CTA dgamma/dbeta partial sums) in a fixed array inside
 * the library and allocates nothing: no cudaMalloc, no cudaFree, no allocating
 * library call.
 *
 * The array holds TB_LAYERNORM_NOALLOC_SCRATCH_BYTES (16 MiB).  Every GPU that
 * loads the library holds it until the process exits.  A shape whose partial
 * sums would not fit runs with fewer CTAs; D > 2,097,152 (more than the array
 * holds for a single CTA) is rejected with TB_ERR_WORKSPACE.
 *
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call before
 * any stream capture.  All calls share the one array and it keeps the last
 * call's contents (each call overwrites every part it later reads, so nothing
 * has to start at zero): calls whose work overlaps on the GPU -- for example on
 * two streams at once -- race on it and must be serialised by the caller.
 *
 * Arguments, results and errors are those of tb_layernorm_bwd without
 * `workspace` and `workspace_bytes`; results equal tb_layernorm_bwd's bit for
 * bit whenever the partial sums fit with the usual number of CTAs (for example
 * 16,384 x 4,096 bf16), and agree within rounding otherwise.
 */
#define TB_LAYERNORM_NOALLOC_SCRATCH_BYTES (16u << 20)

tb_status tb_layernorm_bwd_noalloc(const void* dY, const void* x, const float* mean,
                                   const float* inv_std, const float* gamma,
                                   void* dX, float* dgamma, float* dbeta,
                                   int64_t rows, int64_t D, tb_dtype io_dtype, void* stream);

/* ======================================================================== */
/* Rotary positions; per-head RMS norm of queries and keys                   */
/* ======================================================================== */
/*
 * The queries and keys of one attention layer on their way from the projection
 * to the attention product, and their gradients on the way back.  (The pages
 * have no counterpart: they take attention's softmax backward by itself.)
 *
 * A rotated pair (a, b) with frequency w_i, at position p and angle t = p * w_i:
 *     a' = magnitude * (a cos t - b sin t),  b' = magnitude * (a sin t + b cos t)
 * Pair i of a head, i < rotary_dim / 2, is elements (i, i + rotary_dim/2) in the
 * half layout and (2i, 2i + 1) in the interleaved one.  Elements from rotary_dim
 * on are not rotated.  The norm of one head of D elements, before the rotation:
 *     inv_rms = 1/sqrt(mean_D(x^2) + eps),   n = gamma * x * inv_rms
 * with one gamma [D] for all query heads and one for all key heads.
 * All arithmetic is fp32, rounded once to the storage type.
 */

/* One tensor of heads, [batch, seq, heads, head_dim]: element (b, s, h, d) is at
 * data + b*stride_batch + s*stride_seq + h*stride_head + d, in elements.  Strides
 * are >= 0 and those of a size of 1 are ignored, so that any of [batch, seq,
 * heads, dim], [batch, heads, seq, dim] and a slice of a joint projection's output
 * can be passed as they are; a 0 stride repeats an input.  heads <= 1,048,576. */
typedef struct tb_heads {
    void* data;
    int64_t stride_batch, stride_seq, stride_head;
    int64_t heads;
} tb_heads;

typedef enum tb_rope_layout {
    TB_ROPE_HALF = 0,         /* pairs (i, i + rotary_dim/2) */
    TB_ROPE_INTERLEAVED = 1   /* pairs (2i, 2i + 1)          */
} tb_rope_layout;

/* How a call turns positions into angles. */
typedef struct tb_rope_angles {
    const uint64_t* freqs;     /* device [rotary_dim/2]: the part of a turn that one
                                  position adds, in 2^-64 turn (tb_rope_freqs); 8-byte
                                  aligned; may be NULL when rotary_dim is 0         */
    const int64_t* positions;  /* device: position of (b, s) at b*positions_stride + s,
                                  8-byte aligned; NULL: s                            */
    int64_t positions_stride;  /* 0: one row for every batch entry, else >= seq      */
    int64_t offset;            /* added to every position                            */
    int rotary_dim;            /* even, 0 .. head_dim                                */
    tb_rope_layout layout;
    float magnitude;           /* factor on sines and cosines, finite; usually 1     */
} tb_rope_angles;

typedef enum tb_rope_scale_kind {
    TB_ROPE_SCALE_NONE = 0,
    TB_ROPE_SCALE_LINEAR = 1,      /* every frequency divided by factor              */
    TB_ROPE_SCALE_NTK = 2,         /* base * factor^(rotary_dim / (rotary_dim - 2))  */
    TB_ROPE_SCALE_YARN = 3,        /* pairs making more than `fast` turns over
                                      original_context keep their frequency, pairs
                                      making fewer than `slow` are divided by factor,
                                      a linear blend over the pair's index between;
                                      magnitude 0.1 ln(factor) + 1                   */
    TB_ROPE_SCALE_WAVELENGTH = 4   /* the same with the blend linear in the turns and
                                      magnitude 1                                    */
} tb_rope_scale_kind;

typedef struct tb_rope_scaling {
    tb_rope_scale_kind kind;
    double factor;             /* >= 1 */
    double original_context;   /* YARN, WAVELENGTH: positions trained on, > 0        */
    double fast, slow;         /* YARN, WAVELENGTH: turns, fast > slow > 0           */
} tb_rope_scaling;

/*
 * tb_rope_freqs -- fill a host table with the frequencies base^(-2i/rotary_dim)
 * radians per position, scaled for a longer context, as whole 2^-64 parts of a
 * turn.  p * freq in wrapping 64-bit arithmetic is the angle of position p modulo
 * one turn exactly, however far p is.  Needs no GPU; copy the table to the device.
 *   rotary_dim  even, 0 .. 1024
 *   base        > 0 (10000 is usual), > 1 with YARN
 *   scaling     NULL: none
 *   freqs       out: host [rotary_dim/2]
 *   magnitude   out: the value for tb_rope_angles.magnitude
 * Errors: TB_ERR_INVALID_VALUE.
 */
tb_status tb_rope_freqs(int rotary_dim, double base, const tb_rope_scaling* scaling,
                        uint64_t* freqs, float* magnitude);

/*
 * tb_rope -- rotate queries and keys; tb_rope_bwd -- its gradient, the transposed
 * rotation (also scaled by magnitude), which needs no forward values.
 *   q, k            inputs; k may be NULL (then k_out is NULL too)
 *   q_out, k_out    outputs with as many heads as their input.  An output may be the
 *                   very same rows as its input (a call in place); otherwise it must
 *                   share no element with any input or output.  Views that walk one
 *                   buffer with the same strides are told apart exactly; views with
 *                   different strides count as sharing when their address ranges meet.
 *   batch, seq      >= 0, batch * seq < 2^31; nothing is enqueued when either is 0.
 *                   Elements of a buffer outside the views are not touched.
 *   head_dim        1 .. 1024
 *   dtype           TB_F32, TB_BF16 or TB_F16, of all four
 * Heads are read by vectors of 16 bytes, 8 bytes or two elements, the widest for which
 * head_dim and rotary_dim are multiples of two vectors and pointers and strides of one:
 * 16-bit heads of up to 512, 256 and 256 elements, fp32 heads of up to 256 (16 bytes) and
 * 256 (two elements).  Others take a general kernel, one element at a time.  The sines of
 * 16-bit calls are good to 2^-20, those of fp32 calls to fp32 accuracy.
 * Errors: TB_ERR_INVALID_VALUE, TB_ERR_UNSUPPORTED_DTYPE, TB_ERR_MISALIGNED,
 * TB_ERR_ALIAS, TB_ERR_CUDA.
 */
tb_status tb_rope(const tb_heads* q, const tb_heads* k, const tb_heads* q_out,
                  const tb_heads* k_out, int64_t batch, int64_t seq, int64_t head_dim,
                  const tb_rope_angles* angles, tb_dtype dtype, void* stream);

tb_status tb_rope_bwd(const tb_heads* dq_out, const tb_heads* dk_out, const tb_heads* dq,
                      const tb_heads* dk, int64_t batch, int64_t seq, int64_t head_dim,
                      const tb_rope_angles* angles, tb_dtype dtype, void* stream);

/*
 * tb_qk_norm_rope -- the per-head RMS norm of queries and keys and their rotation
 * in one pass.  As tb_rope, with
 *   gamma_q, gamma_k       fp32 [head_dim]; gamma_k may be NULL when k is
 *   eps                    >= 0
 *   inv_rms_q, inv_rms_k   out: fp32 [batch, seq, heads], contiguous, what the
 *                          gradient needs; either may be NULL (serving)
 * rotary_dim = 0 gives the norm alone.  A head of zeros gives inv_rms = 1/sqrt(eps)
 * and zeros (NaN when eps is 0).
 */
tb_status tb_qk_norm_rope(const tb_heads* q, const tb_heads* k, const float* gamma_q,
                          const float* gamma_k, float eps, const tb_heads* q_out,
                          const tb_heads* k_out, float* inv_rms_q, float* inv_rms_k,
                          int64_t batch, int64_t seq, int64_t head_dim,
                          const tb_rope_angles* angles, tb_dtype dtype, void* stream);

/*
 * tb_qk_norm_rope_bwd -- its gradient.  With dn the transposed rotation of dq_out,
 * xhat = x * inv_rms and dxhat = dn * gamma, for queries and keys alike:
 *     dq       = inv_rms * (dxhat - xhat * mean_D(dxhat * xhat))
 *     dgamma_q = sum over batch, seq and heads of dn * xhat   (overwritten)
 * dgamma is reduced in a fixed order: results are bitwise reproducible.
 *   dq_out, dk_out   gradients of the forward's outputs
 *   q, k             the forward's inputs, inv_rms_q, inv_rms_k what it saved
 *   dq, dk           outputs; each may be the same rows as its dq_out or its q
 *   workspace        device scratch of tb_qk_norm_rope_bwd_workspace_size() bytes,
 *                    16-byte aligned, contents ignored.  Calls that may run at the
 *                    same time need workspaces of their own.
 * No token or no head writes zeros to dgamma.
 * Errors: as tb_rope, plus TB_ERR_WORKSPACE.
 */
tb_status tb_qk_norm_rope_bwd_workspace_size(int64_t batch, int64_t seq, int64_t heads_q,
                                             int64_t heads_k, int64_t head_dim,
                                             tb_dtype dtype, size_t* bytes);

tb_status tb_qk_norm_rope_bwd(const tb_heads* dq_out, const tb_heads* dk_out,
                              const tb_heads* q, const tb_heads* k,
                              const float* inv_rms_q, const float* inv_rms_k,
                              const float* gamma_q, const float* gamma_k,
                              const tb_heads* dq, const tb_heads* dk,
                              float* dgamma_q, float* dgamma_k,
                              int64_t batch, int64_t seq, int64_t head_dim,
                              const tb_rope_angles* angles, tb_dtype dtype,
                              void* workspace, size_t workspace_bytes, void* stream);

/* ======================================================================== */
/* Softmax cross entropy of a linear output layer                            */
/* ======================================================================== */
/*
 * The loss at a decoder's output without its logits in memory.  With hidden states
 * H [rows, D] and output weights W [vocab, D], logits l = H W^T:
 *     lse  = log sum_v exp(l_v)
 *     loss = lse - l[target]
 * and, for the gradient dloss of each row's loss,
 *     G  = exp(l - lse) - onehot(target)
 *     dH = dloss * (G W),   dW = G^T (dloss * H)
 * The loss keeps the logits in accumulators only; the gradient forms them again, one
 * piece of the vocabulary at a time, and holds one piece of G (rounded to dtype) in the
 * workspace, at most about 256 MiB unless rows exceeds 65,536 (then 4,096 bytes a row).  Beside
 * G the gradient's workspace holds a copy of H, fp32 sums of dH (rows * D * 4 bytes, times the
 * parts that the vocabulary is split into) where it takes several pieces or parts, and fp32 sums
 * of dW (a piece's columns * D * 4 bytes, times the parts of the rows) where the rows are split.
 * Both calls' workspaces hold padded copies of H and W where D is not a multiple of 8.  (The
 * pages take the softmax backward on stored probabilities: tb_softmax_bwd.)
 *
 * A row whose target is ignore_index takes no part, whatever its H is: its loss is +0, its
 * dH is 0 and it adds nothing to dW.  Its lse is written.  A target outside [0, vocab) that
 * is not ignore_index gives a loss of NaN and the gradient of an ignored row, and the forward
 * call sets the device error word to TB_ERR_INVALID_VALUE (tb_device_error).  A row with a
 * dloss of 0 takes no part in the gradient either.  A logit of +inf gives lse = +inf.
 *
 * tb_linear_xent
 *   H, W             device [rows, D] and [vocab, D], TB_BF16 or TB_F16, 16-byte aligned; 2-byte
 *                    where D is not a multiple of 8 (rows of such a matrix start on any element)
 *   targets          device int64 [rows]
 *   loss, lse        out: fp32 [rows]
 *   ignore_index     any value; -100 is usual
 *   workspace        device scratch of tb_linear_xent_workspace_size() bytes, 16-byte
 *                    aligned, contents ignored.  Calls that may run at the same time need
 *                    workspaces of their own, and so do graphs that may.
 * tb_linear_xent_bwd
 *   dloss            fp32 [rows]: gradient of each row's loss (for a mean over the rows
 *                    that count, 1 / their number)
 *   lse              what the forward call wrote
 *   dH, dW           out: [rows, D] and [vocab, D] in dtype, overwritten; either may be
 *                    NULL when it is not wanted
 * Sums are fp32, in the tensor cores' accumulators, which truncate: a sum of n terms of one sign
 * comes out smaller by about 1e-9 n of itself, where n is at most 1,280 in the loss's logits and
 * 65,536 in dH and dW (longer sums are added from such parts), and D in the logits that the
 * gradient forms again for G, whose own rounding is far above that.  Results are bitwise reproducible on one device
 * model.  Two values are
 * rounded to dtype on the way: G, and for dW the rows of H times dloss / max |dloss| (exact
 * where every dloss is the same, as for a mean).  TB_F16 holds G times 2^14, so that
 * probabilities down to 2^-38 count; of a dloss that is an 8th of the largest or less up to eight
 * powers of two go into G instead of H (probabilities down to 2^-30), so that elements of H around 1
 * keep their bits with weights 2^22 below the largest.
 * Logits of any size are taken, -1e10 or the type's lowest value as a mask among them; an lse so
 * large that fp32 has no place for the logarithm beside it is the row's largest logit.
 * Results must not overlap inputs, each other or the workspace.  rows == 0 writes zeros to
 * dW and nothing else.
 * Errors: TB_ERR_INVALID_VALUE (null or negative; D or vocab below 1; rows, D or vocab above
 * 2^24, rows * D or vocab * D above 2^40; dH and dW both NULL),
 * TB_ERR_UNSUPPORTED_DTYPE (TB_F32 has no such tensor-core product), TB_ERR_MISALIGNED,
 * TB_ERR_ALIAS, TB_ERR_WORKSPACE, TB_ERR_CUDA.
 */
tb_status tb_linear_xent_workspace_size(int64_t rows, int64_t D, int64_t vocab,
                                        tb_dtype dtype, size_t* bytes);

tb_status tb_linear_xent(const void* H, const void* W, const int64_t* targets,
                         float* loss, float* lse, int64_t rows, int64_t D, int64_t vocab,
                         int64_t ignore_index, tb_dtype dtype,
                         void* workspace, size_t workspace_bytes, void* stream);

tb_status tb_linear_xent_bwd_workspace_size(int64_t rows, int64_t D, int64_t vocab,
                                            tb_dtype dtype, size_t* bytes);

tb_status tb_linear_xent_bwd(const float* dloss, const void* H, const void* W,
                             const int64_t* targets, const float* lse, void* dH, void* dW,
                             int64_t rows, int64_t D, int64_t vocab, int64_t ignore_index,
                             tb_dtype dtype, void* workspace, size_t workspace_bytes,
                             void* stream);

/* ======================================================================== */
/* Causal attention over whole prompts                                       */
/* ======================================================================== */
/*
 * The attention product between the rotated queries and keys and the output projection, without
 * the scores in memory.  (The pages take attention's softmax backward on stored probabilities:
 * tb_softmax_bwd_causal.)  For token i of a sequence and the tokens j <= i of the same one:
 *     s_ij  = scale * q_i . k_j,   lse_i = log sum_j exp(s_ij)
 *     out_i = sum_j exp(s_ij - lse_i) v_j
 * for every query head; heads_q / heads_k query heads in a row share a head of k and v.
 *
 * A sequence is one batch entry, or, with offsets, a run of tokens of the one row: sequence i is
 * tokens offsets[i] .. offsets[i + 1] - 1, any number of them, 0 and 1 included.  Tokens before the
 * first or behind the last sequence are not written, and whatever they hold (NaN included) reaches
 * no other token; nor does a token reach another sequence's.  Within a sequence k and v are finite:
 * an infinity or NaN may reach the results of up to 255 tokens before it.  Offsets that do not count
 * up within 0 .. seq set the device error word to TB_ERR_INVALID_VALUE (tb_device_error): of a sequence
 * with tokens or without, each pair of them is looked at.  Their sequences are cut to the row, and
 * what that call leaves in out and lse, or in the gradients, is undefined; nothing else is written.
 *
 * tb_attention
 *   q, k, v          [batch, seq, heads, head_dim] by tb_heads; k and v have the same number of
 *                    heads, a divisor of q's
 *   out              as many heads as q; shares no element with q, k or v
 *   lse              out: fp32 [batch, heads_q, seq], contiguous, what the gradient needs; NULL
 *                    when it is not wanted (serving)
 *   batch, seq       >= 0, batch <= 2^20, seq <= 2^25
 *   head_dim         a multiple of 8, 8 .. 128
 *   offsets          device int64 [sequences + 1], 8-byte aligned; NULL: every batch entry is a
 *                    sequence (sequences is 0 then).  With offsets batch is 1 and sequences <= 2^24.
 *   scale            > 0, <= 2^127; 1 / sqrt(head_dim) is usual
 *   dtype            TB_BF16 or TB_F16
 * Data starts on 16 bytes and strides are multiples of 8 elements, not 0 (except of a size of 1)
 * and below 2^39.
 * Sums are fp32.  P = exp(s - m), m the maximum of keys before or one that is at most ln 8192 below it, is
 * rounded to dtype on its way into the second product; the sum below it is not.  (TB_F16: below 2^-14 P has fewer
 * bits, each key's is off by 2^-25 at most.)  Scores may be of any size: fp32 holds them, m is taken off before the
 * power, and keys whose scores lie far below the others' or overflow to -inf take no part.  lse is m rounded to fp32, and
 * with the logarithm of the sum rounded once more.  Results are bitwise reproducible.
 * Errors: TB_ERR_INVALID_VALUE, TB_ERR_UNSUPPORTED_DTYPE (TB_F32 has no such tensor-core product),
 * TB_ERR_MISALIGNED, TB_ERR_ALIAS, TB_ERR_CUDA.
 */
tb_status tb_attention(const tb_heads* q, const tb_heads* k, const tb_heads* v, const tb_heads* out,
                       float* lse, int64_t batch, int64_t seq, int64_t head_dim,
                       const int64_t* offsets, int64_t sequences, float scale, tb_dtype dtype,
                       void* stream);

/*
 * tb_attention_bwd -- its gradient.  With p_ij = exp(s_ij - lse_i):
 *     dp_ij = dout_i . v_j,   ds_ij = p_ij (dp_ij - dout_i . out_i)
 *     dv_j = sum_i p_ij dout_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j
 * dk and dv are summed over the query heads that share a key head.
 *   dout             gradient of out
 *   q, k, v          the forward's inputs; out, lse: what it wrote
 *   dq, dk, dv       out: as q, k and v, overwritten; they share no element with an input or with
 *                    each other (views of one joint buffer are told apart)
 *   workspace        device scratch of tb_attention_bwd_workspace_size() bytes, 16-byte aligned,
 *                    contents ignored: 8 bytes a row of out, and, where tiles of keys are too few
 *                    for the machine, fp32 sums of dk and dv from several pieces of the query
 *                    heads that share a key head.  Calls that may run at the same time need workspaces of
 *                    their own, and so do graphs that may.
 * Other arguments, sequences, alignment and errors as tb_attention, plus TB_ERR_WORKSPACE; q and dout
 * are finite within a sequence as k and v are.  Sums are fp32; P and dS are rounded to dtype on their way
 * into the last three products.  TB_F16 holds P times 2^14, and dS times a power of two by the largest
 * norms of a row of dout and of v, so that small gradients keep their bits.  Where |lse| is above 1,024
 * a score is rounded to fp32 and lse taken off before the power.  Every sum is taken in a
 * fixed order: results are bitwise reproducible.
 */
tb_status tb_attention_bwd_workspace_size(int64_t batch, int64_t seq, int64_t heads_q,
                                          int64_t heads_k, int64_t head_dim, tb_dtype dtype,
                                          size_t* bytes);

tb_status tb_attention_bwd(const tb_heads* dout, const tb_heads* q, const tb_heads* k,
                           const tb_heads* v, const tb_heads* out, const float* lse,
                           const tb_heads* dq, const tb_heads* dk, const tb_heads* dv,
                           int64_t batch, int64_t seq, int64_t head_dim, const int64_t* offsets,
                           int64_t sequences, float scale, tb_dtype dtype, void* workspace,
                           size_t workspace_bytes, void* stream);

/* ======================================================================== */
/* Gated feed-forward projections                                            */
/* ======================================================================== */
/*
 * The first half of a gated feed-forward block, both projections with the activation and
 * the product in one pass, and its gradient.  (The pages have no counterpart.)  With inputs
 * X [rows, D] and weights Wg, Wu [F, D]:
 *     G = X Wg^T,  U = X Wu^T,  H = act(G) * U
 * and, for the gradient dH,
 *     dG = dH * U * act'(G),  dU = dH * act(G)
 *     dX = dG Wg + dU Wu,  dWg = dG^T X,  dWu = dU^T X
 * The block's last projection is a plain matrix product.
 */
typedef enum tb_activation {
    TB_ACT_SILU = 0,          /* x / (1 + exp(-x))                                        */
    TB_ACT_GELU = 1,          /* x (1 + erf(x / sqrt(2))) / 2                             */
    TB_ACT_GELU_TANH = 2      /* x (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) / 2        */
} tb_activation;

/*
 * tb_gated_linear
 *   X, Wg, Wu        device [rows, D], [F, D] and [F, D], TB_BF16 or TB_F16; halves of one
 *                    weight [2 F, D] are taken as they are
 *   H                out: [rows, F]
 *   G, U             out: [rows, F], rounded to dtype, what the gradient needs; both NULL
 *                    when it is not wanted (H is formed from the unrounded sums either way)
 *   workspace        device scratch of tb_gated_linear_workspace_size() bytes, 16-byte
 *                    aligned, contents ignored; may be NULL when that is 0.  It holds fp32
 *                    sums of G and U where few tiles make the call split the contraction.
 *                    Calls that may run at the same time need workspaces of their own, and
 *                    so do graphs that may.
 * tb_gated_linear_bwd
 *   dH               [rows, F]: gradient of H
 *   G, U             what the forward call kept
 *   dX, dWg, dWu     out: [rows, D], [F, D] and [F, D], overwritten; dX, or dWg and dWu
 *                    together, may be NULL when they are not wanted
 *   workspace        as above, of tb_gated_linear_bwd_workspace_size() bytes.  It holds dG
 *                    and dU (4 bytes an element of H) and fp32 sums of results whose
 *                    contraction is split.
 * D and F are multiples of 8 and every buffer is 16-byte aligned.  Sums are fp32, in the tensor
 * cores' accumulators, which truncate: a sum of n terms of one sign comes out smaller by about
 * 1e-9 n of itself, n at most 65,536 (longer sums are added from such parts).  dG and dU are
 * rounded to dtype on their way into the products; TB_F16 holds them times a power of two that
 * brings the largest of them to 2^14 .. 2^15, so that small gradients keep their bits.  Results
 * are bitwise reproducible on one device model.  Results must not overlap inputs, each other or
 * the workspace.  rows == 0 writes zeros to dWg and dWu and nothing else.
 * Errors: TB_ERR_INVALID_VALUE (null or negative; D or F no multiple of 8 or below 8; rows, D or
 * F above 2^24, a product of two of them above 2^38; only one of G and U, or of dWg and dWu;
 * no result wanted; unknown activation), TB_ERR_UNSUPPORTED_DTYPE (TB_F32 has no such tensor-core
 * product), TB_ERR_MISALIGNED, TB_ERR_ALIAS, TB_ERR_WORKSPACE, TB_ERR_CUDA.
 */
tb_status tb_gated_linear_workspace_size(int64_t rows, int64_t D, int64_t F, tb_dtype dtype,
                                         size_t* bytes);

tb_status tb_gated_linear(const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U,
                          int64_t rows, int64_t D, int64_t F, tb_activation act, tb_dtype dtype,
                          void* workspace, size_t workspace_bytes, void* stream);

tb_status tb_gated_linear_bwd_workspace_size(int64_t rows, int64_t D, int64_t F, tb_dtype dtype,
                                             size_t* bytes);

tb_status tb_gated_linear_bwd(const void* dH, const void* X, const void* Wg, const void* Wu,
                              const void* G, const void* U, void* dX, void* dWg, void* dWu,
                              int64_t rows, int64_t D, int64_t F, tb_activation act,
                              tb_dtype dtype, void* workspace, size_t workspace_bytes,
                              void* stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* TB_H_ */
