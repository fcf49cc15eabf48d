/*
 * ssim_train_amd.h -- C ABI of the training step's operators around the SSIM
 * loss, for AMD Instinct MI355X (gfx950): the global gradient norm and
 * clipping by it, AdamW, and the joint between two blocks of an image network
 * (the norm after a block, its gate, the scaled residual sum and the norm
 * before the next block) with its gradient.
 *
 * Conventions, as in ssim_loss_amd.h:
 *   - Tensors are device pointers owned by the caller, contiguous, aligned to
 *     their element size.  Element counts and offsets are 64-bit.  The library
 *     never allocates device memory, frees or synchronises; all work is
 *     enqueued on `stream` (a hipStream_t; NULL is the default stream).
 *   - `items` and `in` are host memory, read before the call returns.
 *   - Every argument check happens before any HIP call; a failed check returns
 *     a negative SSIM_ERR_* code (ssim_train_strerror) and enqueues nothing.
 *     No C++ exception crosses the ABI.
 *   - Workspaces need no initialisation and hold nothing between calls.  Calls
 *     that may overlap in time need distinct ones.
 *   - The launches are kernels only, so every call may be captured in a HIP
 *     graph.  Results are deterministic: the same inputs give the same bits.
 *   - Element types are SSIM_DTYPE_F32, _F16 and _BF16.  Arithmetic is fp32,
 *     sums of squares over tensors fp64; each output is rounded once, to
 *     nearest even.
 */
#ifndef SSIM_TRAIN_AMD_H
#define SSIM_TRAIN_AMD_H

#include <stddef.h>
#include <stdint.h>

#include "ssim_loss_amd.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSIM_TRAIN_ABI_VERSION 1

/* a code beside SSIM_ERR_*: a hyperparameter (max_norm, lr, beta1, beta2, eps,
 * weight_decay, gate_act) is not a number or out of its range */
enum { SSIM_ERR_VALUE = -10 };

int ssim_train_abi_version(void);

/* Static text for a return code of this header's calls.  Never NULL. */
const char* ssim_train_strerror(int code);

/* ---------------------------------------------------------------------------
 * Gradients of many tensors.
 *   norm = sqrt(sum over all tensors and elements of g^2)
 *   c    = min(1, max_norm / (norm + 1e-6))
 *   out  = c g
 * The sum runs in fp64, so neither large nor tiny gradients over- or underflow
 * in it.  A NaN or infinite gradient makes the norm NaN or infinite; then c is
 * NaN or 0, and the outputs follow the formula (0 times infinity is NaN).
 */
typedef struct {
  const void* grad; /* n elements of `dtype` */
  void* out;        /* n elements of `dtype`; may be `grad` itself */
  int64_t n;        /* 0: the item is skipped and its pointers are not looked at */
  int32_t dtype;
  int32_t reserved; /* 0 */
} ssim_clip_item;

/* Bytes of the workspace of the three calls below (8-byte aligned).  Host-only. */
size_t ssim_update_workspace_bytes(void);

/* Writes the norm (fp32) to `norm` (device) and c * grad to every item's out.
 * An out may be its own grad; it must not otherwise overlap any item's arrays,
 * the norm or the workspace.
 *   max_norm : finite, >= 0
 * SSIM_ERR_SHAPE: count or n negative, a pointer not aligned to its element
 * size or the workspace not to 8 bytes; SSIM_ERR_OVERFLOW: sizes past 2^46
 * bytes; also SSIM_ERR_NULL, _DTYPE, _VALUE, _ALIAS, _DEVICE, _HIP. */
int ssim_clip_grads(const ssim_clip_item* items, int64_t count, double max_norm, float* norm,
                    void* workspace, void* stream);

/* The norm alone: `out` and `max_norm` do not take part. */
int ssim_grad_norm(const ssim_clip_item* items, int64_t count, float* norm, void* workspace,
                   void* stream);

/* One AdamW update of every item, its gradients clipped by their global norm:
 *   g' = c g                       (c as above; 1 without clipping)
 *   m  = beta1 m + (1 - beta1) g'
 *   v  = beta2 v + (1 - beta2) g'^2
 *   w  = (1 - lr weight_decay) w - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * with t the number of updates including this one.
 */
typedef struct {
  const void* grad;  /* n elements of grad_dtype */
  void* param;       /* n elements of param_dtype */
  float* exp_avg;    /* m: n fp32 */
  float* exp_avg_sq; /* v: n fp32 */
  float* master;     /* the weights w in fp32, of which param receives a rounded
                        copy; NULL: param holds the weights */
  int64_t n;         /* 0: skipped */
  int32_t grad_dtype; /* param_dtype or SSIM_DTYPE_F32 */
  int32_t param_dtype;
} ssim_adamw_item;

typedef struct {
  double lr;           /* >= 0; not looked at if lr_device is given */
  double beta1, beta2; /* in [0, 1); they and their complements enter in fp32 */
  double eps;          /* >= 0 */
  double weight_decay; /* >= 0 */
  double max_norm;     /* >= 0; infinity: no clipping */
  const float* lr_device; /* NULL, or the learning rate on the device (a captured
                             graph then follows a schedule) */
} ssim_adamw_options;

/*   step : device int64[2], the number of updates done before this one, to which
 *          the call adds one, and a word of the library's that is 0 before the
 *          first call and after every call
 *   norm : device fp32, receives the gradients' norm before clipping; may be
 *          NULL if max_norm is infinite
 * No array of an item may overlap another array of any item, the step, the
 * norm or the workspace.  Codes as for ssim_clip_grads. */
int ssim_adamw_step(const ssim_adamw_item* items, int64_t count, const ssim_adamw_options* options,
                    int64_t* step, float* norm, void* workspace, void* stream);

/* ---------------------------------------------------------------------------
 * The joint between two blocks of a network.  For each of `rows` rows of
 * `width` elements, with mean over the row:
 *   bh       = branch / sqrt(mean(branch^2) + eps)
 *   residual = x + act(gate) scale post_weight bh
 *   normed   = residual / sqrt(mean(residual^2) + eps) pre_weight
 * (normed is formed from the residual before that is rounded).
 */
enum {
  SSIM_GATE_NONE = 0,   /* act(g) = g */
  SSIM_GATE_SIGMOID = 1 /* act(g) = 1 / (1 + exp(-g)) */
};

#define SSIM_BLOCK_NORM_MAX_WIDTH 16384

typedef struct {
  const void* x;            /* [rows, width] of x_dtype: the residual stream */
  const void* branch;       /* [rows, width] of branch_dtype: the block's output */
  const void* gate;         /* [rows / gate_rows, width] of branch_dtype, or NULL: 1 */
  const float* scale;       /* [width] fp32, or NULL: 1 */
  const float* post_weight; /* [width] fp32, or NULL: 1 */
  const float* pre_weight;  /* [width] fp32, or NULL: 1 */
  int64_t rows;             /* >= 0 */
  int64_t width;            /* 1 .. SSIM_BLOCK_NORM_MAX_WIDTH */
  int64_t gate_rows;        /* consecutive rows that share one row of the gate; divides rows */
  double eps;               /* >= 0 */
  int32_t x_dtype;          /* branch_dtype or SSIM_DTYPE_F32 */
  int32_t branch_dtype;
  int32_t gate_act;         /* SSIM_GATE_* */
  int32_t reserved;         /* 0 */
} ssim_block_norm_inputs;

/* residual: [rows, width] of x_dtype; normed: [rows, width] of branch_dtype;
 * stats: NULL, or [rows, 2] fp32 that receives the two reciprocal roots of
 * each row, for the backward.  Outputs overlap neither inputs nor each other.
 * SSIM_ERR_SHAPE also: rows, width or gate_rows out of range. */
int ssim_block_norm_forward(const ssim_block_norm_inputs* in, void* residual, void* normed,
                            float* stats, void* stream);

/* Bytes of the backward's workspace (16-byte aligned) for these inputs (only
 * sizes, types and whether gate is NULL are looked at).  0 for invalid
 * arguments or rows = 0.  Host-only. */
size_t ssim_block_norm_workspace_bytes(const ssim_block_norm_inputs* in);

/* The gradients for the upstream gradients d_residual (x_dtype) and d_normed
 * (branch_dtype), both [rows, width]; either may be NULL: 0.  `stats` is what
 * the forward wrote for the same inputs.  Each gradient has its input's shape
 * and type and may be NULL: not wanted.  Sums over rows run in fp32 within a
 * workgroup's rows and in fp64 over the workgroups, in a fixed order. */
typedef struct {
  void* x;
  void* branch;
  void* gate;
  float* scale;
  float* post_weight;
  float* pre_weight;
} ssim_block_norm_grads;

int ssim_block_norm_backward(const ssim_block_norm_inputs* in, const float* stats,
                             const void* d_residual, const void* d_normed,
                             const ssim_block_norm_grads* grads, void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSIM_TRAIN_AMD_H */
