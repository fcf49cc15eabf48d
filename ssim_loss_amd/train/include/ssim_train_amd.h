/*
 * ssim_train_amd.h -- C ABI of the training step's operators around the SSIM
 * loss, for AMD Instinct MI355X (gfx950): the global gradient norm and
 * clipping by it, AdamW, the joint between two blocks of an image network
 * (the norm after a block, its gate, the scaled residual sum and the norm
 * before the next block), and what lies inside a block: rotary positions,
 * attention and the gated layer; all with their gradients.
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

#define SSIM_TRAIN_ABI_VERSION 2

/* a code beside SSIM_ERR_*: a hyperparameter (max_norm, lr, beta1, beta2, eps,
 * weight_decay, gate_act, base, scale, act or another selector) is not a number
 * or out of its range */
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

/* ---------------------------------------------------------------------------
 * Rotary positions with several axes.  The first elements of each head are
 * split into parts, one to an axis, of axis_size[a] elements (even); what is
 * left behind them passes as it is.  Pair i of axis a turns by the angle
 * positions[.., a] base^(-2 i / axis_size[a]):
 *   y0 = x0 cos - x1 sin,  y1 = x1 cos + x0 sin
 * The angle is reduced in fp64, so positions may lie far out and between whole
 * numbers: it is off by at most 2^-50 of the position.
 */
enum {
  SSIM_PAIRS_ADJACENT = 0, /* elements 2 i and 2 i + 1 of the part */
  SSIM_PAIRS_HALVES = 1    /* elements i and i + axis_size / 2 */
};
enum { SSIM_POSITION_F32 = 0, SSIM_POSITION_I32 = 1, SSIM_POSITION_I64 = 2 };

#define SSIM_ROTARY_MAX_AXES 4
#define SSIM_ROTARY_MAX_DIM 512

typedef struct {
  const void* q;         /* [batch, tokens, q_heads, dim] of dtype */
  const void* k;         /* [batch, tokens, k_heads, dim], or NULL: queries alone */
  const void* positions; /* [batch, tokens, axes] of position_type, the axes beside each other */
  int64_t q_stride[3];   /* elements from one batch entry, token, head to the next, >= 0 */
  int64_t k_stride[3];
  int64_t position_stride[2]; /* ... of batch entries and tokens */
  int64_t batch, tokens; /* >= 0 */
  int32_t q_heads, k_heads, dim; /* 1 .. 65536, 1 .. 65536, 1 .. SSIM_ROTARY_MAX_DIM */
  int32_t axes;          /* 1 .. SSIM_ROTARY_MAX_AXES */
  int32_t axis_size[SSIM_ROTARY_MAX_AXES];
  int32_t pairs;         /* SSIM_PAIRS_* */
  int32_t position_type; /* SSIM_POSITION_* */
  int32_t dtype;
  int32_t inverse;       /* 1: by the opposite angle, which is the gradient's way */
  double base;           /* > 0 */
} ssim_rotary_inputs;

/* q_out: [batch, tokens, q_heads, dim], contiguous; k_out likewise, or NULL
 * with k.  They overlap neither the inputs nor each other. */
int ssim_rotary(const ssim_rotary_inputs* in, void* q_out, void* k_out, void* stream);

/* ---------------------------------------------------------------------------
 * Softmax attention.  Query head h uses key head h / (heads / kv_heads).
 *   s_ij = scale q_i . k_j,  p_ij = exp(s_ij) / sum_j exp(s_ij),  out_i = sum_j p_ij v_j
 * over the keys that query i of sequence b sees: with ql = q_lengths[b] and
 * kl = k_lengths[b] (q_tokens and k_tokens without them; clamped to 0 .. tokens),
 * none if i >= ql, else j < kl and, with causal order, j <= i + kl - ql.  A query
 * that sees no key, or whose scores are all minus infinity, gives zeros, and a
 * query or key that takes no part has a gradient of zeros.  Queries past ql and
 * keys and values past kl are not read.  The others, and the gradient that arrives
 * at them, must be finite: what is not may reach rows that do not see it (scores of
 * minus infinity excepted).  A query whose largest s_ij is above 10^9 (fp16: 10^8)
 * gives NaN, and one whose all are as far below 0 zeros: fp32 does not tell them apart.
 * Scores, sums and statistics are fp32: a probability that the gradients form again
 * is off by some 2^-23 of its score, by a hundredth where scores are 10^5.  For half
 * types the probabilities and, in the gradients, their derivatives are rounded to the
 * type before the products.
 */
#define SSIM_ATTENTION_MAX_DIM 128

typedef struct {
  const void* q;       /* [batch, q_tokens, heads, dim] of dtype */
  const void* k;       /* [batch, k_tokens, kv_heads, dim] */
  const void* v;       /* [batch, k_tokens, kv_heads, dim] */
  const int32_t* q_lengths; /* [batch] on the device, or NULL */
  const int32_t* k_lengths;
  int64_t q_stride[3]; /* elements from one batch entry, token, head to the next; */
  int64_t k_stride[3]; /* each a multiple of 16 bytes, a token's at least dim and less */
  int64_t v_stride[3]; /* than 2^24 bytes, and q, k, v aligned to 16 bytes */
  int64_t batch, q_tokens, k_tokens; /* >= 0, tokens < 2^24 */
  int32_t heads, kv_heads; /* 1 .. 65536; kv_heads divides heads */
  int32_t dim;         /* a multiple of 8, to SSIM_ATTENTION_MAX_DIM */
  int32_t causal;
  int32_t dtype;
  int32_t reserved;    /* 0 */
  double scale;        /* > 0; at most 3.4e37 */
} ssim_attention_inputs;

/* Bytes of the workspace (16-byte aligned) of the forward; 0 also where it needs
 * none.  Host-only. */
size_t ssim_attention_workspace_bytes(const ssim_attention_inputs* in);

/* out: [batch, q_tokens, heads, dim], contiguous; lse: NULL, or fp32
 * [batch, heads, q_tokens] for the backward (log2 of the sum of exp(s_ij), plus
 * infinity for a query without keys); rest: NULL, or an array as out for the
 * backward, what out's rounding left (fp32: not looked at).  workspace may be NULL
 * where it needs none. */
int ssim_attention_forward(const ssim_attention_inputs* in, void* out, float* lse, void* rest,
                           void* workspace, void* stream);

/* Bytes of the backward's workspace (16-byte aligned).  Host-only. */
size_t ssim_attention_backward_workspace_bytes(const ssim_attention_inputs* in);

/* The gradients for d_out, laid out as out; out, lse and rest (fp32: not looked at)
 * are the forward's for the same inputs, and these and d_out are aligned to 16 bytes.  dq, dk, dv: contiguous, of q's, k's and v's shapes; each may be
 * NULL: not wanted.  No atomics: the same bits every time. */
int ssim_attention_backward(const ssim_attention_inputs* in, const void* out, const float* lse,
                            const void* rest, const void* d_out, void* dq, void* dk, void* dv, void* workspace,
                            void* stream);

/* ---------------------------------------------------------------------------
 * The gated layer of a feed-forward block:
 *   g = x w_gate^T + b_gate,  u = x w_up^T + b_up,  out = act(g) u
 */
enum {
  SSIM_ACT_SILU = 0,    /* g / (1 + exp(-g)) */
  SSIM_ACT_GELU = 1,    /* g (1 + erf(g / sqrt 2)) / 2 */
  SSIM_ACT_SIGMOID = 2  /* 1 / (1 + exp(-g)) */
};

typedef struct {
  const void* x;      /* [rows, width] */
  const void* w_gate; /* [hidden, width] */
  const void* w_up;   /* [hidden, width] */
  const void* b_gate; /* [hidden], or NULL: 0 */
  const void* b_up;
  int64_t rows;       /* >= 0 */
  int64_t width;      /* 1 .. 2^20 */
  int64_t hidden;     /* 1 .. 2^20 */
  int32_t act;        /* SSIM_ACT_* */
  int32_t dtype;      /* of all tensors */
} ssim_gated_linear_inputs;

/* Elements of each of the two arrays that the forward keeps for the backward. */
size_t ssim_gated_linear_saved_elements(const ssim_gated_linear_inputs* in);

/* Bytes of the workspace (16-byte aligned) of the forward, 0 also where it needs
 * none, and of the backward.  Host-only. */
size_t ssim_gated_linear_workspace_bytes(const ssim_gated_linear_inputs* in);
size_t ssim_gated_linear_backward_workspace_bytes(const ssim_gated_linear_inputs* in);

/* out: [rows, hidden].  g, u: NULL, or 16-byte aligned arrays of
 * ssim_gated_linear_saved_elements floats that receive g and u for the backward. */
int ssim_gated_linear_forward(const ssim_gated_linear_inputs* in, void* out, float* g, float* u,
                              void* workspace, void* stream);

/* The gradients for d_out ([rows, hidden]), each of its input's shape; NULL: not
 * wanted.  Those of g and u are rounded to dtype before the products (fp16: times a
 * power of two, by which the products' sums are divided, that brings the largest of
 * them that is finite into its range). */
typedef struct {
  void* x;
  void* w_gate;
  void* w_up;
  void* b_gate;
  void* b_up;
} ssim_gated_linear_grads;

int ssim_gated_linear_backward(const ssim_gated_linear_inputs* in, const float* g, const float* u,
                               const void* d_out, const ssim_gated_linear_grads* grads,
                               void* workspace, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSIM_TRAIN_AMD_H */
