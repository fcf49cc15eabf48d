// attention_api.hip -- host side of attention: argument checks, the split of the
// work, launches.

#include "attention.hpp"

namespace {

using namespace ssim_train;

constexpr int64_t kMaxTokens = (int64_t)1 << 24;
constexpr int64_t kMaxStride = (int64_t)1 << 24;  // bytes between tokens: a tile's offsets stay below 2^32
constexpr int64_t kMaxBlocks = (int64_t)1 << 24;

const AttentionTable& table_of(int dtype) {
  switch (dtype) {
    case SSIM_DTYPE_F16: return attention_table_f16();
    case SSIM_DTYPE_BF16: return attention_table_bf16();
    default: return attention_table_f32();
  }
}

// A kernel's shape (AttentionTable's index), and how many workgroups a (batch, key
// head) takes: by its rows (queries of all heads that share the keys, or keys).
struct Shape {
  int shape, tiles;
  int threads() const { return shape == 1 ? 512 : 256; }
};
Shape shape_of(const void* const (&kernels)[3], int64_t rows, int64_t pairs, bool causal) {
  // Where 32 rows to a workgroup do not fill the GPU, its waves take the other axis in
  // turn: 2 x 257 x 6 x 64 fp32, gradients of queries 19.1, with 128 rows to one 40.3 us.
  if (rows <= 32 || ceil_div(rows, 32) * pairs <= kCUs) return {2, (int)ceil_div(rows, 32)};
  // Eight waves: half the caches' traffic, but coarser.  1 x 16384 x 16 x 128 bf16,
  // forward: 1948, of four waves 2044 us; causal, 4 x 4096: 183 and 156.
  if (kernels[1] && !causal && ceil_div(rows, 256) * pairs >= 4 * kCUs) return {1, (int)ceil_div(rows, 256)};
  return {0, (int)ceil_div(rows, 128)};
}

struct Plan {
  Shape forward, grad_q, grad_kv;
  int splits;  // of the forward's keys
};

Plan make_plan(const ssim_attention_inputs& in) {
  Plan p;
  const int64_t rows = in.q_tokens * (in.heads / in.kv_heads), pairs = in.batch * in.kv_heads;
  const AttentionTable& t = table_of(in.dtype);
  const int blocks = (in.dim - 1) / 32;
  p.forward = shape_of(t.forward[blocks], rows, pairs, in.causal);
  p.grad_q = shape_of(t.grad_q[blocks], rows, pairs, in.causal);
  p.grad_kv = shape_of(t.grad_kv[blocks], in.k_tokens, pairs, in.causal);
  // Few workgroups: each takes a part of the keys, 512 of them at least, and a second
  // launch joins the parts.
  const int64_t groups = p.forward.tiles * pairs;
  const int64_t target = p.forward.shape == 2 && in.dim * elem_bytes(in.dtype) > 128 ? kCUs : 2 * kCUs;
  const int64_t most = in.k_tokens / 512;
  int64_t splits = groups > 0 ? target / groups : 1;
  if (splits > most) splits = most;
  p.splits = splits < 1 ? 1 : (int)splits;
  return p;
}

bool stride_ok(const int64_t* s, const ssim_attention_inputs& in, int64_t tokens) {
  const int64_t bytes = elem_bytes(in.dtype);
  for (int k = 0; k < 3; ++k)
    if (s[k] < 0 || s[k] > (int64_t)1 << 44 || s[k] * bytes % 16 != 0) return false;
  return tokens <= 1 || (s[1] >= in.dim && s[1] * bytes < kMaxStride);
}

struct Spans {
  int64_t q, k, v;
  bool any_bad() const { return q < 0 || k < 0 || v < 0; }
};
Spans spans_of(const ssim_attention_inputs& in) {
  return {span(in.q_stride, in.batch, in.q_tokens, in.heads, in.dim),
          span(in.k_stride, in.batch, in.k_tokens, in.kv_heads, in.dim),
          span(in.v_stride, in.batch, in.k_tokens, in.kv_heads, in.dim)};
}

int check_inputs(const ssim_attention_inputs* in) {
  if (!in) return SSIM_ERR_NULL;
  if (!known_dtype(in->dtype)) return SSIM_ERR_DTYPE;
  if (in->causal < 0 || in->causal > 1) return SSIM_ERR_VALUE;
  if (!(in->scale > 0.0 && in->scale <= 3.4028234663852886e37)) return SSIM_ERR_VALUE;  // (times log2 e it is fp32's)
  if (in->batch < 0 || in->q_tokens < 0 || in->k_tokens < 0 || in->q_tokens >= kMaxTokens ||
      in->k_tokens >= kMaxTokens)
    return SSIM_ERR_SHAPE;
  if (in->heads < 1 || in->heads > 65536 || in->kv_heads < 1 || in->heads % in->kv_heads != 0) return SSIM_ERR_SHAPE;
  if (in->dim < 8 || in->dim > SSIM_ATTENTION_MAX_DIM || in->dim % 8 != 0) return SSIM_ERR_SHAPE;
  if (!stride_ok(in->q_stride, *in, in->q_tokens) || !stride_ok(in->k_stride, *in, in->k_tokens) ||
      !stride_ok(in->v_stride, *in, in->k_tokens))
    return SSIM_ERR_SHAPE;
  if (in->batch > 1 << 24) return SSIM_ERR_OVERFLOW;
  const int64_t pairs = in->batch * in->kv_heads, rows = in->q_tokens * (in->heads / in->kv_heads);
  // (a tile's end, too, is counted in 32 bits)
  if (rows > ((int64_t)1 << 31) - 512 || pairs > kMaxBlocks / kNormParts || pairs * rows > (int64_t)1 << 36 ||
      spans_of(*in).any_bad())
    return SSIM_ERR_OVERFLOW;
  const Plan p = make_plan(*in);
  if (pairs * p.forward.tiles * p.splits > kMaxBlocks || pairs * p.grad_q.tiles > kMaxBlocks ||
      pairs * p.grad_kv.tiles > kMaxBlocks)
    return SSIM_ERR_OVERFLOW;
  return SSIM_OK;
}

Strided strided(const void* p, const int64_t* s, int bytes) {
  return {static_cast<const char*>(p), s[0] * bytes, s[2] * bytes, (uint32_t)(s[1] * bytes)};
}

AttentionParams params_of(const ssim_attention_inputs& in, const Plan& plan) {
  AttentionParams p;
  memset(&p, 0, sizeof(p));
  const int bytes = elem_bytes(in.dtype);
  p.q = strided(in.q, in.q_stride, bytes);
  p.k = strided(in.k, in.k_stride, bytes);
  p.v = strided(in.v, in.v_stride, bytes);
  p.q_length = in.q_lengths;
  p.k_length = in.k_lengths;
  p.q_tokens = (int)in.q_tokens;
  p.k_tokens = (int)in.k_tokens;
  p.heads = in.heads;
  p.kv_heads = in.kv_heads;
  p.group = in.heads / in.kv_heads;
  p.dim = in.dim;
  p.batch = (int)in.batch;
  p.causal = in.causal;
  p.spread = in.batch * in.kv_heads % 8 == 0;
  p.scale = (float)frexp(in.scale, &p.scale_power);
  p.scale2 = (float)(in.scale * 1.4426950408889634);
  if (p.scale2 == 0.0f) p.scale2 = 0x1p-149f;  // (times any score it is next to nothing, and times minus infinity that)
  p.splits = plan.splits;
  p.tiles = plan.forward.tiles;
  return p;
}

size_t rows_of(const ssim_attention_inputs& in) { return (size_t)in.batch * in.heads * in.q_tokens; }
size_t delta_bytes(const ssim_attention_inputs& in) { return (rows_of(in) * 4 + 15) & ~(size_t)15; }
size_t norm_bytes(const ssim_attention_inputs& in) {
  return table_of(in.dtype).norms ? (size_t)in.batch * in.kv_heads * kNormParts * 8 : 0;
}

}  // namespace

extern "C" {

size_t ssim_attention_workspace_bytes(const ssim_attention_inputs* in) {
  if (check_inputs(in) != SSIM_OK) return 0;
  const Plan p = make_plan(*in);
  if (p.splits == 1) return 0;
  return (rows_of(*in) * p.splits * (in->dim + 1) * 4 + 15) & ~(size_t)15;
}

int ssim_attention_forward(const ssim_attention_inputs* in, void* out, float* lse, void* rest,
                           void* workspace, void* stream) {
  int rc = check_inputs(in);
  if (rc != SSIM_OK) return rc;
  if (in->batch == 0 || in->q_tokens == 0) return SSIM_OK;
  const size_t ws = ssim_attention_workspace_bytes(in), rows = rows_of(*in);
  if (!in->q || (in->k_tokens > 0 && (!in->k || !in->v)) || !out || (ws > 0 && !workspace)) return SSIM_ERR_NULL;
  const int bytes = elem_bytes(in->dtype);
  const Spans spans = spans_of(*in);
  const Array ins[] = {{in->q, (size_t)spans.q * bytes, 16},
                       {in->k, (size_t)spans.k * bytes, 16},
                       {in->v, (size_t)spans.v * bytes, 16},
                       {in->q_lengths, 4 * (size_t)in->batch, 4},
                       {in->k_lengths, 4 * (size_t)in->batch, 4}};
  const Array outs[] = {{out, rows * in->dim * bytes, bytes}, {lse, rows * 4, 4}, {rest, rows * in->dim * bytes, bytes},
                        {workspace, ws, ws ? 16 : 1}};
  rc = check_arrays(ins, 5, outs, 4);
  if (rc != SSIM_OK) return rc;
  rc = check_current_device();
  if (rc != SSIM_OK) return rc;

  const Plan plan = make_plan(*in);
  AttentionParams p = params_of(*in, plan);
  p.out = out;
  p.lse = lse;
  if (in->dtype != SSIM_DTYPE_F32) p.rest = rest;
  if (plan.splits > 1) {
    p.part_out = static_cast<float*>(workspace);
    p.part_lse = p.part_out + rows * plan.splits * in->dim;
  }
  const AttentionTable& t = table_of(in->dtype);
  const int blocks = (in->dim - 1) / 32;
  rc = launch(t.forward[blocks][plan.forward.shape],
              dim3((unsigned)(in->batch * in->kv_heads * plan.forward.tiles * plan.splits)), plan.forward.threads(), p, stream);
  if (rc != SSIM_OK || plan.splits == 1) return rc;
  return launch(t.join, dim3((unsigned)ceil_div(rows, kAttentionThreads / kWave)), kAttentionThreads, p, stream);
}

size_t ssim_attention_backward_workspace_bytes(const ssim_attention_inputs* in) {
  if (check_inputs(in) != SSIM_OK) return 0;
  return delta_bytes(*in) + norm_bytes(*in);
}

int ssim_attention_backward(const ssim_attention_inputs* in, const void* out, const float* lse,
                            const void* rest, const void* d_out, void* dq, void* dk, void* dv, void* workspace,
                            void* stream) {
  int rc = check_inputs(in);
  if (rc != SSIM_OK) return rc;
  if (in->batch == 0) return SSIM_OK;
  const bool any_q = in->q_tokens > 0, any_k = in->k_tokens > 0;
  if (!(any_q && dq) && !(any_k && (dk || dv))) return SSIM_OK;
  if (((any_q || ssim_attention_backward_workspace_bytes(in) > 0) && !workspace) ||
      (any_q && (!in->q || !out || !lse || !d_out || (in->dtype != SSIM_DTYPE_F32 && !rest))) || (any_k && (!in->k || !in->v)))
    return SSIM_ERR_NULL;
  const int bytes = elem_bytes(in->dtype);
  const Spans spans = spans_of(*in);
  const size_t rows = rows_of(*in), keys = (size_t)in->batch * in->k_tokens * in->kv_heads * in->dim * bytes;
  const size_t ws = ssim_attention_backward_workspace_bytes(in);
  const Array ins[] = {{in->q, (size_t)spans.q * bytes, 16},
                       {in->k, (size_t)spans.k * bytes, 16},
                       {in->v, (size_t)spans.v * bytes, 16},
                       {in->q_lengths, 4 * (size_t)in->batch, 4},
                       {in->k_lengths, 4 * (size_t)in->batch, 4},
                       {out, rows * in->dim * bytes, 16},
                       {lse, rows * 4, 4},
                       {rest, rows * in->dim * bytes, 16},
                       {d_out, rows * in->dim * bytes, 16}};
  const Array outs[] = {{dq, rows * in->dim * bytes, bytes}, {dk, keys, bytes}, {dv, keys, bytes},
                        {workspace, ws, ws ? 16 : 1}};
  rc = check_arrays(ins, 9, outs, 4);
  if (rc != SSIM_OK) return rc;
  rc = check_current_device();
  if (rc != SSIM_OK) return rc;

  const Plan plan = make_plan(*in);
  AttentionParams p = params_of(*in, plan);
  p.o = out;
  p.o_rest = rest;
  p.lse = const_cast<float*>(lse);
  p.d_out = d_out;
  p.delta = static_cast<float*>(workspace);
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  const AttentionTable& t = table_of(in->dtype);
  const int blocks = (in->dim - 1) / 32;
  const unsigned pairs = (unsigned)(in->batch * in->kv_heads);
  if (t.norms) {
    p.norms = reinterpret_cast<float*>(static_cast<char*>(workspace) + delta_bytes(*in));
    rc = launch(t.norms, dim3(pairs * kNormParts), kAttentionThreads, p, stream);
    if (rc != SSIM_OK) return rc;
  }
  const bool kv = any_k && (dk || dv);
  if (plan.grad_q.shape == 2 && plan.grad_kv.shape == 2 && pairs * (plan.grad_q.tiles + plan.grad_kv.tiles) <= kCUs) {
    if (any_q) {
      rc = launch(t.delta, dim3((unsigned)ceil_div(rows, kAttentionThreads / 16)), kAttentionThreads, p, stream);
      if (rc != SSIM_OK) return rc;
    }
    p.tiles = dq ? plan.grad_q.tiles : 0;
    p.kv_tiles = kv ? plan.grad_kv.tiles : 0;
    p.q_blocks = (int)(pairs * p.tiles);
    return launch(t.grads[blocks], dim3(pairs * (p.tiles + p.kv_tiles)), kAttentionThreads, p, stream);
  }
  if (any_q) {  // (it forms delta for the other kernel)
    p.tiles = plan.grad_q.tiles;
    rc = launch(t.grad_q[blocks][plan.grad_q.shape], dim3(pairs * plan.grad_q.tiles), plan.grad_q.threads(), p, stream);
    if (rc != SSIM_OK) return rc;
  }
  if (!kv) return SSIM_OK;
  p.tiles = plan.grad_kv.tiles;
  return launch(t.grad_kv[blocks][plan.grad_kv.shape], dim3(pairs * plan.grad_kv.tiles), plan.grad_kv.threads(), p, stream);
}

}  // extern "C"
