// block_norm_api.hip -- host side of the joint between two blocks: argument
// checks, the choice of a kernel's shape, launches.

#include "block_norm.hpp"

namespace {

using namespace ssim_train;

constexpr int kCUs = 256;  // of an MI355X; the workspace's size must not need a device query

const NormTable& table_of(int dtype) {
  switch (dtype) {
    case SSIM_DTYPE_F16: return norm_table_f16();
    case SSIM_DTYPE_BF16: return norm_table_bf16();
    default: return norm_table_f32();
  }
}

constexpr int64_t kEnds = 8;
constexpr int64_t kMaxCutGroups = 32768;  // the last sums' grid has a row for each

// How the rows are dealt out.
struct Plan {
  bool wide, grouped;
  int shape;
  int threads, blocks;            // of the forward
  int back_threads, back_blocks;  // of the backward
  bool cut;  // a gate row's rows go to whole workgroups (in `parts` parts), not each group to a worker
  int parts;
  int64_t groups, part_rows;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Workgroups of `workers` rows at once, about `target` of them, with the same
// number of rows each.
int64_t blocks_for(int64_t rows, int64_t workers, int64_t target) {
  const int64_t need = ceil_div(rows, workers);
  if (need <= target) return need;
  const int64_t each = (2 * need + target) / (2 * target);  // to the nearest
  return ceil_div(need, each);
}

int threads_of(int shape, int row_waves, int items, int64_t vectors) {
  if (shape_lanes(shape)) return row_waves * kWave;
  return (int)ceil_div(ceil_div(vectors, items), kWave) * kWave;
}

Plan make_plan(const ssim_block_norm_inputs& in) {
  Plan p;
  const int xb = elem_bytes(in.x_dtype), bb = elem_bytes(in.branch_dtype);
  const int64_t vectors = ceil_div(in.width, 16 / bb);
  p.shape = in.width < 16 / bb     ? kNarrow
            : vectors <= 8         ? kLanes8
            : vectors <= 16        ? kLanes16
            : vectors <= 32        ? kLanes32
            : vectors <= kWave     ? kWave1
            : vectors <= 2 * kWave ? kWave2
            : vectors <= 4 * kWave ? kGroup1
            : vectors <= 8 * kWave ? kGroup1w
            : vectors <= 16 * kWave ? kGroup2
            : vectors <= 32 * kWave ? kGroup4
                                    : kGroup8;
  const int lanes = shape_lanes(p.shape);
  p.wide = in.x_dtype != in.branch_dtype;
  p.threads = threads_of(p.shape, kRowWaves, shape_fwd_items(p.shape, xb, bb), vectors);
  p.back_threads = threads_of(p.shape, kRowWavesBack, shape_items(p.shape, bb), vectors);
  p.grouped = in.gate && in.gate_rows > 1;

  // Forward: rows in work whose loads are 48 KB on each CU; where a row is a
  // workgroup's 28 KB, 32 KB with the next row's loads out beside them.  Fewer
  // leave the memory idle; more read the weights more often and end unevenly.
  // Measured with 24, 28 and 36 KB where a row is a workgroup's: 4100 x 1153 fp16
  // 12.2, 11.5 and 11.7 us, 32768 x 2048 bf16 beside fp32 163, 163 and 182 us;
  // with 32 and 48 KB where it is a wave's: 65536 x 512 bf16 63 and 55 us.
  const int64_t row_bytes = in.width * (xb + bb + (in.gate && !p.grouped ? bb : 0));
  const int64_t in_work = lanes ? 48 << 10 : shape_early(p.shape) ? 32 << 10 : 28 << 10;
  const int64_t rows_per_cu = ceil_div(in_work, row_bytes);
  const int fwd_workers = lanes ? kRowWaves * kWave / lanes : 1;
  p.blocks = (int)blocks_for(in.rows, fwd_workers, kCUs * ceil_div(rows_per_cu, fwd_workers));

  // Backward: 16 KB, since each workgroup leaves a row of partial sums.
  // Measured with 16 and 32 KB: 4100 x 1152 fp16 18.8 and 23.4 us, 32768 x
  // 2048 bf16 beside fp32 266 and 290 us.  Blocks in fp32 leave room for two
  // workgroups of eight waves on a CU, and one waits at its barriers too long
  // (16384 x 2048: 195 us with two, 230 with one).
  const int workers = lanes ? kRowWavesBack * kWave / lanes : 1;
  const int64_t back_bytes = in.width * (2 * xb + 2 * bb + (in.gate && !p.grouped ? bb : 0));
  int64_t per_cu = ceil_div(ceil_div(16 << 10, back_bytes), workers);
  if (bb == 4 && p.shape <= kGroup2 && per_cu < 1024 / p.back_threads) per_cu = 1024 / p.back_threads;
  const int64_t target = kCUs * per_cu;
  p.parts = 1;
  p.groups = p.part_rows = 0;
  p.cut = false;
  if (!p.grouped) {
    p.back_blocks = (int)blocks_for(in.rows, workers, target);
    return p;
  }
  p.groups = in.rows / in.gate_rows;
  p.part_rows = in.gate_rows;
  if (p.groups == 0) {
    p.back_blocks = 0;
    return p;
  }
  int64_t parts = target / p.groups;
  const int64_t most = ceil_div(in.gate_rows, workers);
  if (parts > most) parts = most;
  if (parts > 1) {
    p.part_rows = ceil_div(ceil_div(in.gate_rows, parts), workers) * workers;
    p.parts = (int)ceil_div(in.gate_rows, p.part_rows);
    p.cut = p.parts > 1;
  }
  // A group to a worker, or to a workgroup, whose workers share its rows: by the
  // rows that a worker takes one after another, where a workgroup's beginning and
  // end (weights, sums) take the time of kEnds.  Forward and gradients in bf16, by
  // worker and by workgroup: 129 groups of 1024 rows of 64 785 and 36 us, 500 of
  // 256 of 384 386 and 192, 1000 of 64 of 64 65 and 35; 4000 of 64 of 64 94 and 111,
  // 500 of 16 of 1000 56 and 65.  (2000 of 64 of 64, 70 and 59, falls to the worker.)
  if (!p.cut) {
    p.back_blocks = (int)blocks_for(p.groups, workers, target);
    const int64_t each = ceil_div(p.groups, (int64_t)p.back_blocks * workers) * in.gate_rows;
    p.cut = p.groups <= kMaxCutGroups && ceil_div(p.groups, target) * (most + kEnds) < each;
  }
  if (p.cut) p.back_blocks = (int)(p.groups * p.parts);
  return p;
}

int check_inputs(const ssim_block_norm_inputs* in) {
  if (!in) return SSIM_ERR_NULL;
  if (!known_dtype(in->x_dtype) || !known_dtype(in->branch_dtype) ||
      (in->x_dtype != in->branch_dtype && in->x_dtype != SSIM_DTYPE_F32))
    return SSIM_ERR_DTYPE;
  if (in->gate_act != SSIM_GATE_NONE && in->gate_act != SSIM_GATE_SIGMOID) return SSIM_ERR_VALUE;
  if (!(in->eps >= 0.0 && in->eps <= 3.4028234663852886e38)) return SSIM_ERR_VALUE;
  if (in->rows < 0 || in->width < 1 || in->width > SSIM_BLOCK_NORM_MAX_WIDTH) return SSIM_ERR_SHAPE;
  if (in->gate && (in->gate_rows < 1 || in->rows % in->gate_rows != 0)) return SSIM_ERR_SHAPE;
  if (in->rows > ((int64_t)1 << 46) / (4 * in->width)) return SSIM_ERR_OVERFLOW;
  return SSIM_OK;
}

struct Array {
  const void* p;
  size_t bytes;
  int align;
};

// alignment of all, and no output over an input or another output
int check_arrays(const Array* ins, int n_in, const Array* outs, int n_out) {
  for (int k = 0; k < n_in; ++k)
    if (misaligned(ins[k].p, ins[k].align)) return SSIM_ERR_SHAPE;
  for (int k = 0; k < n_out; ++k) {
    if (misaligned(outs[k].p, outs[k].align)) return SSIM_ERR_SHAPE;
    for (int l = 0; l < n_in; ++l)
      if (overlaps(outs[k].p, outs[k].bytes, ins[l].p, ins[l].bytes)) return SSIM_ERR_ALIAS;
    for (int l = 0; l < k; ++l)
      if (overlaps(outs[k].p, outs[k].bytes, outs[l].p, outs[l].bytes)) return SSIM_ERR_ALIAS;
  }
  return SSIM_OK;
}

size_t workspace_bytes(const ssim_block_norm_inputs& in, const Plan& p) {
  const size_t arrays = p.cut ? 3 : 2;
  return ((size_t)p.back_blocks * (size_t)in.width * 4 * arrays + 15) & ~(size_t)15;
}

NormParams params_of(const ssim_block_norm_inputs& in, const Plan& p) {
  NormParams k;
  memset(&k, 0, sizeof(k));
  k.x = in.x;
  k.b = in.branch;
  k.gate = in.gate;
  k.scale = in.scale;
  k.post = in.post_weight;
  k.pre = in.pre_weight;
  k.rows = in.rows;
  k.gate_rows = in.gate ? in.gate_rows : 1;
  k.width = (int)in.width;
  k.act = in.gate_act;
  k.eps = (float)in.eps;
  k.inv_width = (float)(1.0 / (double)in.width);
  k.groups = p.groups;
  k.part_rows = p.part_rows;
  k.cut = p.cut;
  k.parts = p.parts;
  k.blocks = p.back_blocks;
  return k;
}

int launch(const void* kernel, dim3 grid, int threads, NormParams& k, void* stream) {
  void* args[] = {&k};
  if (hipLaunchKernel(kernel, grid, dim3(threads), args, 0, static_cast<hipStream_t>(stream)) !=
      hipSuccess) {
    (void)hipGetLastError();
    return SSIM_ERR_HIP;
  }
  return SSIM_OK;
}

}  // namespace

extern "C" {

int ssim_block_norm_forward(const ssim_block_norm_inputs* in, void* residual, void* normed,
                            float* stats, void* stream) {
  int rc = check_inputs(in);
  if (rc != SSIM_OK) return rc;
  if (in->rows == 0) return SSIM_OK;
  if (!in->x || !in->branch || !residual || !normed) return SSIM_ERR_NULL;
  const int xb = elem_bytes(in->x_dtype), bb = elem_bytes(in->branch_dtype);
  const size_t n = (size_t)in->rows * (size_t)in->width, w = 4 * (size_t)in->width;
  const size_t gate = in->gate ? n / (size_t)in->gate_rows * bb : 0;
  const Array ins[] = {{in->x, n * xb, xb}, {in->branch, n * bb, bb}, {in->gate, gate, bb},
                       {in->scale, w, 4},   {in->post_weight, w, 4},  {in->pre_weight, w, 4}};
  const Array outs[] = {{residual, n * xb, xb}, {normed, n * bb, bb}, {stats, 8 * (size_t)in->rows, 4}};
  rc = check_arrays(ins, 6, outs, 3);
  if (rc != SSIM_OK) return rc;
  rc = check_current_device();
  if (rc != SSIM_OK) return rc;

  const Plan p = make_plan(*in);
  NormParams k = params_of(*in, p);
  k.r = residual;
  k.h = normed;
  k.stats = stats;
  return launch(table_of(in->branch_dtype).forward[p.wide][p.shape], dim3(p.blocks), p.threads, k,
                stream);
}

size_t ssim_block_norm_workspace_bytes(const ssim_block_norm_inputs* in) {
  if (check_inputs(in) != SSIM_OK || in->rows == 0) return 0;
  return workspace_bytes(*in, make_plan(*in));
}

int ssim_block_norm_backward(const ssim_block_norm_inputs* in, const float* stats,
                             const void* d_residual, const void* d_normed,
                             const ssim_block_norm_grads* grads, void* workspace, void* stream) {
  int rc = check_inputs(in);
  if (rc != SSIM_OK) return rc;
  if (!grads) return SSIM_ERR_NULL;
  const bool weights = (grads->scale && in->scale) || (grads->post_weight && in->post_weight) ||
                       (grads->pre_weight && in->pre_weight);
  const bool rows = in->rows > 0;
  if (rows && (!in->x || !in->branch || !stats || !workspace)) return SSIM_ERR_NULL;
  // a gradient of an input that is not there
  if ((grads->gate && !in->gate) || (grads->scale && !in->scale) ||
      (grads->post_weight && !in->post_weight) || (grads->pre_weight && !in->pre_weight))
    return SSIM_ERR_NULL;
  const Plan p = make_plan(*in);
  const int xb = elem_bytes(in->x_dtype), bb = elem_bytes(in->branch_dtype);
  const size_t n = (size_t)in->rows * (size_t)in->width, w = 4 * (size_t)in->width;
  const size_t gate = in->gate ? n / (size_t)in->gate_rows * bb : 0;
  const Array ins[] = {{in->x, n * xb, xb},       {in->branch, n * bb, bb},
                       {in->gate, gate, bb},      {in->scale, w, 4},
                       {in->post_weight, w, 4},   {in->pre_weight, w, 4},
                       {d_residual, n * xb, xb},  {d_normed, n * bb, bb},
                       {stats, 8 * (size_t)in->rows, 4}};
  const Array outs[] = {{grads->x, n * xb, xb},     {grads->branch, n * bb, bb},
                        {grads->gate, gate, bb},    {grads->scale, w, 4},
                        {grads->post_weight, w, 4}, {grads->pre_weight, w, 4},
                        {workspace, rows ? workspace_bytes(*in, p) : 0, rows ? 16 : 1}};
  rc = check_arrays(ins, 9, outs, 7);
  if (rc != SSIM_OK) return rc;
  if (!weights && !(rows && (grads->x || grads->branch || grads->gate))) return SSIM_OK;
  rc = check_current_device();
  if (rc != SSIM_OK) return rc;

  NormParams k = params_of(*in, p);
  k.stats = const_cast<float*>(stats);
  k.dr = d_residual;
  k.dh = d_normed;
  k.dx = grads->x;
  k.db = grads->branch;
  k.dg = grads->gate;
  k.dscale = grads->scale;
  k.dpost = grads->post_weight;
  k.dpre = grads->pre_weight;
  const size_t part = (size_t)p.back_blocks * (size_t)in->width;
  float* ws = static_cast<float*>(workspace);
  const bool cut = p.cut && grads->gate && rows;
  if (k.dscale || k.dpost) k.part_total = ws;
  if (k.dpre) k.part_pre = ws + part;
  if (cut) k.part_gate = ws + 2 * part;
  const NormTable& t = table_of(in->branch_dtype);
  if (rows) {
    rc = launch(t.backward[p.wide][p.shape][p.grouped], dim3(p.back_blocks), p.back_threads, k, stream);
    if (rc != SSIM_OK) return rc;
  }
  if (!weights && !cut) return SSIM_OK;
  const unsigned columns = (unsigned)ceil_div(in->width, kSumColumns);
  return launch(t.sums, dim3(columns, cut ? 2 + (unsigned)p.groups : 2), kSumColumns * kSumSlices, k,
                stream);
}

}  // extern "C"
