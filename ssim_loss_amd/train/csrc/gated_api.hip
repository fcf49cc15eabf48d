// gated_api.hip -- host side of the gated layer: argument checks, the choice of
// tiles, launches.

#include "gated.hpp"

#include <algorithm>

namespace {

using namespace ssim_train;

constexpr int64_t kMaxWidth = (int64_t)1 << 20;
constexpr int64_t kFewRows = 64;

const GatedTable& table_of(int dtype) {
  switch (dtype) {
    case SSIM_DTYPE_F16: return gated_table_f16();
    case SSIM_DTYPE_BF16: return gated_table_bf16();
    default: return gated_table_f32();
  }
}

int per_chunk(const ssim_gated_linear_inputs& in) { return 16 / elem_bytes(in.dtype); }
int64_t padded(const ssim_gated_linear_inputs& in, int64_t n) { return ceil_div(n, per_chunk(in)) * per_chunk(in); }
size_t to_16(size_t n) { return (n + 15) & ~(size_t)15; }

bool takes_few(const ssim_gated_linear_inputs& in) { return in.rows <= kFewRows && in.width >= per_chunk(in); }

// The tiled products load whole chunks of 16 bytes at multiples of 16: other
// widths and tensors that start elsewhere are copied to rows that do first.
bool needs_copy(const ssim_gated_linear_inputs& in, const void* p) {
  return in.width % per_chunk(in) != 0 || misaligned(p, 16);
}
struct Copies {
  bool any;
  size_t x, w;  // bytes of each, 0: not copied
};
Copies copies_of(const ssim_gated_linear_inputs& in) {
  // (all or none: they share a row's length)
  Copies c = {needs_copy(in, in.x) || needs_copy(in, in.w_gate) || needs_copy(in, in.w_up), 0, 0};
  if (c.any) {
    const size_t row = (size_t)padded(in, in.width) * elem_bytes(in.dtype);
    c.x = (size_t)in.rows * row;
    c.w = (size_t)in.hidden * row;
  }
  return c;
}

int check_inputs(const ssim_gated_linear_inputs* in) {
  if (!in) return SSIM_ERR_NULL;
  if (!known_dtype(in->dtype)) return SSIM_ERR_DTYPE;
  if (in->act < SSIM_ACT_SILU || in->act > SSIM_ACT_SIGMOID) return SSIM_ERR_VALUE;
  if (in->rows < 0 || in->width < 1 || in->width > kMaxWidth || in->hidden < 1 || in->hidden > kMaxWidth)
    return SSIM_ERR_SHAPE;
  if (in->rows > (int64_t)1 << 28) return SSIM_ERR_OVERFLOW;
  return SSIM_OK;
}

GatedParams params_of(const ssim_gated_linear_inputs& in) {
  GatedParams p;
  memset(&p, 0, sizeof(p));
  p.x = in.x;
  p.w[0] = in.w_gate;
  p.w[1] = in.w_up;
  p.bias[0] = in.b_gate;
  p.bias[1] = in.b_up;
  p.rows = in.rows;
  p.x_pitch = p.w_pitch = in.width;
  p.h_pitch = padded(in, in.hidden);
  p.width = p.width_ext = (int)in.width;
  p.hidden = (int)in.hidden;
  p.act = in.act;
  return p;
}

// x and the weights in rows that the tiled products can load, from `ws` on
int make_copies(const ssim_gated_linear_inputs& in, const Copies& c, const GatedTable& t, GatedParams& p, char*& ws,
                void* stream) {
  if (!c.any) return SSIM_OK;
  p.width_ext = (int)padded(in, in.width);
  p.from[0] = in.x;
  p.from[1] = in.w_gate;
  p.from[2] = in.w_up;
  for (int k = 0; k < 3; ++k) {
    p.to[k] = ws;
    ws += k ? c.w : c.x;
  }
  p.x = p.to[0];
  p.w[0] = p.to[1];
  p.w[1] = p.to[2];
  const int64_t most = in.rows > in.hidden ? in.rows : in.hidden;
  const int64_t blocks = ceil_div(most * p.width_ext, 256 * 2 * per_chunk(in));
  const int rc = launch(t.copy, dim3((unsigned)(blocks < 8 * kCUs ? blocks : 8 * kCUs), 3), 256, p, stream);
  if (rc != SSIM_OK) return rc;
  p.x_pitch = p.w_pitch = p.width_ext;
  return SSIM_OK;
}

// Which tiles a product takes, and into how many parts its summed axis is cut.  The
// time of a choice is taken as its rounds (workgroups that fit on the GPU at once)
// times a workgroup's share: its tile's elements by the depth, over what the
// matrix instructions reach with it, and its beginning and end, which are those of
// kEnds of the depth.  A cut costs the sums' way through memory.
struct Choice {
  int tiles;  // 0: 64, 1: 128, 2: 256
  int splits;
  int64_t m_tiles, n_tiles;
  int64_t blocks() const { return m_tiles * n_tiles * splits; }
};
constexpr int kMaxSplits = 16;

Choice choose(const ssim_gated_linear_inputs& in, int product) {
  const int64_t m = product == kForward ? in.hidden : in.width;
  const int64_t n = product == kGradW ? in.hidden : in.rows;
  const int factor = product == kGradW ? 2 : 1;  // results
  const int64_t depth_bytes =
      (product == kForward ? in.width : product == kGradX ? 2 * in.hidden : in.rows) * elem_bytes(in.dtype);
  const int64_t depth = ceil_div(depth_bytes, kDepthBytes);
  // rows of a tile along m and n, workgroups to a CU, and how near the matrix instructions' rate they come
  struct {
    int m, n, at_once;
    double rate;
  } const shapes[3] = {{product == kForward ? 128 : 64, 64, product == kForward ? 2 : 3, 0.5}, {128, 128, 2, 0.85}, {256, 256, 1, 1.0}};
  constexpr double kEnds = 4.0;
  // (in fp32 the matrix instructions take 16 times as long for the same bytes, and memory is far from it)
  const double unit = elem_bytes(in.dtype) == 4 ? 8.0 : 1.0;
  Choice best = {};
  double least = 1e300;
  for (int s = 0; s < 3; ++s) {
    const auto& t = shapes[s];
    const int64_t mt = ceil_div(m, product == kForward ? t.m / 2 : t.m), nt = ceil_div(n, t.n) * factor;
    for (int splits = 1; splits <= kMaxSplits; splits *= 2) {
      if (splits > 1 && (product == kForward || depth < 4 * splits)) break;
      const double rounds = (double)ceil_div(mt * nt * splits, (int64_t)kCUs * t.at_once) * t.at_once;
      double time = rounds * t.m * t.n * (ceil_div(depth, splits) / t.rate + kEnds / unit);
      if (splits > 1) {
        // 64 elements of a tile's depth take as long as 1.3 bytes of memory traffic a CU's share; and a launch
        const double bytes = (double)m * n * factor * (8.0 * splits + 4.0) / kCUs;
        time += (bytes * 50.0 + 256.0 * 256.0 * 2.0) / unit;
      }
      if (time < least) {
        least = time;
        best = {s, splits, mt, nt};
      }
    }
  }
  return best;
}
size_t part_bytes(const ssim_gated_linear_inputs& in, int product) {
  const Choice c = choose(in, product);
  if (c.splits == 1) return 0;
  return to_16((size_t)(product == kGradW ? 2 * in.hidden : in.rows) * in.width * c.splits * 4);
}

void set_product(GatedParams& p, const Choice& c, int product, void* part) {
  p.m_tiles[product] = (int)c.m_tiles;
  p.n_tiles[product] = (int)c.n_tiles;
  p.splits[product] = c.splits;
  p.part[product] = static_cast<float*>(part);
}
constexpr int64_t kMaxBlocks = 1 << 22;

int launch_product(const GatedTable& t, GatedParams& p, const Choice& c, int product, void* stream) {
  if (c.blocks() > kMaxBlocks) return SSIM_ERR_OVERFLOW;
  return launch(t.product[product][c.tiles], dim3((unsigned)c.blocks()), c.tiles == 2 ? 512 : 256, p, stream);
}

struct Slopes {
  int column_blocks, row_blocks, rows_of_block;
};
Slopes slopes_of(const ssim_gated_linear_inputs& in) {
  Slopes s;
  s.column_blocks = (int)ceil_div(padded(in, in.hidden), (int64_t)kWave * per_chunk(in));
  int64_t blocks = ceil_div(8 * kCUs, s.column_blocks);
  const int64_t most = ceil_div(in.rows, 16);  // four rows to a wave at least
  if (blocks > most) blocks = most;
  s.rows_of_block = (int)ceil_div(in.rows, blocks < 1 ? 1 : blocks);
  s.row_blocks = in.rows > 0 ? (int)ceil_div(in.rows, s.rows_of_block) : 0;
  return s;
}

size_t top_count(const Slopes& s) { return (size_t)s.column_blocks * s.row_blocks; }

struct BackwardSpace {
  Copies copies;
  size_t d, bias, tops, part[3], total;
};
BackwardSpace space_of(const ssim_gated_linear_inputs& in) {
  BackwardSpace s;
  s.copies = copies_of(in);
  s.d = (size_t)in.rows * padded(in, in.hidden) * elem_bytes(in.dtype);
  s.bias = to_16((size_t)slopes_of(in).row_blocks * 2 * in.hidden * 4);
  s.tops = table_of(in.dtype).tops ? to_16(4 * top_count(slopes_of(in))) + 16 : 0;  // (the range behind them)
  s.part[kForward] = 0;
  s.part[kGradX] = part_bytes(in, kGradX);
  s.part[kGradW] = part_bytes(in, kGradW);
  s.total = s.copies.x + 2 * s.copies.w + 2 * s.d + s.bias + s.tops + s.part[kGradX] + s.part[kGradW];
  return s;
}

}  // namespace

extern "C" {

size_t ssim_gated_linear_saved_elements(const ssim_gated_linear_inputs* in) {
  if (check_inputs(in) != SSIM_OK) return 0;
  return (size_t)in->rows * padded(*in, in->hidden);
}

size_t ssim_gated_linear_workspace_bytes(const ssim_gated_linear_inputs* in) {
  if (check_inputs(in) != SSIM_OK || in->rows == 0 || takes_few(*in)) return 0;
  const Copies c = copies_of(*in);
  return c.x + 2 * c.w;
}

int ssim_gated_linear_forward(const ssim_gated_linear_inputs* in, void* out, float* g, float* u,
                              void* workspace, void* stream) {
  int rc = check_inputs(in);
  if (rc != SSIM_OK) return rc;
  if (in->rows == 0) return SSIM_OK;
  const size_t ws = ssim_gated_linear_workspace_bytes(in);
  if (!in->x || !in->w_gate || !in->w_up || !out || !g != !u || (ws > 0 && !workspace)) return SSIM_ERR_NULL;
  const int bytes = elem_bytes(in->dtype);
  const size_t weight = (size_t)in->hidden * in->width * bytes, saved = ssim_gated_linear_saved_elements(in) * 4;
  const Array ins[] = {{in->x, (size_t)in->rows * in->width * bytes, bytes},
                       {in->w_gate, weight, bytes},
                       {in->w_up, weight, bytes},
                       {in->b_gate, (size_t)in->hidden * bytes, bytes},
                       {in->b_up, (size_t)in->hidden * bytes, bytes}};
  const Array outs[] = {{out, (size_t)in->rows * in->hidden * bytes, bytes},
                        {g, saved, 16},
                        {u, saved, 16},
                        {workspace, ws, ws ? 16 : 1}};
  rc = check_arrays(ins, 5, outs, 4);
  if (rc != SSIM_OK) return rc;
  rc = check_current_device();
  if (rc != SSIM_OK) return rc;

  const GatedTable& t = table_of(in->dtype);
  GatedParams p = params_of(*in);
  p.out = out;
  p.saved[0] = g;
  p.saved[1] = u;
  if (takes_few(*in))
    return launch(t.few[in->rows <= 16 ? 0 : in->rows <= 32 ? 1 : 2], dim3((unsigned)ceil_div(in->hidden, 16)), 256, p,
                  stream);
  char* at = static_cast<char*>(workspace);
  rc = make_copies(*in, copies_of(*in), t, p, at, stream);
  if (rc != SSIM_OK) return rc;
  const Choice c = choose(*in, kForward);
  set_product(p, c, kForward, nullptr);
  return launch_product(t, p, c, kForward, stream);
}

size_t ssim_gated_linear_backward_workspace_bytes(const ssim_gated_linear_inputs* in) {
  if (check_inputs(in) != SSIM_OK) return 0;
  return space_of(*in).total;
}

int ssim_gated_linear_backward(const ssim_gated_linear_inputs* in, const float* g, const float* u,
                               const void* d_out, const ssim_gated_linear_grads* grads,
                               void* workspace, void* stream) {
  int rc = check_inputs(in);
  if (rc != SSIM_OK) return rc;
  if (!grads) return SSIM_ERR_NULL;
  const bool weights = grads->w_gate || grads->w_up, biases = grads->b_gate || grads->b_up;
  // a gradient of an input that is not there
  if ((grads->b_gate && !in->b_gate) || (grads->b_up && !in->b_up)) return SSIM_ERR_NULL;
  if (!weights && !biases && !(grads->x && in->rows > 0)) return SSIM_OK;
  if (in->rows > 0 && (!in->x || !in->w_gate || !in->w_up || !g || !u || !d_out || !workspace)) return SSIM_ERR_NULL;
  const int bytes = elem_bytes(in->dtype);
  const size_t weight = (size_t)in->hidden * in->width * bytes, bias = (size_t)in->hidden * bytes;
  const size_t saved = ssim_gated_linear_saved_elements(in) * 4, xs = (size_t)in->rows * in->width * bytes;
  const BackwardSpace space = space_of(*in);
  const bool rows = in->rows > 0;
  const Array ins[] = {{in->x, xs, bytes},
                       {in->w_gate, weight, bytes},
                       {in->w_up, weight, bytes},
                       {g, saved, rows ? 16 : 1},
                       {u, saved, rows ? 16 : 1},
                       {d_out, (size_t)in->rows * in->hidden * bytes, bytes}};
  const Array outs[] = {{grads->x, xs, bytes},          {grads->w_gate, weight, bytes},
                        {grads->w_up, weight, bytes},   {grads->b_gate, bias, bytes},
                        {grads->b_up, bias, bytes},     {workspace, rows ? space.total : 0, rows ? 16 : 1}};
  rc = check_arrays(ins, 6, outs, 6);
  if (rc != SSIM_OK) return rc;
  rc = check_current_device();
  if (rc != SSIM_OK) return rc;

  const GatedTable& t = table_of(in->dtype);
  GatedParams p = params_of(*in);
  p.saved[0] = const_cast<float*>(g);
  p.saved[1] = const_cast<float*>(u);
  p.d_out = d_out;
  p.dx = grads->x;
  p.dw[0] = grads->w_gate;
  p.dw[1] = grads->w_up;
  p.db[0] = grads->b_gate;
  p.db[1] = grads->b_up;
  const Slopes s = slopes_of(*in);
  p.row_blocks = s.row_blocks;
  p.rows_of_block = s.rows_of_block;
  char* at = static_cast<char*>(workspace);
  if (rows) {
    if (weights || grads->x) {
      rc = make_copies(*in, space.copies, t, p, at, stream);
      if (rc != SSIM_OK) return rc;
    }
    p.d[0] = at;
    p.d[1] = at + space.d;
    p.part_bias = biases ? reinterpret_cast<float*>(at + 2 * space.d) : nullptr;
    if (t.tops && (weights || grads->x)) {
      char* tops = at + 2 * space.d + space.bias;
      p.tops = reinterpret_cast<float*>(tops);
      p.range = reinterpret_cast<int*>(tops + space.tops - 16);
      p.top_count = (int)top_count(s);
      rc = launch(t.tops, dim3(s.column_blocks, s.row_blocks), 256, p, stream);
      if (rc != SSIM_OK) return rc;
    }
    rc = launch(t.slopes, dim3(s.column_blocks, s.row_blocks), 256, p, stream);
    if (rc != SSIM_OK) return rc;
  }
  char* part = at + 2 * space.d + space.bias + space.tops;
  const Choice x = choose(*in, kGradX), w = choose(*in, kGradW);
  set_product(p, x, kGradX, part);
  set_product(p, w, kGradW, part + space.part[kGradX]);
  const bool x_wanted = grads->x && rows;
  if (x_wanted && weights && x.tiles == 0 && w.tiles == 0 && x.blocks() + w.blocks() <= kMaxBlocks) {
    p.x_blocks = (int)x.blocks();
    rc = launch(t.both, dim3((unsigned)(x.blocks() + w.blocks())), 256, p, stream);
  } else {
    if (x_wanted) rc = launch_product(t, p, x, kGradX, stream);
    if (rc == SSIM_OK && weights) rc = launch_product(t, p, w, kGradW, stream);
  }
  if (rc != SSIM_OK) return rc;
  const bool join_x = x_wanted && x.splits > 1, join_w = weights && w.splits > 1;
  if (!join_x && !join_w && !biases) return SSIM_OK;
  int64_t groups = ceil_div(in->hidden, kWave);
  if (join_x) groups = std::max(groups, ceil_div(in->rows * in->width, 1024));
  if (join_w) groups = std::max(groups, ceil_div(in->hidden * in->width, 1024));
  return launch(t.finish, dim3((unsigned)std::min<int64_t>(groups, 4 * kCUs), 5), 256, p, stream);
}

}  // extern "C"
