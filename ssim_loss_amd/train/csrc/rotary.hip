// rotary.hip -- rotary positions with several axes: pair i of axis a turns by
// positions[a] base^(-2 i / size).
//
// The bound is memory: each element is read and written once.  A thread takes the
// same V pairs of a token in one head after another, so their sines are formed
// once for several heads; a pair's two vectors lie beside each other (adjacent) or
// half an axis apart.  The angle is formed in turns and reduced in fp64: at
// position 10^5 an fp32 angle would be off by 4e-3.

#include "train_common.hpp"

namespace {

using namespace ssim_train;

constexpr int kThreads = 256;
constexpr int kPowers = 8;  // an axis has less than 2^8 pairs of the widest head

struct RotaryParams {
  const void* in[2];   // queries, keys
  void* out[2];
  int64_t stride[2][3];
  int heads[2];
  const void* positions;
  int64_t position_stride[2];
  int64_t batch_tokens, tokens;
  int dim, axes, position_type, inverse;
  int size[SSIM_ROTARY_MAX_AXES];
  double power[SSIM_ROTARY_MAX_AXES][kPowers];  // base^(-2 2^n / size); [..][0] also holds the turn's share
  double turn;                                  // 1 / (2 pi)
  int units;       // of a head: V pairs each, or two vectors that pass
  int head_parts;  // threads that share a token's heads
};

__device__ __forceinline__ double position_of(const RotaryParams& p, int64_t at) {
  switch (p.position_type) {
    case SSIM_POSITION_I32: return static_cast<const int32_t*>(p.positions)[at];
    case SSIM_POSITION_I64: return (double)static_cast<const int64_t*>(p.positions)[at];
    default: return static_cast<const float*>(p.positions)[at];
  }
}

// cos and sin of `turns` full turns: to a quarter turn's nearest multiple in fp64
__device__ __forceinline__ void turn_of(double turns, float& c, float& s) {
  const double quarters = turns * 4.0;
  const double whole = rint(quarters);
  float sn, cs;
  sincospif((float)(quarters - whole) * 0.5f, &sn, &cs);
  const int n = (int)(whole - 4.0 * floor(whole * 0.25));
  const float a = n & 1 ? sn : cs, b = n & 1 ? cs : sn;
  c = n == 1 || n == 2 ? -a : a;
  s = n >= 2 ? -b : b;
}

template <class T, int V, bool kHalves>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p) {
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t row = id / p.units;  // (token, share of its heads)
  int unit = (int)(id - row * p.units);
  const int64_t bt = row / p.head_parts;
  const int part = (int)(row - bt * p.head_parts);
  if (bt >= p.batch_tokens) return;
  const int64_t b = bt / p.tokens, token = bt - b * p.tokens;

  // the unit's axis, its two vectors and its first pair
  int at = 0, axis = -1, pair = 0, far = V;
  bool second = true;
#pragma unroll
  for (int a = 0; a < SSIM_ROTARY_MAX_AXES; ++a) {
    if (a < p.axes && axis < 0) {
      const int here = p.size[a] / (2 * V);
      if (unit < here) {
        axis = a;
        pair = unit * V;
        at += kHalves ? pair : 2 * pair;
        if (kHalves) far = p.size[a] / 2;
      } else {
        unit -= here;
        at += p.size[a];
      }
    }
  }
  if (axis < 0) {
    at += unit * 2 * V;
    second = at + V < p.dim;
    if (!second) far = 0;
  }
  Wide<V> cs, sn;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    cs[k] = 1.0f;
    sn[k] = 0.0f;
  }
  if (axis >= 0) {
    double rate = p.turn;
    // (the loop over powers with constant indexes keeps the table in scalar registers)
    double where = position_of(p, b * p.position_stride[0] + token * p.position_stride[1] + axis);
    double first = 0.0;
#pragma unroll
    for (int a = 0; a < SSIM_ROTARY_MAX_AXES; ++a) {
      if (a != axis) continue;
#pragma unroll
      for (int n = 0; n < kPowers; ++n)
        if (pair >> n & 1) rate *= p.power[a][n];
      first = p.power[a][0];
    }
    if (p.inverse) where = -where;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float c, s;
      turn_of(where * rate, c, s);
      cs[k] = c;
      sn[k] = s;
      rate *= first;
    }
  }

#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if (!p.in[w]) continue;
    const int heads = p.heads[w];
    const T* in = static_cast<const T*>(p.in[w]) + b * p.stride[w][0] + token * p.stride[w][1] + at;
    T* out = static_cast<T*>(p.out[w]) + (bt * heads) * p.dim + at;
#pragma unroll 4
    for (int h = part; h < heads; h += p.head_parts) {
      const T* from = in + h * p.stride[w][2];
      const Wide<V> x = widen<T, V>(load_once<T, V>(from)), y = widen<T, V>(load_once<T, V>(from + far));
      Wide<V> r, s;
      if constexpr (kHalves || V == 1) {
        r = x * cs - y * sn;
        s = y * cs + x * sn;
      } else {  // the pairs lie within the vectors
#pragma unroll
        for (int k = 0; k < V; k += 2) {
          r[k] = x[k] * cs[k / 2] - x[k + 1] * sn[k / 2];
          r[k + 1] = x[k + 1] * cs[k / 2] + x[k] * sn[k / 2];
          s[k] = y[k] * cs[V / 2 + k / 2] - y[k + 1] * sn[V / 2 + k / 2];
          s[k + 1] = y[k + 1] * cs[V / 2 + k / 2] + y[k] * sn[V / 2 + k / 2];
        }
      }
      T* to = out + (int64_t)h * p.dim;
      if (axis < 0) {  // as they are, NaN's bits and infinities too
        store<T, V>(to, load<T, V>(from));
        if (second) store<T, V>(to + far, load<T, V>(from + far));
      } else {
        store<T, V>(to, narrow<T, V>(r));
        store<T, V>(to + far, narrow<T, V>(s));
      }
    }
  }
}

template <class T>
const void* kernel_of(int v, bool halves) {
  constexpr int kFull = 16 / (int)sizeof(T);
  if (v == kFull)
    return halves ? (const void*)rotary_kernel<T, kFull, true> : (const void*)rotary_kernel<T, kFull, false>;
  if (v == 4) return halves ? (const void*)rotary_kernel<T, 4, true> : (const void*)rotary_kernel<T, 4, false>;
  return halves ? (const void*)rotary_kernel<T, 1, true> : (const void*)rotary_kernel<T, 1, false>;
}

bool strides_ok(const int64_t* s, int n) {
  for (int k = 0; k < n; ++k)
    if (s[k] < 0 || s[k] > (int64_t)1 << 46) return false;
  return true;
}

int check_inputs(const ssim_rotary_inputs* in) {
  if (!in) return SSIM_ERR_NULL;
  if (!known_dtype(in->dtype)) return SSIM_ERR_DTYPE;
  if (in->position_type < SSIM_POSITION_F32 || in->position_type > SSIM_POSITION_I64) return SSIM_ERR_DTYPE;
  if ((in->pairs != SSIM_PAIRS_ADJACENT && in->pairs != SSIM_PAIRS_HALVES) || in->inverse < 0 || in->inverse > 1)
    return SSIM_ERR_VALUE;
  if (!(in->base > 0.0 && in->base <= 1.7976931348623157e308)) return SSIM_ERR_VALUE;
  if (in->batch < 0 || in->tokens < 0 || in->dim < 1 || in->dim > SSIM_ROTARY_MAX_DIM || in->q_heads < 1 ||
      in->q_heads > 65536 || (in->k && (in->k_heads < 1 || in->k_heads > 65536)))
    return SSIM_ERR_SHAPE;
  if (in->axes < 1 || in->axes > SSIM_ROTARY_MAX_AXES) return SSIM_ERR_SHAPE;
  int sum = 0;
  for (int a = 0; a < in->axes; ++a) {
    if (in->axis_size[a] < 2 || in->axis_size[a] % 2 != 0 || in->axis_size[a] > in->dim) return SSIM_ERR_SHAPE;
    sum += in->axis_size[a];
  }
  if (sum > in->dim) return SSIM_ERR_SHAPE;
  if (!strides_ok(in->q_stride, 3) || !strides_ok(in->position_stride, 2) || (in->k && !strides_ok(in->k_stride, 3)))
    return SSIM_ERR_SHAPE;
  if (in->batch > 0 && in->tokens > ((int64_t)1 << 46) / in->batch / 65536 / SSIM_ROTARY_MAX_DIM)
    return SSIM_ERR_OVERFLOW;
  return SSIM_OK;
}

// bytes from the first element to the last
size_t span(const int64_t* stride, int64_t batch, int64_t tokens, int64_t heads, int64_t dim, int bytes) {
  return (size_t)((batch - 1) * stride[0] + (tokens - 1) * stride[1] + (heads - 1) * stride[2] + dim) * bytes;
}

}  // namespace

extern "C" int ssim_rotary(const ssim_rotary_inputs* in, void* q_out, void* k_out, void* stream) {
  int rc = check_inputs(in);
  if (rc != SSIM_OK) return rc;
  if (in->batch == 0 || in->tokens == 0) return SSIM_OK;
  if (!in->q || !in->positions || !q_out || (in->k && !k_out)) return SSIM_ERR_NULL;
  const int bytes = elem_bytes(in->dtype), position_bytes = in->position_type == SSIM_POSITION_I64 ? 8 : 4;
  const int64_t n = in->batch * in->tokens;
  const int64_t flat[3] = {in->position_stride[0], in->position_stride[1], 0};
  const Array ins[] = {{in->q, span(in->q_stride, in->batch, in->tokens, in->q_heads, in->dim, bytes), bytes},
                       {in->k, in->k ? span(in->k_stride, in->batch, in->tokens, in->k_heads, in->dim, bytes) : 0, bytes},
                       {in->positions, span(flat, in->batch, in->tokens, 1, in->axes, position_bytes), position_bytes}};
  const Array outs[] = {{q_out, (size_t)(n * in->q_heads * in->dim) * bytes, bytes},
                        {in->k ? k_out : nullptr, in->k ? (size_t)(n * in->k_heads * in->dim) * bytes : 0, bytes}};
  rc = check_arrays(ins, 3, outs, 2);
  if (rc != SSIM_OK) return rc;
  rc = check_current_device();
  if (rc != SSIM_OK) return rc;

  RotaryParams p;
  memset(&p, 0, sizeof(p));
  p.in[0] = in->q;
  p.in[1] = in->k;
  p.out[0] = q_out;
  p.out[1] = k_out;
  p.heads[0] = in->q_heads;
  p.heads[1] = in->k ? in->k_heads : 0;
  for (int k = 0; k < 3; ++k) {
    p.stride[0][k] = in->q_stride[k];
    p.stride[1][k] = in->k_stride[k];
  }
  p.positions = in->positions;
  p.position_stride[0] = in->position_stride[0];
  p.position_stride[1] = in->position_stride[1];
  p.batch_tokens = n;
  p.tokens = in->tokens;
  p.dim = in->dim;
  p.axes = in->axes;
  p.position_type = in->position_type;
  p.inverse = in->inverse;
  p.turn = 0.15915494309189533577;
  // vectors as wide as divide every axis (half of it where its halves are apart) and the rest
  const bool halves = in->pairs == SSIM_PAIRS_HALVES;
  int v = 16 / bytes, rest = in->dim;
  auto fits = [&](int w) {
    for (int a = 0; a < in->axes; ++a)
      if (in->axis_size[a] % (2 * w) != 0) return false;
    return rest % w == 0;
  };
  for (int a = 0; a < in->axes; ++a) rest -= in->axis_size[a];
  if (!fits(v)) v = fits(4) ? 4 : 1;
  p.units = (int)ceil_div(rest, 2 * v);
  for (int a = 0; a < in->axes; ++a) {
    p.size[a] = in->axis_size[a];
    p.units += in->axis_size[a] / (2 * v);
    double power = pow(in->base, -2.0 / in->axis_size[a]);
    for (int k = 0; k < kPowers; ++k, power *= power) p.power[a][k] = power;
  }
  // heads to a thread: few enough that there are threads for every CU
  const int64_t one = n * p.units;
  const int most = in->q_heads > p.heads[1] ? in->q_heads : p.heads[1];
  int64_t parts = ceil_div((int64_t)kCUs * 1024, one);
  p.head_parts = (int)(parts < most ? parts : most);
  const int64_t blocks = ceil_div(one * p.head_parts, kThreads);
  if (blocks > 0x7fffffff / kThreads * 2) return SSIM_ERR_OVERFLOW;
  const void* kernel = in->dtype == SSIM_DTYPE_F32   ? kernel_of<F32>(v, halves)
                       : in->dtype == SSIM_DTYPE_F16 ? kernel_of<F16>(v, halves)
                                                     : kernel_of<BF16>(v, halves);
  return launch(kernel, dim3((unsigned)blocks), kThreads, p, stream);
}
