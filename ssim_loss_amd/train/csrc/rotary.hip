// rotary.hip -- rotary positions with several axes: pair i of axis a turns by
// positions[a] base^(-2 i / size).
//
// The bound is memory: each element is read and written once (2 x 16384 x 32 heads x
// 128 bf16: 107 us, 5.0 TB/s; a large copy reaches 5.1).  A workgroup has a few tokens:
// each of their sines is formed once, by one thread, and lies in LDS for all heads;
// formed by each thread that needs them they took longer than the memory (1025 x 4
// tokens, 32 heads x 72 fp16, 14 to 20 us by the number of such threads, so 12).  Then a thread takes V pairs of a head
// at a time, two vectors beside each other (adjacent) or half an axis apart, whose
// loads are out before the sines are formed.
// The angle is formed in turns and reduced in fp64: at position 10^5 an fp32 angle
// would be off by 4e-3.

#include "train_common.hpp"

namespace {

using namespace ssim_train;

constexpr int kThreads = 256;
constexpr int kAtOnce = 2;   // units that a thread has in work
constexpr int kUnits = 4;    // ... and takes; 2 to 16 were tried: 2 x 16384 x 32 x 128 bf16 107 to 121 us
constexpr int kPowers = 8;   // an axis has at most 2^8 pairs
constexpr int kMaxPairs = SSIM_ROTARY_MAX_DIM / 2;
constexpr int kSines = 1024; // of a workgroup
constexpr int kMaxAtOnce = 64;

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
  double power[SSIM_ROTARY_MAX_AXES][kPowers];  // base^(-2 2^n / size)
  double turn;       // 1 / (2 pi)
  int units;         // of a head: V pairs each, or two vectors that pass
  int pairs;         // of a head
  int at_once;       // tokens of a workgroup
  int head_parts;    // workgroups that share the heads of such tokens
  int heads_of_part;
  unsigned by_units, by_heads, by_pairs;  // ceil(2^32 / units), ... of heads_of_part, of pairs
};

// a / b with by = ceil(2^32 / b), for a b < 2^32; 0: b = 1
__device__ __forceinline__ unsigned divided(unsigned a, unsigned by) { return by ? __umulhi(a, by) : a; }

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

struct Unit {
  int at;    // its first vector's first element in the head
  int far;   // from there to the second's; 0: there is none
  int pair;  // its first pair of all the head's; -1: it passes
};

template <class T, int V, bool kHalves>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p) {
  __shared__ __attribute__((aligned(16))) float cosines[kSines + 16], sines[kSines + 16];
  __shared__ Unit units[kMaxPairs + 1];
  __shared__ int64_t offsets[2][kMaxAtOnce], place[kMaxAtOnce];  // of the tokens: queries, keys, positions
  const int64_t block = blockIdx.x / p.head_parts;
  const int part = (int)(blockIdx.x - block * p.head_parts);
  const int64_t first_token = block * p.at_once;
  const int tokens = (int)(p.batch_tokens - first_token < p.at_once ? p.batch_tokens - first_token : p.at_once);
  const int first_head = part * p.heads_of_part;
  const int heads = min(p.heads_of_part, p.heads[0] + p.heads[1] - first_head);

  for (int u = threadIdx.x; u < p.units; u += kThreads) {
    Unit e = {0, 0, -1};
    int unit = u, pair = 0;
    bool found = false;
#pragma unroll
    for (int a = 0; a < SSIM_ROTARY_MAX_AXES; ++a) {
      if (a >= p.axes || found) continue;
      const int here = p.size[a] / (2 * V);
      if (unit < here) {
        e = {e.at + (kHalves ? V : 2 * V) * unit, kHalves ? p.size[a] / 2 : V, pair + unit * V};
        found = true;
      } else {
        unit -= here;
        e.at += p.size[a];
        pair += p.size[a] / 2;
      }
    }
    if (!found) {
      e.at += unit * 2 * V;
      e.far = e.at + V < p.dim ? V : 0;
    }
    units[u] = e;
  }
  if ((int)threadIdx.x < tokens) {
    const int64_t bt = first_token + threadIdx.x, b = bt / p.tokens, token = bt - b * p.tokens;
#pragma unroll
    for (int w = 0; w < 2; ++w) offsets[w][threadIdx.x] = b * p.stride[w][0] + token * p.stride[w][1];
    place[threadIdx.x] = b * p.position_stride[0] + token * p.position_stride[1];
  }
  __syncthreads();

  // A thread's units, in steps of kThreads: of a token, a head, a unit of it.
  const unsigned count = (unsigned)(tokens * p.heads_of_part * p.units);
  Vec<T, V> x[kAtOnce], y[kAtOnce];
  Unit unit[kAtOnce];
  int token[kAtOnce];
  T* to[kAtOnce];  // NULL: there is no such unit
  auto load_units = [&](unsigned first) {
#pragma unroll
    for (int n = 0; n < kAtOnce; ++n) {
      const unsigned id = first + n * kThreads;
      const unsigned row = divided(min(id, count - 1), p.by_units);
      unit[n] = units[min(id, count - 1) - row * p.units];
      token[n] = (int)divided(row, p.by_heads);
      const int head = (int)row - token[n] * p.heads_of_part;
      const bool there = id < count && head < heads;
      const int h = first_head + min(head, heads - 1), w = h >= p.heads[0], hw = w ? h - p.heads[0] : h;
      const T* from = static_cast<const T*>(p.in[w]) + offsets[w][token[n]] + hw * p.stride[w][2] + unit[n].at;
      x[n] = load<T, V>(from);
      y[n] = load<T, V>(from + unit[n].far);
      to[n] = there ? static_cast<T*>(p.out[w]) + ((first_token + token[n]) * p.heads[w] + hw) * p.dim + unit[n].at : nullptr;
    }
  };
  load_units(threadIdx.x);

  for (unsigned id = threadIdx.x; id < (unsigned)(tokens * p.pairs); id += kThreads) {
    const int t = (int)divided(id, p.by_pairs), k = (int)(id - t * p.pairs);
    int pair = k, axis = 0;
#pragma unroll
    for (int a = 0; a + 1 < SSIM_ROTARY_MAX_AXES; ++a)
      if (axis == a && a + 1 < p.axes && pair >= p.size[a] / 2) {
        pair -= p.size[a] / 2;
        axis = a + 1;
      }
    double rate = p.turn;
    // (constant indexes keep the table in scalar registers)
#pragma unroll
    for (int a = 0; a < SSIM_ROTARY_MAX_AXES; ++a)
#pragma unroll
      for (int n = 0; n < kPowers; ++n)
        if (axis == a && (pair >> n & 1)) rate *= p.power[a][n];
    const double where = position_of(p, place[t] + axis);
    float c, s;
    turn_of((p.inverse ? -where : where) * rate, c, s);
    cosines[id] = c;
    sines[id] = s;
  }
  __syncthreads();

  for (unsigned first = threadIdx.x; first < count; first += kAtOnce * kThreads) {
    if (first != threadIdx.x) load_units(first);
#pragma unroll
    for (int n = 0; n < kAtOnce; ++n) {
      if (!to[n]) continue;
      if (unit[n].pair < 0) {  // as they are, NaN's bits and infinities too
        store<T, V>(to[n], x[n]);
        if (unit[n].far) store<T, V>(to[n] + unit[n].far, y[n]);
        continue;
      }
      const int at = token[n] * p.pairs + unit[n].pair;
      const Wide<V> cs = load<float, V>(cosines + at), sn = load<float, V>(sines + at);
      const Wide<V> u = widen<T, V>(x[n]), v = widen<T, V>(y[n]);
      Wide<V> r, s;
      if constexpr (kHalves || V == 1) {
        r = u * cs - v * sn;
        s = v * cs + u * sn;
      } else {  // the pairs lie within the vectors
#pragma unroll
        for (int k = 0; k < V; k += 2) {
          r[k] = u[k] * cs[k / 2] - u[k + 1] * sn[k / 2];
          r[k + 1] = u[k + 1] * cs[k / 2] + u[k] * sn[k / 2];
          s[k] = v[k] * cs[V / 2 + k / 2] - v[k + 1] * sn[V / 2 + k / 2];
          s[k + 1] = v[k + 1] * cs[V / 2 + k / 2] + v[k] * sn[V / 2 + k / 2];
        }
      }
      store<T, V>(to[n], narrow<T, V>(r));
      store<T, V>(to[n] + unit[n].far, narrow<T, V>(s));
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
  const int64_t heads = in->k && in->k_heads > in->q_heads ? in->k_heads : in->q_heads;
  if (in->batch > 0 && in->tokens > ((int64_t)1 << 44) / in->batch / (heads * in->dim)) return SSIM_ERR_OVERFLOW;
  return SSIM_OK;
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
  const int64_t q_span = span(in->q_stride, in->batch, in->tokens, in->q_heads, in->dim),
                k_span = in->k ? span(in->k_stride, in->batch, in->tokens, in->k_heads, in->dim) : 0,
                position_span = span(flat, in->batch, in->tokens, 1, in->axes);
  if (q_span < 0 || k_span < 0 || position_span < 0) return SSIM_ERR_OVERFLOW;
  const Array ins[] = {{in->q, (size_t)q_span * bytes, bytes},
                       {in->k, (size_t)k_span * bytes, bytes},
                       {in->positions, (size_t)position_span * position_bytes, position_bytes}};
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
  for (int a = 0; a < in->axes; ++a) p.pairs += in->axis_size[a] / 2;
  // Tokens to a workgroup: as many as give its threads kUnits units each, while
  // there are workgroups enough and room for the sines.  Of few tokens with many
  // heads the heads go to several workgroups.
  const int heads = in->q_heads + p.heads[1];
  const int64_t of_token = (int64_t)heads * p.units;
  int64_t at_once = kThreads * kUnits / of_token;
  if (at_once > n / (2 * kCUs)) at_once = n / (2 * kCUs);
  if (at_once > kSines / p.pairs) at_once = kSines / p.pairs;
  if (at_once > kMaxAtOnce) at_once = kMaxAtOnce;
  if (at_once < 1) at_once = 1;
  p.at_once = (int)at_once;
  int64_t parts = ceil_div(of_token * at_once, kThreads * kUnits);
  const int64_t groups = ceil_div(n, at_once);
  if (groups * parts < 2 * kCUs) parts = ceil_div(2 * kCUs, groups);
  if (parts > ceil_div(of_token * at_once, kThreads)) parts = ceil_div(of_token * at_once, kThreads);
  constexpr int64_t kMaxBlocks = ((int64_t)1 << 32) / kThreads - 1;
  if (groups * parts > kMaxBlocks) parts = ceil_div(of_token * at_once, 64 * kThreads * kUnits);  // (longer workgroups)
  p.heads_of_part = (int)ceil_div(heads, parts);
  p.head_parts = (int)ceil_div(heads, p.heads_of_part);
  auto inverse_of = [](int64_t d) { return d == 1 ? 0u : (unsigned)((((uint64_t)1 << 32) + d - 1) / d); };
  p.by_units = inverse_of(p.units);
  p.by_heads = inverse_of(p.heads_of_part);
  p.by_pairs = inverse_of(p.pairs);
  const int64_t blocks = groups * p.head_parts;
  if (blocks > kMaxBlocks) return SSIM_ERR_OVERFLOW;
  const void* kernel = in->dtype == SSIM_DTYPE_F32   ? kernel_of<F32>(v, halves)
                       : in->dtype == SSIM_DTYPE_F16 ? kernel_of<F16>(v, halves)
                                                     : kernel_of<BF16>(v, halves);
  return launch(kernel, dim3((unsigned)blocks), kThreads, p, stream);
}
