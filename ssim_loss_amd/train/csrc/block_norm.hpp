// block_norm.hpp -- kernels of the joint between two blocks of a network:
//   bh = b / sqrt(mean(b^2) + eps)          the norm after a block
//   r  = x + a c bh                         a = act(gate), c = scale post_weight
//   h  = r / sqrt(mean(r^2) + eps) pre      the norm before the next block
// and their gradients.
//
// A row stays in registers between its reductions, so each tensor is read and
// written once; the bound is that traffic (32768 x 2048 bf16 beside fp32, forward:
// 161 us, 5.8 TB/s; 16384 x 4096 bf16: forward 101 us, 5.3 TB/s, backward 145 us,
// 5.6 TB/s; a large copy reaches 5.1).  A row belongs to 8, 16, 32 or 64 lanes of
// a wave (narrow rows: the reductions need no barrier) or to a workgroup.  A
// thread takes I vectors of 16 bytes of the block's type, those of its neighbours
// beside it; rows start at any element, and all vectors, a row's last one too, are
// loaded at full width.  The weights of a thread's columns stay in registers over
// all rows of the workgroup (but of the widest, see kAnew and kReload).

#pragma once

#include "train_common.hpp"

namespace ssim_train {

constexpr int kMaxWaves = 8;     // of a workgroup
constexpr int kWideWaves = 16;    // of one whose threads load their vectors twice
constexpr int kRowWaves = 4;     // rows (waves) of a workgroup where a wave takes a row: forward
constexpr int kRowWavesBack = 8; // and backward
constexpr int kSumColumns = 64; // columns a workgroup of the last sum takes
constexpr int kSumSlices = 16;  // ... and shares of the partial sums it adds at once

struct NormParams {
  const void* x;
  const void* b;
  const void* gate;
  const float* scale;
  const float* post;
  const float* pre;
  int64_t rows, gate_rows;
  int width, act;
  float eps, inv_width;
  // forward
  void* r;
  void* h;
  // stats: [rows][2], 1/sqrt(mean(b^2) + eps) and 1/sqrt(mean(r^2) + eps)
  float* stats;
  // backward
  const void* dr;
  const void* dh;
  void* dx;
  void* db;
  void* dg;
  float* dscale;
  float* dpost;
  float* dpre;
  // sums over a workgroup's rows, [blocks][width] each: of a e bh, of dh rh,
  // and, with gate rows shared and their rows cut, of e bh
  float* part_total;
  float* part_pre;
  float* part_gate;
  int blocks;
  // gate rows shared: groups of gate_rows rows, each a worker's; or cut: each in
  // `parts` parts of part_rows rows, a workgroup's
  int64_t groups, part_rows;
  int parts, cut;
};

// One vector of a row, as stored, with one load and no branch: a vector that
// would pass the row's end is the row's last V elements instead, and settle()
// moves them down to where they belong, with zeros behind the row's end.
// kNarrow: a row of less than V elements, which is taken element by element (by
// kernels of its own: in the others that path costs registers and time).
template <class T, int V, bool kNarrow>
__device__ __forceinline__ Vec<T, V> load_cols(const T* row, int col, int width) {
  if constexpr (!kNarrow) return load<T, V>(row + min(col, width - V));
  Vec<T, V> v = {};
  if (col == 0) {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (k < width) v[k] = row[k];
  }
  return v;
}
template <class T, int V, bool kNarrow>
__device__ __forceinline__ void settle(Vec<T, V>& v, int col, int width) {
  int shift = col + V - width;  // elements
  if (kNarrow || shift <= 0) return;
  constexpr int kWords = V * (int)sizeof(T) / 4;
  union {
    Vec<T, V> v;
    uint32_t w[kWords];
  } u = {v};
  if constexpr (sizeof(T) == 2) {
    if (shift & 1) {
#pragma unroll
      for (int k = 0; k < kWords; ++k)
        u.w[k] = (u.w[k] >> 16) | (k + 1 < kWords ? u.w[k + 1] << 16 : 0u);
    }
    shift >>= 1;
  }
#pragma unroll
  for (int step = 1; step < kWords; step *= 2) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      const uint32_t from = k + step < kWords ? u.w[k + step] : 0u;
      u.w[k] = (shift & step) ? from : u.w[k];
    }
  }
#pragma unroll
  for (int k = 0; k < kWords; ++k) u.w[k] = shift >= kWords ? 0u : u.w[k];
  v = u.v;
}
template <class T, int V>
__device__ __forceinline__ void store_cols(T* row, int col, int width, Wide<V> w) {
  const Vec<T, V> v = narrow<T, V>(w);
  if (col + V <= width) {
    if constexpr (sizeof(T) == 2) store_once<T, V>(row + col, v);
    else store<T, V>(row + col, v);
    return;
  }
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (col + k < width) row[col + k] = v[k];
}
// a weight's columns; 1 where there is none
template <int V, bool kNarrow>
__device__ __forceinline__ Wide<V> load_weight(const float* w, int col, int width) {
  if (w) {
    Vec<float, V> v = load_cols<float, V, kNarrow>(w, col, width);
    settle<float, V, kNarrow>(v, col, width);
    return v;
  }
  Wide<V> one;
#pragma unroll
  for (int k = 0; k < V; ++k) one[k] = 1.0f;
  return one;
}

// a / b of numbers >= 0, which rarely need 64 bits
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// act(g).  fp32 tensors take the exact exponential and quotient; for half types
// the fast ones (errors of one step each, and a few 2^-24 of the argument) are
// far below their rounding.
template <class TB>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (sizeof(TB) == 4) return 1.0f / (1.0f + expf(-g));
  else return __builtin_amdgcn_rcpf(1.0f + __expf(-g));
}
// act'(g) of an a = sigmoid(g).  1 - a of an open gate is a exp(-g): taken from
// the rounded a it would be off by all that a's last bit is of it (g = 12: 0.9%,
// g = 17: the whole).
template <class TB>
__device__ __forceinline__ float sigmoid_slope(float g, float a) {
  const float e = sizeof(TB) == 4 ? expf(-g) : __expf(-g);
  return a * (g > 0.0f ? a * e : 1.0f - a);
}
// (the branch is once for all: one for each element left nothing to overlap)
template <class TB, int V>
__device__ __forceinline__ Wide<V> activate(Wide<V> g, int act) {
  if (act == SSIM_GATE_SIGMOID) {
#pragma unroll
    for (int k = 0; k < V; ++k) g[k] = sigmoid<TB>(g[k]);
  }
  return g;
}

template <class TB, int V>
__device__ __forceinline__ Wide<V> slope(Wide<V> g, Wide<V> a) {
#pragma unroll
  for (int k = 0; k < V; ++k) g[k] = sigmoid_slope<TB>(g[k], a[k]);
  return g;
}

// 1 / sqrt(v), v >= 0: the instruction, which is off by a step, and one step of
// Newton's method, since a root's error is the whole row's.  The instruction
// takes subnormal numbers for 0, so they are scaled; 0 and infinity stay what it
// gives.
__device__ __forceinline__ float inv_root(float v) {
  const bool tiny = v < 0x1p-100f;
  const float w = tiny ? v * 0x1p60f : v;
  const float y = __builtin_amdgcn_rsqf(w);
  const float rest = fmaf(-w * y, y, 1.0f);
  const float z = fmaf(0.5f * y, rest, y);
  return (rest == rest ? z : y) * (tiny ? 0x1p30f : 1.0f);
}

// N sums over a row's threads at once.  kLanes: so many lanes of a wave hold the
// row; 0: the workgroup does, with lds[N][kWaves], whose entries past the
// workgroup's waves are zero.  Two calls that follow each other take different
// lds arrays: then the barrier within one separates the other's uses.
template <int kLanes, int N, int kWaves>
__device__ __forceinline__ void row_sums(float (&s)[N], float (*lds)[kWaves]) {
#pragma unroll
  for (int k = 0; k < N; ++k) s[k] = lanes_sum<kLanes ? kLanes : kWave>(s[k]);
  if constexpr (kLanes == 0) {
    if ((threadIdx.x & (kWave - 1)) == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) lds[k][threadIdx.x / kWave] = s[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float t = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) t += lds[k][w];
      s[k] = t;
    }
  }
}

// Which of a workgroup's rows this thread works on; a scalar where it is the
// whole wave's.
template <int kLanes>
__device__ __forceinline__ int worker_of() {
  if constexpr (kLanes == 0) return 0;
  else if constexpr (kLanes == kWave) return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  else return (int)threadIdx.x / kLanes;
}

// what the forward loads of one vector of a row
template <class TX, class TB, int V>
struct FwdRaw {
  Vec<TX, V> x;
  Vec<TB, V> b, gate;
};

// The first row's loads are issued before the weights', each other's at the end
// of the row before it or (kEarly) at its start.
template <class TX, class TB, int I, int kLanes, int kWaves, bool kEarly, bool kNarrow>
__device__ __forceinline__ void norm_forward(const NormParams& p) {
  constexpr int V = 16 / sizeof(TB);
  __shared__ float lds[2][1][kWaves];
  const int width = p.width;
  const int threads = kLanes ? kLanes : (int)blockDim.x;
  const int q = kLanes ? (int)threadIdx.x & (kLanes - 1) : (int)threadIdx.x;
  constexpr int kWorkers = kLanes ? kRowWaves * kWave / kLanes : 1;
  const int64_t stride = (int64_t)gridDim.x * kWorkers;
  int64_t row = (int64_t)blockIdx.x * kWorkers + worker_of<kLanes>();
  // the gate row of the row that is fetched next, and how far into its rows
  // that one lies; kept by addition, since a quotient costs as much as a row
  int64_t gate_row = row, gate_at = 0, gate_step = stride, gate_rest = 0;
  if (p.gate_rows > 1) {
    gate_row = quotient(row, p.gate_rows);
    gate_at = row - gate_row * p.gate_rows;
    gate_step = quotient(stride, p.gate_rows);
    gate_rest = stride - gate_step * p.gate_rows;
  }
  FwdRaw<TX, TB, V> next[I];
  auto fetch = [&](int64_t of) {
    const TB* b = (const TB*)p.b + of * width;
    const TX* x = (const TX*)p.x + of * width;
    const TB* gate = (const TB*)p.gate + gate_row * width;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int col = (i * threads + q) * V;
      next[i].b = load_cols<TB, V, kNarrow>(b, col, width);
      next[i].x = load_cols<TX, V, kNarrow>(x, col, width);
      next[i].gate = 0;
      if (p.gate) next[i].gate = load_cols<TB, V, kNarrow>(gate, col, width);
    }
    gate_row += gate_step;
    gate_at += gate_rest;
    if (gate_at >= p.gate_rows) {
      gate_at -= p.gate_rows;
      ++gate_row;
    }
  };
  if (row < p.rows) fetch(row);
  if constexpr (kLanes == 0) {
    if (threadIdx.x < 2 * kWaves) (&lds[0][0][0])[threadIdx.x] = 0;
    __syncthreads();
  }
  // (16 waves have not the registers for the weights: each row's are loaded
  // anew, and the compiler may not see that they are the same ones)
  constexpr bool kAnew = kWaves == kWideWaves;
  Wide<V> c[I], pre[I];
  auto load_inner = [&](int i) {
    int at = q;
    if constexpr (kAnew) asm volatile("" : "+v"(at));
    const int col = (i * threads + at) * V;
    c[i] = load_weight<V, kNarrow>(p.scale, col, width) * load_weight<V, kNarrow>(p.post, col, width);
  };
  auto load_outer = [&](int i) {
    int at = q;
    if constexpr (kAnew) asm volatile("" : "+v"(at));
    pre[i] = load_weight<V, kNarrow>(p.pre, (i * threads + at) * V, width);
  };
  if constexpr (!kAnew) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
      load_inner(i);
      load_outer(i);
    }
  }
  for (; row < p.rows; row += stride) {
    FwdRaw<TX, TB, V> raw[I];
#pragma unroll
    for (int i = 0; i < I; ++i) raw[i] = next[i];
    const bool more = row + stride < p.rows;
    if (kEarly && more) fetch(row + stride);
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int col = (i * threads + q) * V;
      settle<TB, V, kNarrow>(raw[i].b, col, width);
      settle<TX, V, kNarrow>(raw[i].x, col, width);
      if (p.gate) settle<TB, V, kNarrow>(raw[i].gate, col, width);
    }
    float s[1] = {0};
    Wide<V> v[I], ac[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
      v[i] = widen<TB, V>(raw[i].b);
#pragma unroll
      for (int k = 0; k < V; ++k) s[0] = fmaf(v[i][k], v[i][k], s[0]);
      if constexpr (kAnew) load_inner(i);
      ac[i] = c[i];
      if (p.gate) ac[i] *= activate<TB, V>(widen<TB, V>(raw[i].gate), p.act);
    }
    row_sums<kLanes>(s, lds[0]);
    const float ib = inv_root(fmaf(s[0], p.inv_width, p.eps));
    s[0] = 0;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const Wide<V> xw = widen<TX, V>(raw[i].x);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float r = fmaf(ac[i][k], v[i][k] * ib, xw[k]);
        v[i][k] = r;
        s[0] = fmaf(r, r, s[0]);
      }
    }
    // (columns past the row's end hold zeros, so they add nothing)
    row_sums<kLanes>(s, lds[1]);
    const float ir = inv_root(fmaf(s[0], p.inv_width, p.eps));
    TX* r = (TX*)p.r + row * width;
    TB* h = (TB*)p.h + row * width;
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int col = (i * threads + q) * V;
      if (col >= width) continue;
      if constexpr (kAnew) load_outer(i);
      store_cols<TX, V>(r, col, width, v[i]);
      store_cols<TB, V>(h, col, width, v[i] * ir * pre[i]);
    }
    if (p.stats && q == 0) {
      p.stats[2 * row] = ib;
      p.stats[2 * row + 1] = ir;
    }
    if (!kEarly && more) fetch(row + stride);
  }
}

// what the backward loads of one vector of a row
template <class TX, class TB, int V>
struct Raw {
  Vec<TX, V> x, dr;
  Vec<TB, V> b, dh, gate;
};
template <class TX, class TB, int V, bool kGrouped, bool kNarrow>
__device__ __forceinline__ Raw<TX, TB, V> load_raw(const NormParams& p, int64_t at, int col) {
  Raw<TX, TB, V> f;
  f.b = load_cols<TB, V, kNarrow>((const TB*)p.b + at, col, p.width);
  f.x = load_cols<TX, V, kNarrow>((const TX*)p.x + at, col, p.width);
  f.gate = 0;
  f.dr = 0;
  f.dh = 0;
  if (!kGrouped && p.gate) f.gate = load_cols<TB, V, kNarrow>((const TB*)p.gate + at, col, p.width);
  if (p.dr) f.dr = load_cols<TX, V, kNarrow>((const TX*)p.dr + at, col, p.width);
  if (p.dh) f.dh = load_cols<TB, V, kNarrow>((const TB*)p.dh + at, col, p.width);
  return f;
}
template <class TX, class TB, int V, bool kGrouped, bool kNarrow>
__device__ __forceinline__ void settle_raw(Raw<TX, TB, V>& f, int col, int width) {
  settle<TB, V, kNarrow>(f.b, col, width);
  settle<TX, V, kNarrow>(f.x, col, width);
  settle<TX, V, kNarrow>(f.dr, col, width);
  settle<TB, V, kNarrow>(f.dh, col, width);
  if constexpr (!kGrouped) settle<TB, V, kNarrow>(f.gate, col, width);
}
// and forms of it (names as below)
template <int V>
struct Terms {
  Wide<V> bh, rh, u, a;
};
template <class TX, class TB, int V, bool kGrouped>
__device__ __forceinline__ Terms<V> form_terms(const NormParams& p, const Raw<TX, TB, V>& raw,
                                               Wide<V> dw, float ib, float ir, Wide<V> c,
                                               Wide<V> pre, Wide<V> group_a) {
  Terms<V> f;
  if constexpr (kGrouped) {
    f.a = group_a;
  } else if (p.gate) {
    f.a = activate<TB, V>(widen<TB, V>(raw.gate), p.act);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) f.a[k] = 1.0f;
  }
  f.bh = widen<TB, V>(raw.b) * ib;
  const Wide<V> x = widen<TX, V>(raw.x), dr = widen<TX, V>(raw.dr);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    f.rh[k] = fmaf(f.a[k] * c[k], f.bh[k], x[k]) * ir;
    f.u[k] = fmaf(ir, dw[k] * pre[k], dr[k]);
  }
  return f;
}

// The gradients.  With wd = dh pre, rh = r ir, u = dr + ir wd:
//   e  = u - ir rh mean(wd rh)              the gradient of x
//   t  = e a c,  db = ib (t - bh mean(t bh))
//   dg = e c bh act'(g)
//   dscale = post sum_rows(a e bh), dpost = scale (the same sum), dpre = sum_rows(dh rh)
// mean(t bh) = mean(u ac bh) - ir mean(wd rh) mean(rh ac bh): with the two
// reciprocal roots kept by the forward, one reduction of three sums serves
// both norms.  r is formed again from x, so that its rounding to x's type does
// not enter.
// kGrouped: one gate row for many rows.  Then only S = sum of e bh is summed
// over a group's rows, and dg = c act'(g) S, sum of a e bh = a S.
// kReload: a thread of a very wide row cannot hold it; its vectors, the weights'
// and the gate's are loaded again, from the caches, after the reduction, and its
// sums over rows lie in LDS.
template <class TX, class TB, int I, int kLanes, bool kGrouped, bool kNarrow, bool kReload>
__device__ __forceinline__ void norm_backward(const NormParams& p) {
  constexpr int V = 16 / sizeof(TB);
  constexpr int kWaves = kReload ? kWideWaves : kMaxWaves;
  // (two vectors of a thread twice over do not fit its registers, unless the
  // group's are missing)
  constexpr bool kPrefetch = kReload || I == 1 || (I == 2 && kLanes && !kGrouped);
  __shared__ float lds[2][3][kWaves];
  if constexpr (kLanes == 0) {
    for (int k = threadIdx.x; k < 6 * kWaves; k += blockDim.x) (&lds[0][0][0])[k] = 0;
    __syncthreads();
  }
  const int width = p.width;
  const int threads = kLanes ? kLanes : (int)blockDim.x;
  const int q = kLanes ? (int)threadIdx.x & (kLanes - 1) : (int)threadIdx.x;
  const int worker = worker_of<kLanes>();
  constexpr int kWorkers = kLanes ? kRowWavesBack * kWave / kLanes : 1;

  // The first column of this thread's vector i.  Where vectors are loaded again,
  // the compiler may not see that it is the same one: it would keep the values,
  // or their addresses, in registers that are not there.
  auto col_of = [&](int i) {
    int at = q;
    if constexpr (kReload) asm volatile("" : "+v"(at));
    return (i * threads + at) * V;
  };
  constexpr int kHeld = kReload ? 1 : I;  // vectors of the weights and of a row that stay
  Wide<V> c[kHeld], pre[kHeld], a[kGrouped ? kHeld : 1];
  // The sums over rows, S and total as above.  kReload: dpre and the one that
  // grows with each row lie in LDS, each thread's in a place of its own.
  constexpr int kRowSums = kReload ? 1 : I;
  Wide<V> dpre[kRowSums], S[kGrouped ? kRowSums : 1], total[kGrouped ? I : kRowSums];
  __shared__ __attribute__((aligned(32))) float kept[2][kReload ? kWaves * kWave * V * I : 8];
  auto kept_at = [&](int which, int i) -> Wide<V>& {
    return *reinterpret_cast<Wide<V>*>(&kept[which][kReload ? (i * threads + q) * V : 0]);
  };
  auto dpre_at = [&](int i) -> Wide<V>& {
    if constexpr (kReload) return kept_at(0, i);
    else return dpre[i];
  };
  auto S_at = [&](int i) -> Wide<V>& {
    if constexpr (kReload) return kept_at(1, i);
    else return S[kGrouped ? i : 0];
  };
  auto total_at = [&](int i) -> Wide<V>& {
    if constexpr (kReload && !kGrouped) return kept_at(1, i);
    else return total[i];
  };
  auto load_weights = [&](int i, int col) {
    const int to = kReload ? 0 : i;
    c[to] = load_weight<V, kNarrow>(p.scale, col, width) * load_weight<V, kNarrow>(p.post, col, width);
    pre[to] = load_weight<V, kNarrow>(p.pre, col, width);
  };
  auto group_gate = [&](int64_t group, int col) {
    Vec<TB, V> g = load_cols<TB, V, kNarrow>((const TB*)p.gate + group * width, col, width);
    settle<TB, V, kNarrow>(g, col, width);
    return g;
  };
  auto load_gate = [&](int64_t group, int i, int col) {
    a[kReload ? 0 : i] = activate<TB, V>(widen<TB, V>(group_gate(group, col)), p.act);
  };
#pragma unroll
  for (int i = 0; i < I; ++i) {
    if constexpr (!kReload) load_weights(i, col_of(i));
    total_at(i) = 0;
    dpre_at(i) = 0;
  }

  // the segments of rows this worker takes: all rows, dealt out one by one;
  // or groups, or parts of a group
  int64_t seg = 0, segs = 1, seg_stride = 1;
  int parity = 0;  // of the reductions' lds arrays, over all rows
  if constexpr (kGrouped) {
    segs = p.groups * p.parts;
    seg = blockIdx.x;
    seg_stride = gridDim.x;
    if (!p.cut) {
      seg = seg * kWorkers + worker;
      seg_stride *= kWorkers;
    }
  }
  for (; seg < segs; seg += seg_stride) {
    int64_t row, end, stride, group = 0;
    if constexpr (kGrouped) {
      group = quotient(seg, p.parts);
      const int64_t part = seg - group * p.parts;
      row = group * p.gate_rows + part * p.part_rows;
      end = row + p.part_rows;
      if (end > (group + 1) * p.gate_rows) end = (group + 1) * p.gate_rows;
      stride = 1;
      if (p.cut) {
        row += worker;
        stride = kWorkers;
      }
#pragma unroll
      for (int i = 0; i < I; ++i) {
        if constexpr (!kReload) load_gate(group, i, col_of(i));
        S_at(i) = 0;
      }
    } else {
      row = (int64_t)blockIdx.x * kWorkers + worker;
      stride = (int64_t)gridDim.x * kWorkers;
      end = p.rows;
    }
    // a row's loads are issued while the row before it is worked on
    Raw<TX, TB, V> next[kHeld];
    float next_ib = 0, next_ir = 0;
    auto fetch = [&](int64_t of) {
      if constexpr (!kReload) {
#pragma unroll
        for (int i = 0; i < I; ++i)
          next[i] = load_raw<TX, TB, V, kGrouped, kNarrow>(p, of * width, col_of(i));
      }
      next_ib = p.stats[2 * of];
      next_ir = p.stats[2 * of + 1];
    };
    if (kPrefetch && row < end) fetch(row);
    for (; row < end; row += stride, parity ^= 1) {
      const int64_t at = row * width;
      Raw<TX, TB, V> raw[kHeld];
      if (!kPrefetch) fetch(row);
      if constexpr (!kReload) {
#pragma unroll
        for (int i = 0; i < I; ++i) raw[i] = next[i];
      }
      const float ib = next_ib, ir = next_ir;
      if (kPrefetch && row + stride < end) fetch(row + stride);
      float s[3] = {0, 0, 0};
      Terms<V> terms[kHeld];
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const int col = col_of(i), j = kReload ? 0 : i;
        if constexpr (kReload) {
          __builtin_amdgcn_sched_barrier(0);  // one vector at a time, for its registers
          load_weights(i, col);
          if constexpr (kGrouped) load_gate(group, i, col);
          raw[j] = load_raw<TX, TB, V, kGrouped, kNarrow>(p, at, col);
        }
        settle_raw<TX, TB, V, kGrouped, kNarrow>(raw[j], col, width);
        const Wide<V> dw = widen<TB, V>(raw[j].dh);
        const Terms<V> f = form_terms<TX, TB, V, kGrouped>(p, raw[j], dw, ib, ir, c[j], pre[j],
                                                           a[kGrouped ? j : 0]);
        Wide<V> sum = dpre_at(i);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float acbh = f.a[k] * c[j][k] * f.bh[k];
          s[0] = fmaf(dw[k] * pre[j][k], f.rh[k], s[0]);
          s[1] = fmaf(f.u[k], acbh, s[1]);
          s[2] = fmaf(f.rh[k], acbh, s[2]);
          sum[k] = fmaf(dw[k], f.rh[k], sum[k]);
        }
        dpre_at(i) = sum;
        terms[j] = f;
      }
      row_sums<kLanes>(s, lds[parity]);
      const float m1 = ir * (s[0] * p.inv_width);
      const float m2 = s[1] * p.inv_width - m1 * (s[2] * p.inv_width);
      TX* dx = (TX*)p.dx + (p.dx ? at : 0);
      TB* db = (TB*)p.db + (p.db ? at : 0);
      TB* dg = (TB*)p.dg + (p.dg ? at : 0);
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const int col = col_of(i), j = kReload ? 0 : i;
        if constexpr (kReload) {
          __builtin_amdgcn_sched_barrier(0);
          load_weights(i, col);
          if constexpr (kGrouped) load_gate(group, i, col);
          raw[j] = load_raw<TX, TB, V, kGrouped, kNarrow>(p, at, col);
          settle_raw<TX, TB, V, kGrouped, kNarrow>(raw[j], col, width);
          terms[j] = form_terms<TX, TB, V, kGrouped>(p, raw[j], widen<TB, V>(raw[j].dh), ib, ir,
                                                     c[j], pre[j], a[kGrouped ? j : 0]);
        }
        const Terms<V>& f = terms[j];
        const Wide<V> e = f.u - f.rh * m1, eb = e * f.bh;
        if constexpr (kGrouped) S_at(i) += eb;
        else total_at(i) += eb * f.a;
        if (col >= width) continue;
        if (p.dx) store_cols<TX, V>(dx, col, width, e);
        if (p.db) store_cols<TB, V>(db, col, width, (e * (f.a * c[j]) - f.bh * m2) * ib);
        if constexpr (!kGrouped) {
          if (p.dg) {
            Wide<V> d = eb * c[j];
            if (p.act == SSIM_GATE_SIGMOID) d *= slope<TB, V>(widen<TB, V>(raw[j].gate), f.a);
            store_cols<TB, V>(dg, col, width, d);
          }
        }
      }
    }
    if constexpr (kGrouped) {
      TB* dg = (TB*)p.dg + (p.dg ? group * width : 0);
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const int col = col_of(i), j = kReload ? 0 : i;
        if constexpr (kReload) {
          __builtin_amdgcn_sched_barrier(0);
          load_weights(i, col);
          load_gate(group, i, col);
        }
        total_at(i) += S_at(i) * a[j];
        if (!p.cut && p.dg && col < width) {
          Wide<V> d = S_at(i) * c[j];
          if (p.act == SSIM_GATE_SIGMOID) d *= slope<TB, V>(widen<TB, V>(group_gate(group, col)), a[j]);
          store_cols<TB, V>(dg, col, width, d);
        }
      }
    }
  }

  // the workgroup's sums
  float* out[3] = {p.part_total, p.part_pre, kGrouped && p.cut ? p.part_gate : nullptr};
#pragma unroll
  for (int k = 0; k < (kGrouped ? 3 : 2); ++k) {
    if (!out[k]) continue;
    float* to = out[k] + (int64_t)blockIdx.x * width;
    if constexpr (kLanes != 0) {
      __shared__ float rows[kWorkers][kLanes * V * I];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < I; ++i) {
        Wide<V> v;
        if constexpr (kGrouped) v = k == 0 ? total_at(i) : k == 1 ? dpre_at(i) : S_at(i);
        else v = k == 0 ? total_at(i) : dpre_at(i);
#pragma unroll
        for (int e = 0; e < V; ++e) rows[worker][(i * kLanes + q) * V + e] = v[e];
      }
      __syncthreads();
      for (int col = threadIdx.x; col < width; col += kRowWavesBack * kWave) {
        float v = 0;
#pragma unroll
        for (int w = 0; w < kWorkers; ++w) v += rows[w][col];
        to[col] = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const int col = (i * threads + q) * V;
        Wide<V> v;
        if constexpr (kGrouped) v = k == 0 ? total_at(i) : k == 1 ? dpre_at(i) : S_at(i);
        else v = k == 0 ? total_at(i) : dpre_at(i);
        if (col < width) store_cols<float, V>(to, col, width, v);
      }
    }
  }
}

// The last sums, in fp64 over the workgroups' partial sums.  blockIdx.y: 0 the
// scale's and the post weight's gradients, 1 the pre weight's, 2 + g the
// gradient of gate row g (where its rows were cut).
template <class TB>
__device__ __forceinline__ void norm_sums(const NormParams& p) {
  __shared__ double lds[kSumSlices][kSumColumns];
  const int lane = threadIdx.x % kSumColumns, slice = threadIdx.x / kSumColumns;
  const int col = blockIdx.x * kSumColumns + lane;
  const int job = blockIdx.y;
  const float* from = job == 0 ? p.part_total : job == 1 ? p.part_pre : p.part_gate;
  int64_t n = p.blocks;
  if (job >= 2) {
    n = p.parts;
    from += (int64_t)(job - 2) * p.parts * p.width;
  }
  if ((job == 0 && !p.dscale && !p.dpost) || (job == 1 && !p.dpre)) return;
  double s = 0;
  if (col < p.width) {
#pragma unroll 8
    for (int64_t k = slice; k < n; k += kSumSlices) s += (double)from[k * p.width + col];
  }
  lds[slice][lane] = s;
  __syncthreads();
  if (slice != 0 || col >= p.width) return;
  s = 0;
#pragma unroll
  for (int k = 0; k < kSumSlices; ++k) s += lds[k][lane];
  if (job == 0) {
    if (p.dscale) p.dscale[col] = (float)(s * (p.post ? (double)p.post[col] : 1.0));
    if (p.dpost) p.dpost[col] = (float)(s * (p.scale ? (double)p.scale[col] : 1.0));
  } else if (job == 1) {
    p.dpre[col] = (float)s;
  } else {
    const int64_t at = (int64_t)(job - 2) * p.width + col;
    const float g = (float)((const TB*)p.gate)[at];
    double d = s * (p.scale ? (double)p.scale[col] : 1.0) * (p.post ? (double)p.post[col] : 1.0);
    if (p.act == SSIM_GATE_SIGMOID) d *= (double)sigmoid_slope<TB>(g, sigmoid<TB>(g));
    ((TB*)p.dg)[at] = (TB)(float)d;
  }
}

// ---- the kernels of one block type
// How a row is spread: over so many lanes of a wave, or a workgroup of at most
// so many waves; vectors a thread.
enum NormShape {
  kNarrow,  // 8 lanes, less than a vector
  kLanes8,  // 8 lanes, one vector
  kLanes16, // 16 lanes, one
  kLanes32, // 32 lanes, one
  kWave1,   // one wave, one
  kWave2,   // one wave, two
  kGroup1,  // 4 waves, one
  kGroup1w, // 8 waves, one
  kGroup2,  // 8 waves, two
  kGroup4,  // 8 waves, four
  kGroup8,  // 8 waves, eight (fp32 blocks)
  kNormShapes
};
constexpr int shape_lanes(int s) {  // 0: a workgroup's row
  return s <= kLanes8 ? 8 : s == kLanes16 ? 16 : s == kLanes32 ? 32 : s <= kWave2 ? kWave : 0;
}
constexpr int shape_items(int s) {
  return s == kWave2 || s == kGroup2 ? 2 : s == kGroup4 ? 4 : s == kGroup8 ? 8 : 1;
}
constexpr int shape_threads(int s, int row_waves) {
  return (shape_lanes(s) ? row_waves : s == kGroup1 ? 4 : kMaxWaves) * kWave;
}
// A thread of the backward that would hold more than 16 elements of a row has
// not the registers: workgroups of twice as many threads load them twice and keep
// their sums over rows in 128 KB of LDS.  Forward and gradients of 2000 x 16384 in
// bf16 201 us (sums in registers, some of them spilled to memory, 346; elements
// held by eight waves, half of them spilled, 920), of 2000 x 12288 in fp16 without
// a gate 119 (246).
constexpr bool shape_reload(int s, int bytes) { return shape_items(s) * 16 / bytes > 16; }
constexpr int shape_items(int s, int bytes) {
  return shape_reload(s, bytes) ? shape_items(s) / 2 : shape_items(s);
}
constexpr int shape_threads(int s, int row_waves, int bytes) {
  return shape_reload(s, bytes) ? kWideWaves * kWave : shape_threads(s, row_waves);
}
// The forward takes 16 waves for such rows where x is fp32 (fp32, 2000 x 10000: 93
// us, with eight 201; bf16 beside fp32, 2000 x 16384: 95 and 104), eight for half
// types alone (2000 x 16384 bf16 60 us, with 16 64).
constexpr bool shape_fwd_wide(int s, int x_bytes, int bytes) {
  return x_bytes == 4 && shape_reload(s, bytes);
}
constexpr int shape_fwd_items(int s, int x_bytes, int bytes) {
  return shape_fwd_wide(s, x_bytes, bytes) ? shape_items(s, bytes) : shape_items(s);
}
constexpr int shape_fwd_threads(int s, int x_bytes, int bytes) {
  return shape_fwd_wide(s, x_bytes, bytes) ? kWideWaves * kWave : shape_threads(s, kRowWaves);
}
// A workgroup of eight waves to a row waits at its barriers with few others
// beside it; there the next row's loads go out at its start, as long as a thread
// has the registers for them (one or two vectors).  Where many waves are resident
// that gains nothing.
constexpr bool shape_early(int s) { return s == kGroup1w || s == kGroup2; }

struct NormTable {
  const void* forward[2][kNormShapes];      // [x is fp32 beside a half type]
  const void* backward[2][kNormShapes][2];  // [.. ][gate rows shared]
  const void* sums;
};

const NormTable& norm_table_f32();
const NormTable& norm_table_f16();
const NormTable& norm_table_bf16();

template <class TX, class TB, int kShape>
__global__ __launch_bounds__(shape_fwd_threads(kShape, sizeof(TX), sizeof(TB))) void
ssim_block_norm_fwd_kernel(const NormParams p) {
  norm_forward<TX, TB, shape_fwd_items(kShape, sizeof(TX), sizeof(TB)), shape_lanes(kShape),
               shape_fwd_wide(kShape, sizeof(TX), sizeof(TB)) ? kWideWaves : kMaxWaves, shape_early(kShape),
               kShape == kNarrow>(p);
}
template <class TX, class TB, int kShape, bool kGrouped>
__global__ __launch_bounds__(shape_threads(kShape, kRowWavesBack, sizeof(TB))) void
ssim_block_norm_bwd_kernel(const NormParams p) {
  norm_backward<TX, TB, shape_items(kShape, sizeof(TB)), shape_lanes(kShape), kGrouped,
                kShape == kNarrow, shape_reload(kShape, sizeof(TB))>(p);
}
template <class TB>
__global__ __launch_bounds__(kSumColumns* kSumSlices) void ssim_block_norm_sums_kernel(
    const NormParams p) {
  norm_sums<TB>(p);
}

template <class TX, class TB, int kShape>
void fill_shape(NormTable& t, int wide) {
  if constexpr (!(sizeof(TB) == 2 && kShape == kGroup8)) {
    t.forward[wide][kShape] = (const void*)ssim_block_norm_fwd_kernel<TX, TB, kShape>;
    t.backward[wide][kShape][0] = (const void*)ssim_block_norm_bwd_kernel<TX, TB, kShape, false>;
    t.backward[wide][kShape][1] = (const void*)ssim_block_norm_bwd_kernel<TX, TB, kShape, true>;
  }
}
template <class TX, class TB>
void fill_types(NormTable& t, int wide) {
  fill_shape<TX, TB, kNarrow>(t, wide);
  fill_shape<TX, TB, kLanes8>(t, wide);
  fill_shape<TX, TB, kLanes16>(t, wide);
  fill_shape<TX, TB, kLanes32>(t, wide);
  fill_shape<TX, TB, kWave1>(t, wide);
  fill_shape<TX, TB, kWave2>(t, wide);
  fill_shape<TX, TB, kGroup1>(t, wide);
  fill_shape<TX, TB, kGroup1w>(t, wide);
  fill_shape<TX, TB, kGroup2>(t, wide);
  fill_shape<TX, TB, kGroup4>(t, wide);
  fill_shape<TX, TB, kGroup8>(t, wide);
}
template <class TB>
NormTable make_table() {
  NormTable t = {};
  fill_types<TB, TB>(t, 0);
  if constexpr (sizeof(TB) == 2) fill_types<F32, TB>(t, 1);
  t.sums = (const void*)ssim_block_norm_sums_kernel<TB>;
  return t;
}

}  // namespace ssim_train
