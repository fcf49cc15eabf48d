// update.hip -- the gradients of many tensors: their global norm, clipping by
// it, and AdamW with the clipping fused in.
//
// Two launches.  The first sums squares, one fp64 partial sum for each
// workgroup; every workgroup of the second adds up the partial sums (in one
// order, so all get the same clipping factor, without an atomic or a value
// that has to be cleared beforehand) and then scales or updates its share.
//
// The tensors reach a kernel as a table of runs in its arguments (no copy to
// the device, so a call can be captured).  Items that follow each other in
// memory in all their arrays are one run: a network whose parameters are
// packed in a bucket is a single run.  A run is cut into chunks of equal
// size; chunk numbers run through all runs.

#include <math.h>

#include <algorithm>
#include <vector>

#include "train_common.hpp"

namespace {

using namespace ssim_train;

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 2048;  // 256 CUs, 8 workgroups of 4 waves each
constexpr int kWaves = kThreads / kWave;

// What the first launch leaves for the second.
struct Scratch {
  double partial[kMaxBlocks];
  float step_size;  // lr / (1 - beta1^t)
  float decay;      // lr weight_decay
  float inv_bc2;    // 1 / (1 - beta2^t)
};

struct NormRun {
  const void* grad;
  int64_t n;
  uint32_t first;  // its first chunk
  int32_t dtype;
};
struct ClipRun {
  const void* grad;
  void* out;
  int64_t n;
  uint32_t first;
  int32_t dtype;
};
struct AdamRun {
  const void* grad;
  void* param;
  float* m;
  float* v;
  float* master;
  int64_t n;
  uint32_t first;
  int16_t grad_dtype, param_dtype;
};
// Tables sized so that a kernel's arguments stay below 4 KB, and one for few
// runs: a launch with 256 bytes of arguments costs 3.5 us of host time, with
// 3.6 KB 3.9 (six tensors of 118000 elements, clipped in two launches: 7.1 us a
// call with this table, 8.6 with the large one).
constexpr int kNormRuns = 144, kClipRuns = 112, kAdamRuns = 64, kFewRuns = 8;

// Advances the count of updates and forms the update's scalars, by one thread.
struct StepArgs {
  int64_t* step;  // NULL: no update follows
  const float* lr_device;
  double lr, beta1, beta2, weight_decay;
};
template <int N>
struct NormArgs {
  NormRun run[N];
  int count;
  uint32_t chunks;
  int add;  // to the partial sums of the launches before
  Scratch* scratch;
  StepArgs step;
};
template <int N>
struct ClipArgs {
  ClipRun run[N];
  int count;
  uint32_t chunks;
  int partials;
  double max_norm;
  float* norm;
  const Scratch* scratch;
};
template <int N>
struct AdamArgs {
  AdamRun run[N];
  int count;
  uint32_t chunks;
  int partials;  // 0: no clipping
  double max_norm;
  float* norm;
  const Scratch* scratch;
  float beta1, one_minus_beta1, beta2, one_minus_beta2, eps;
};
static_assert(sizeof(NormArgs<kNormRuns>) <= 4096 && sizeof(ClipArgs<kClipRuns>) <= 4096 &&
                  sizeof(AdamArgs<kAdamRuns>) <= 4096,
              "kernel arguments");

// the run that holds chunk c
template <class Run, int N>
__device__ __forceinline__ int find_run(const Run (&run)[N], int count, uint32_t c) {
  if constexpr (N == kFewRuns) {  // by comparing with all: their loads do not wait for each other
    int r = 0;
#pragma unroll
    for (int k = 1; k < N; ++k) r += k < count && run[k].first <= c ? 1 : 0;
    return r;
  }
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (run[mid].first <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v, double* lds) {
  v = wave_sum(v);
  if ((threadIdx.x & (kWave - 1)) == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  double s = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) s += lds[w];
  return s;
}

__device__ __forceinline__ void form_scalars(const StepArgs& s, int64_t t, float* step_size,
                                             float* decay, float* inv_bc2) {
  const double lr = s.lr_device ? (double)*s.lr_device : s.lr;
  double p1 = 1.0, p2 = 1.0, b1 = s.beta1, b2 = s.beta2;  // their t-th powers, by squaring
  for (int64_t k = t; k > 0; k >>= 1) {
    if (k & 1) {
      p1 *= b1;
      p2 *= b2;
    }
    b1 *= b1;
    b2 *= b2;
  }
  *step_size = (float)(lr / (1.0 - p1));
  *decay = (float)(lr * s.weight_decay);
  *inv_bc2 = (float)(1.0 / (1.0 - p2));
}

// ---- the sum of squares.  Reads each gradient once: bound by that read.
// Squares are formed and added in fp64 (two instructions an element, hidden
// behind the read), so no gradient's square over- or underflows.
template <class T, int U>
__device__ __forceinline__ double squares(const T* g, int64_t n) {
  constexpr int V = 16 / sizeof(T), C = kThreads * V;
  double acc[2] = {0, 0};
  const int64_t at = threadIdx.x * V;
  if (n >= (int64_t)C * U) {
    Vec<T, V> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = load<T, V>(g + at + u * C);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Wide<V> w = widen<T, V>(x[u]);
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k & 1] = fma((double)w[k], (double)w[k], acc[k & 1]);
    }
  } else {
    for (int u = 0; u < U; ++u) {
      const int64_t i = at + u * C;
      for (int k = 0; k < V && i + k < n; ++k) {
        const double w = (double)(float)g[i + k];
        acc[0] = fma(w, w, acc[0]);
      }
    }
  }
  return acc[0] + acc[1];
}

template <int U, int N>
__global__ __launch_bounds__(kThreads) void ssim_grad_norm_kernel(const NormArgs<N> a) {
  __shared__ double lds[kWaves];
  double acc = 0;
  for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const int r = find_run(a.run, a.count, c);
    const NormRun& run = a.run[r];
    const int64_t chunk = (int64_t)(16 / (run.dtype == SSIM_DTYPE_F32 ? 4 : 2)) * kThreads * U;
    const int64_t i = (int64_t)(c - run.first) * chunk;
    switch (run.dtype) {
      case SSIM_DTYPE_F32: acc += squares<F32, U>((const F32*)run.grad + i, run.n - i); break;
      case SSIM_DTYPE_F16: acc += squares<F16, U>((const F16*)run.grad + i, run.n - i); break;
      default: acc += squares<BF16, U>((const BF16*)run.grad + i, run.n - i); break;
    }
  }
  acc = block_sum(acc, lds);
  if (threadIdx.x == 0) {
    double* p = a.scratch->partial + blockIdx.x;
    *p = a.add ? *p + acc : acc;
    if (blockIdx.x == 0 && a.step.step) {
      const int64_t t = *a.step.step + 1;
      *a.step.step = t;
      form_scalars(a.step, t, &a.scratch->step_size, &a.scratch->decay, &a.scratch->inv_bc2);
    }
  }
}

// The clipping factor as two, which a gradient is multiplied by one after the
// other. Of a factor below 2^-126 fp32 holds fewer bits the smaller it is
// (gradients of 1e38 and more): then the first is a power of two, else 1.
struct Factor {
  float power, c;
};
__device__ __forceinline__ Factor factor_of(double norm, double max_norm) {
  if (isinf(max_norm)) return {1.0f, 1.0f};
  const double c = max_norm / (norm + 1e-6);
  if (c < 0x1p-126) return {0x1p-100f, (float)(c * 0x1p100)};
  return {1.0f, c > 1.0 ? 1.0f : (float)c};  // (a NaN stays one)
}

// the norm, from all partial sums, and the clipping factor; every workgroup
// computes the same
__device__ __forceinline__ Factor clip_factor(const Scratch* s, int partials, double max_norm,
                                             float* norm_out, double* lds) {
  double v = 0;
  for (int k = threadIdx.x; k < partials; k += kThreads) v += s->partial[k];
  const double norm = sqrt(block_sum(v, lds));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  return factor_of(norm, max_norm);
}

__global__ __launch_bounds__(kThreads) void ssim_norm_only_kernel(const Scratch* s, int partials,
                                                                  float* norm) {
  __shared__ double lds[kWaves];
  clip_factor(s, partials, 0.0, norm, lds);
}

// ---- clipping.  Reads each gradient again and writes it: bound by that.  The
// chunks are taken from the last to the first, since the first launch read the
// last ones last and the 256 MB last-level cache still holds them.
// U > 1: a list that the last-level cache does not hold; neither its second
// read nor the outputs are kept.
template <class T, int U>
__device__ __forceinline__ void scale(const T* g, T* out, int64_t n, Factor f) {
  constexpr int V = 16 / sizeof(T), C = kThreads * V;
  const int64_t at = threadIdx.x * V;
  if (n >= (int64_t)C * U) {
    Vec<T, V> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = load_as<U != 1, T, V>(g + at + u * C);
#pragma unroll
    for (int u = 0; u < U; ++u)
      store_as<U != 1, T, V>(out + at + u * C, narrow<T, V>(widen<T, V>(x[u]) * f.power * f.c));
  } else {
    for (int u = 0; u < U; ++u) {
      const int64_t i = at + u * C;
      for (int k = 0; k < V && i + k < n; ++k) out[i + k] = (T)((float)g[i + k] * f.power * f.c);
    }
  }
}

template <int U, int N>
__global__ __launch_bounds__(kThreads) void ssim_clip_grads_kernel(const ClipArgs<N> a) {
  __shared__ double lds[kWaves];
  const Factor f = clip_factor(a.scratch, a.partials, a.max_norm, a.norm, lds);
  for (uint32_t k = blockIdx.x; k < a.chunks; k += gridDim.x) {
    const uint32_t c = a.chunks - 1 - k;
    const int r = find_run(a.run, a.count, c);
    const ClipRun& run = a.run[r];
    if (f.c == 1.0f && f.power == 1.0f && run.grad == run.out) continue;  // in place and not clipped
    const int64_t chunk = (int64_t)(16 / (run.dtype == SSIM_DTYPE_F32 ? 4 : 2)) * kThreads * U;
    const int64_t i = (int64_t)(c - run.first) * chunk;
    switch (run.dtype) {
      case SSIM_DTYPE_F32:
        scale<F32, U>((const F32*)run.grad + i, (F32*)run.out + i, run.n - i, f);
        break;
      case SSIM_DTYPE_F16:
        scale<F16, U>((const F16*)run.grad + i, (F16*)run.out + i, run.n - i, f);
        break;
      default:
        scale<BF16, U>((const BF16*)run.grad + i, (BF16*)run.out + i, run.n - i, f);
        break;
    }
  }
}

// ---- AdamW
struct Coefs {
  Factor clip;
  float step_size, decay, inv_bc2, beta1, omb1, beta2, omb2, eps;
};

__device__ __forceinline__ void adam_one(const Coefs& k, float g, float& m, float& v, float& w) {
  g = g * k.clip.power * k.clip.c;
  m = fmaf(k.beta1, m, k.omb1 * g);
  v = fmaf(k.beta2, v, k.omb2 * g * g);
  // The decay and the step are added up before they reach w: 1 - lr weight_decay
  // itself has but multiples of 2^-24 (of 1e-7, 1.2e-7; of 1e-8, none).  (An
  // infinite weight stays one.)
  const float step = k.step_size * (m / (sqrtf(v * k.inv_bc2) + k.eps));
  w -= fmaf(k.decay, isinf(w) ? 0.0f : w, step);
}

constexpr int kAdamV = 4;  // elements a thread takes at once: 16 bytes of each fp32 array

// kMaster: the weights are in w and p receives a rounded copy; else they are in p
template <class TG, class TP, bool kMaster, int U>
__device__ __forceinline__ void adam_chunk(const Coefs& k, const AdamRun& run, int64_t i0) {
  constexpr int V = kAdamV, C = kThreads * V;
  constexpr bool kOnce = U != 1;  // the state does not stay in the last-level cache till the next step
  const TG* g = (const TG*)run.grad + i0;
  TP* p = (TP*)run.param + i0;
  float* m = run.m + i0;
  float* v = run.v + i0;
  float* w = run.master + (kMaster ? i0 : 0);
  const int64_t n = run.n - i0;
  const int at = threadIdx.x * V;
  if (n >= (int64_t)C * U) {
    Vec<TG, V> xg[U];
    Vec<TP, V> xp[U];
    Wide<V> xm[U], xv[U], xw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      xg[u] = load<TG, V>(g + at + u * C);
      xm[u] = load_as<kOnce, float, V>(m + at + u * C);
      xv[u] = load_as<kOnce, float, V>(v + at + u * C);
      if constexpr (kMaster) xw[u] = load_as<kOnce, float, V>(w + at + u * C);
      else xp[u] = load_as<kOnce, TP, V>(p + at + u * C);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (!kMaster) xw[u] = widen<TP, V>(xp[u]);
      const Wide<V> gw = widen<TG, V>(xg[u]);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float em = xm[u][e], ev = xv[u][e], ew = xw[u][e];
        adam_one(k, gw[e], em, ev, ew);
        xm[u][e] = em;
        xv[u][e] = ev;
        xw[u][e] = ew;
      }
      store_as<kOnce, float, V>(m + at + u * C, xm[u]);
      store_as<kOnce, float, V>(v + at + u * C, xv[u]);
      if constexpr (kMaster) store_as<kOnce, float, V>(w + at + u * C, xw[u]);
      store_as<kOnce, TP, V>(p + at + u * C, narrow<TP, V>(xw[u]));
    }
  } else {
    for (int u = 0; u < U; ++u)
      for (int e = 0; e < V; ++e) {
        const int64_t i = at + u * C + e;
        if (i >= n) break;
        float em = m[i], ev = v[i], ew;
        if constexpr (kMaster) ew = w[i];
        else ew = (float)p[i];
        adam_one(k, (float)g[i], em, ev, ew);
        m[i] = em;
        v[i] = ev;
        if constexpr (kMaster) w[i] = ew;
        p[i] = (TP)ew;
      }
  }
}

template <class TG, class TP, int U>
__device__ __forceinline__ void adam_run(const Coefs& k, const AdamRun& run, int64_t i0) {
  if (run.master) adam_chunk<TG, TP, true, U>(k, run, i0);
  else adam_chunk<TG, TP, false, U>(k, run, i0);
}

template <int U, int N>
__global__ __launch_bounds__(kThreads) void ssim_adamw_kernel(const AdamArgs<N> a) {
  __shared__ double lds[kWaves];
  Coefs k;
  k.clip = a.partials ? clip_factor(a.scratch, a.partials, a.max_norm, a.norm, lds) : Factor{1.0f, 1.0f};
  k.step_size = a.scratch->step_size;
  k.decay = a.scratch->decay;
  k.inv_bc2 = a.scratch->inv_bc2;
  k.beta1 = a.beta1;
  k.omb1 = a.one_minus_beta1;
  k.beta2 = a.beta2;
  k.omb2 = a.one_minus_beta2;
  k.eps = a.eps;
  for (uint32_t b = blockIdx.x; b < a.chunks; b += gridDim.x) {
    const uint32_t c = a.chunks - 1 - b;
    const int r = find_run(a.run, a.count, c);
    const AdamRun& run = a.run[r];
    const int64_t i = (int64_t)(c - run.first) * (kThreads * kAdamV * U);
    switch (run.grad_dtype * 4 + run.param_dtype) {
      case SSIM_DTYPE_F32 * 4 + SSIM_DTYPE_F32: adam_run<F32, F32, U>(k, run, i); break;
      case SSIM_DTYPE_F16 * 4 + SSIM_DTYPE_F16: adam_run<F16, F16, U>(k, run, i); break;
      case SSIM_DTYPE_BF16 * 4 + SSIM_DTYPE_BF16: adam_run<BF16, BF16, U>(k, run, i); break;
      case SSIM_DTYPE_F32 * 4 + SSIM_DTYPE_F16: adam_run<F32, F16, U>(k, run, i); break;
      default: adam_run<F32, BF16, U>(k, run, i); break;
    }
  }
}

// ---- few gradients in one launch.  A launch costs some 4 us, as much as all of
// the work here, so one launch does both passes: every workgroup adds up the
// squares of all gradients by itself, from the caches, and then scales or
// updates its own share.  Runs are taken as one sequence of 16-byte vectors; a
// run's last one may be short.
constexpr int kSmallThreads = 1024, kSmallRuns = kFewRuns;
constexpr int kSmallShare = 256;  // vectors that a workgroup of AdamW updates at once

template <class Run>
struct SmallTable {
  Run run[kSmallRuns];
  uint32_t first[kSmallRuns + 1];  // vectors before each run; of all runs
};

// the run that holds vector v, by comparing with all of them (no waiting for
// memory, so a thread's vectors are found side by side)
template <class Run>
__device__ __forceinline__ int small_find(const SmallTable<Run>& t, uint32_t v) {
  int r = 0;
#pragma unroll
  for (int k = 1; k < kSmallRuns; ++k) r += v >= t.first[k] ? 1 : 0;
  return r;
}

// A field of run r without indexing the table in memory.
template <class V, class Run, class Get>
__device__ __forceinline__ V small_pick(const SmallTable<Run>& t, int r, Get get) {
  V v = get(t.run[0]);
#pragma unroll
  for (int k = 1; k < kSmallRuns; ++k) v = r == k ? get(t.run[k]) : v;
  return v;
}

// The squares of all gradients, by one workgroup.
template <class T, int V, class Run>
__device__ __forceinline__ double small_squares(const SmallTable<Run>& t, double* lds) {
  constexpr int U = 4;
  const uint32_t vectors = t.first[kSmallRuns];
  double acc[2] = {0, 0};
  for (uint32_t v0 = threadIdx.x; v0 < vectors; v0 += kSmallThreads * U) {
    Vec<T, V> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t v = v0 + u * kSmallThreads;
      x[u] = 0;
      if (v >= vectors) continue;
      const int r = small_find(t, v);
      const T* g = (const T*)small_pick<const void*>(t, r, [](const Run& q) { return q.grad; });
      const uint32_t n = small_pick<uint32_t>(t, r, [](const Run& q) { return (uint32_t)q.n; });
      uint32_t first = 0;
#pragma unroll
      for (int k = 1; k < kSmallRuns; ++k) first = r == k ? t.first[k] : first;
      const uint32_t i = (v - first) * V;
      if (i + V <= n) {
        x[u] = load<T, V>(g + i);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (i + k < n) x[u][k] = g[i + k];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Wide<V> w = widen<T, V>(x[u]);
#pragma unroll
      for (int k = 0; k < V; ++k) acc[k & 1] = fma((double)w[k], (double)w[k], acc[k & 1]);
    }
  }
  const double sum = wave_sum(acc[0] + acc[1]);
  if ((threadIdx.x & (kWave - 1)) == 0) lds[threadIdx.x / kWave] = sum;
  __syncthreads();
  double all = 0;
#pragma unroll
  for (int w = 0; w < kSmallThreads / kWave; ++w) all += lds[w];
  return all;
}

struct SmallClipArgs {
  SmallTable<ClipRun> table;
  double max_norm;
  float* norm;
};

// Not in place but for a single workgroup: the others still read the gradients.
template <class T>
__global__ __launch_bounds__(kSmallThreads) void ssim_clip_small_kernel(const SmallClipArgs a) {
  constexpr int V = 16 / sizeof(T);
  __shared__ double lds[kSmallThreads / kWave];
  const double norm = sqrt(small_squares<T, V>(a.table, lds));
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  const Factor f = factor_of(norm, a.max_norm);
  const uint32_t vectors = a.table.first[kSmallRuns];
  for (uint32_t v = blockIdx.x * kSmallThreads + threadIdx.x; v < vectors;
       v += gridDim.x * kSmallThreads) {
    const int r = small_find(a.table, v);
    uint32_t first = 0;
#pragma unroll
    for (int k = 1; k < kSmallRuns; ++k) first = r == k ? a.table.first[k] : first;
    const ClipRun run = {
        small_pick<const void*>(a.table, r, [](const ClipRun& q) { return q.grad; }),
        small_pick<void*>(a.table, r, [](const ClipRun& q) { return q.out; }),
        small_pick<int64_t>(a.table, r, [](const ClipRun& q) { return q.n; }), 0, 0};
    const int64_t i = (int64_t)(v - first) * V;
    const T* g = (const T*)run.grad + i;
    T* out = (T*)run.out + i;
    if (i + V <= run.n) {
      store<T, V>(out, narrow<T, V>(widen<T, V>(load<T, V>(g)) * f.power * f.c));
    } else {
      for (int k = 0; i + k < run.n; ++k) out[k] = (T)((float)g[k] * f.power * f.c);
    }
  }
}

struct SmallAdamArgs {
  SmallTable<AdamRun> table;  // of vectors of kAdamV elements
  double max_norm;
  float* norm;  // NULL: no clipping
  StepArgs step;
  float beta1, one_minus_beta1, beta2, one_minus_beta2, eps;
};

// Each workgroup reads the count of updates, so none may have advanced it: the
// workgroups count themselves in step[1] after their read, and the last one to
// do so writes both words.  Nobody waits for another.
template <class TG, class TP, bool kMaster>
__global__ __launch_bounds__(kSmallThreads) void ssim_adamw_small_kernel(const SmallAdamArgs a) {
  constexpr int V = kAdamV;
  __shared__ double lds[kSmallThreads / kWave];
  __shared__ float scalars[3];
  int64_t t = 0, before = -1;
  if (threadIdx.x == kSmallThreads - 1) {
    t = __hip_atomic_load(a.step.step, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1;
    before = __hip_atomic_fetch_add(a.step.step + 1, (int64_t)1, __ATOMIC_RELEASE,
                                    __HIP_MEMORY_SCOPE_AGENT);
    form_scalars(a.step, t, &scalars[0], &scalars[1], &scalars[2]);
  }
  Coefs k;
  k.clip = {1.0f, 1.0f};
  if (a.norm) {
    const double norm = sqrt(small_squares<TG, V>(a.table, lds));
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
    k.clip = factor_of(norm, a.max_norm);
  } else {
    __syncthreads();
  }
  k.step_size = scalars[0];
  k.decay = scalars[1];
  k.inv_bc2 = scalars[2];
  k.beta1 = a.beta1;
  k.omb1 = a.one_minus_beta1;
  k.beta2 = a.beta2;
  k.omb2 = a.one_minus_beta2;
  k.eps = a.eps;
  const uint32_t vectors = a.table.first[kSmallRuns];
  const uint32_t at = blockIdx.x * kSmallShare + threadIdx.x;
  const uint32_t end = threadIdx.x < kSmallShare ? vectors : 0;
  for (uint32_t v = at; v < end; v += gridDim.x * kSmallShare) {
    const int r = small_find(a.table, v);
    uint32_t first = 0;
#pragma unroll
    for (int q = 1; q < kSmallRuns; ++q) first = r == q ? a.table.first[q] : first;
    const int64_t i = (int64_t)(v - first) * V;
    const int64_t n = small_pick<int64_t>(a.table, r, [](const AdamRun& q) { return q.n; });
    const TG* g = (const TG*)small_pick<const void*>(a.table, r, [](const AdamRun& q) { return q.grad; }) + i;
    TP* p = (TP*)small_pick<void*>(a.table, r, [](const AdamRun& q) { return q.param; }) + i;
    float* m = small_pick<float*>(a.table, r, [](const AdamRun& q) { return q.m; }) + i;
    float* s = small_pick<float*>(a.table, r, [](const AdamRun& q) { return q.v; }) + i;
    float* w = small_pick<float*>(a.table, r, [](const AdamRun& q) { return q.master; });
    if constexpr (kMaster) w += i;
    if (i + V <= n) {
      const Wide<V> xg = widen<TG, V>(load<TG, V>(g));
      Wide<V> xm = load<float, V>(m), xv = load<float, V>(s), xw;
      if constexpr (kMaster) xw = load<float, V>(w);
      else xw = widen<TP, V>(load<TP, V>(p));
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float em = xm[e], ev = xv[e], ew = xw[e];
        adam_one(k, xg[e], em, ev, ew);
        xm[e] = em;
        xv[e] = ev;
        xw[e] = ew;
      }
      store<float, V>(m, xm);
      store<float, V>(s, xv);
      if constexpr (kMaster) store<float, V>(w, xw);
      store<TP, V>(p, narrow<TP, V>(xw));
    } else {
      for (int e = 0; i + e < n; ++e) {
        float em = m[e], ev = s[e], ew;
        if constexpr (kMaster) ew = w[e];
        else ew = (float)p[e];
        adam_one(k, (float)g[e], em, ev, ew);
        m[e] = em;
        s[e] = ev;
        if constexpr (kMaster) w[e] = ew;
        p[e] = (TP)ew;
      }
    }
  }
  if (before == (int64_t)gridDim.x - 1) {
    a.step.step[0] = t;
    a.step.step[1] = 0;
  }
}

// ------------------------------------------------------------------ host side
struct Span {
  uintptr_t begin, end;
  bool write;
};

// no written array may overlap another array (but a clip item's grad equal to
// its out, which the caller leaves out)
bool spans_clash(std::vector<Span>& spans) {
  auto less = [](const Span& a, const Span& b) { return a.begin < b.begin; };
  if (!std::is_sorted(spans.begin(), spans.end(), less)) std::sort(spans.begin(), spans.end(), less);
  uintptr_t end = 0, write_end = 0;  // of the arrays so far
  for (const Span& s : spans) {
    if (s.begin < write_end || (s.write && s.begin < end)) return true;
    if (s.end > end) end = s.end;
    if (s.write && s.end > write_end) write_end = s.end;
  }
  return false;
}

void add_span(std::vector<Span>& spans, const void* p, size_t bytes, bool write) {
  if (p && bytes) spans.push_back({(uintptr_t)p, (uintptr_t)p + bytes, write});
}

constexpr int64_t kMaxBytes = (int64_t)1 << 46;

// Groups runs into launches: at most kRuns runs and 2^31 chunks each.
template <class Run>
struct Launch {
  size_t begin, end;
  uint32_t chunks;
};

template <class Run, class ChunkOf>
bool plan(std::vector<Run>& runs, size_t most, ChunkOf chunk_of, std::vector<Launch<Run>>& out) {
  out.clear();
  size_t begin = 0;
  int64_t chunks = 0;
  for (size_t k = 0; k < runs.size(); ++k) {
    const int64_t size = chunk_of(runs[k]);
    const int64_t need = (runs[k].n + size - 1) / size;
    if (need > 0x7fffffff) return false;
    if (k - begin == most || chunks + need > 0x7fffffff) {
      out.push_back({begin, k, (uint32_t)chunks});
      begin = k;
      chunks = 0;
    }
    runs[k].first = (uint32_t)chunks;
    chunks += need;
  }
  if (begin < runs.size()) out.push_back({begin, runs.size(), (uint32_t)chunks});
  return true;
}

// (the launch's own status: the last error may be another call's)
int launch_list(const void* kernel, int grid, void** list, void* stream, int threads) {
  if (hipLaunchKernel(kernel, dim3(grid), dim3(threads), list, 0,
                      static_cast<hipStream_t>(stream)) != hipSuccess) {
    (void)hipGetLastError();
    return SSIM_ERR_HIP;
  }
  return SSIM_OK;
}
int launch_kernel(const void* kernel, int grid, void* args, void* stream, int threads = kThreads) {
  void* list[] = {args};
  return launch_list(kernel, grid, list, stream, threads);
}
int launch_norm_only(const Scratch* scratch, int partials, float* norm, void* stream) {
  void* list[] = {&scratch, &partials, &norm};
  return launch_list((const void*)ssim_norm_only_kernel, 1, list, stream, kThreads);
}

int grid_for(uint32_t chunks) { return chunks < (uint32_t)kMaxBlocks ? (int)chunks : kMaxBlocks; }

// A call that moves much streams: it takes larger chunks and leaves nothing in
// the caches but the gradients between the two launches.  Measured on four
// lists in turn, kept and streamed: clipping 66 MB of fp32 22.6 and 23.0 us,
// 141 MB 45.5 and 39.2, 283 MB 88 and 71; AdamW over 115 MB 29 and 28 us, 231 MB
// 54 and 49, 991 MB 224 and 191.  Larger chunks yet for clipping pay with many of
// them only (1416 MB: 359 us with two vectors a thread, 339 with eight; 141 MB
// in bf16: 40 and 52, since the last round of chunks leaves CUs idle).
constexpr int64_t kClipStreamBytes = (int64_t)96 << 20, kClipLargeBytes = (int64_t)512 << 20;
constexpr int64_t kAdamStreamBytes = (int64_t)128 << 20;
constexpr int kClipStreamU = 2, kClipLargeU = 8, kAdamStreamU = 4;

int clip_vectors(int64_t bytes) {
  return bytes > kClipLargeBytes ? kClipLargeU : bytes > kClipStreamBytes ? kClipStreamU : 1;
}

const void* const kNormFew[3] = {(const void*)ssim_grad_norm_kernel<1, kFewRuns>,
                                 (const void*)ssim_grad_norm_kernel<kClipStreamU, kFewRuns>,
                                 (const void*)ssim_grad_norm_kernel<kClipLargeU, kFewRuns>};
const void* const kNormMany[3] = {(const void*)ssim_grad_norm_kernel<1, kNormRuns>,
                                  (const void*)ssim_grad_norm_kernel<kClipStreamU, kNormRuns>,
                                  (const void*)ssim_grad_norm_kernel<kClipLargeU, kNormRuns>};
const void* const kClipFew[3] = {(const void*)ssim_clip_grads_kernel<1, kFewRuns>,
                                 (const void*)ssim_clip_grads_kernel<kClipStreamU, kFewRuns>,
                                 (const void*)ssim_clip_grads_kernel<kClipLargeU, kFewRuns>};
const void* const kClipMany[3] = {(const void*)ssim_clip_grads_kernel<1, kClipRuns>,
                                  (const void*)ssim_clip_grads_kernel<kClipStreamU, kClipRuns>,
                                  (const void*)ssim_clip_grads_kernel<kClipLargeU, kClipRuns>};
const void* const kAdamFew[2] = {(const void*)ssim_adamw_kernel<1, kFewRuns>,
                                 (const void*)ssim_adamw_kernel<kAdamStreamU, kFewRuns>};
const void* const kAdamMany[2] = {(const void*)ssim_adamw_kernel<1, kAdamRuns>,
                                  (const void*)ssim_adamw_kernel<kAdamStreamU, kAdamRuns>};

// The norm launches.  *partials: how many partial sums they leave.
int launch_norm(std::vector<NormRun>& runs, int64_t bytes, Scratch* scratch, const StepArgs& step,
                int* partials, void* stream) {
  const int U = clip_vectors(bytes);
  std::vector<Launch<NormRun>> launches;
  if (!plan(runs, kNormRuns,
            [&](const NormRun& r) { return (int64_t)(16 / elem_bytes(r.dtype)) * kThreads * U; },
            launches))
    return SSIM_ERR_OVERFLOW;
  int grid = 1;
  for (const auto& l : launches) grid = std::max(grid, grid_for(l.chunks));
  *partials = grid;
  if (launches.empty()) launches.push_back({0, 0, 0});
  auto launch = [&](auto& a, const void* const (&kernels)[3], size_t k) {
    const auto& l = launches[k];
    a.count = (int)(l.end - l.begin);
    if (a.count) memcpy(a.run, &runs[l.begin], a.count * sizeof(NormRun));
    a.chunks = l.chunks;
    a.add = k > 0;
    a.scratch = scratch;
    a.step = step;
    if (k > 0) a.step.step = nullptr;
    return launch_kernel(kernels[U == 1 ? 0 : U == kClipStreamU ? 1 : 2], grid, &a, stream);
  };
  if (runs.size() <= kFewRuns && launches.size() == 1) {
    NormArgs<kFewRuns> a;
    return launch(a, kNormFew, 0);
  }
  for (size_t k = 0; k < launches.size(); ++k) {
    NormArgs<kNormRuns> a;
    const int rc = launch(a, kNormMany, k);
    if (rc != SSIM_OK) return rc;
  }
  return SSIM_OK;
}

// The single launch takes up to this many elements (each workgroup reads them
// all), in at most kSmallRuns runs of one type.  Measured in one launch and in
// two, fp32: clipping 17700 elements 5.6 and 8.4 us, 32450 7.8 and 9.2; AdamW 6.9
// and 9.3, 8.9 and 9.4.
constexpr int64_t kSmallElements = 32 << 10;

// Fills the table if these runs go into a single launch.
template <class Run, class TypeOf>
bool fits_small(const std::vector<Run>& runs, TypeOf type_of, int vector, SmallTable<Run>* t) {
  if (runs.empty() || runs.size() > kSmallRuns) return false;
  int64_t vectors = 0;
  memset(t, 0, sizeof(*t));
  for (size_t k = 0; k < runs.size(); ++k) {
    if (type_of(runs[k]) != type_of(runs[0]) || runs[k].n > kSmallElements) return false;
    t->run[k] = runs[k];
    t->first[k] = (uint32_t)vectors;
    vectors += (runs[k].n + vector - 1) / vector;
  }
  for (size_t k = runs.size(); k <= kSmallRuns; ++k) t->first[k] = (uint32_t)vectors;
  return vectors * vector <= kSmallElements;
}

bool follows(const void* a, int64_t n, int bytes, const void* b) {
  return (const char*)a + n * bytes == (const char*)b;
}

int clip_impl(const ssim_clip_item* items, int64_t count, bool scales, double max_norm, float* norm,
              void* workspace, void* stream) {
  if (count < 0) return SSIM_ERR_SHAPE;
  if ((count > 0 && !items) || !norm || !workspace) return SSIM_ERR_NULL;
  if (scales && !(max_norm >= 0.0 && max_norm <= 1.7976931348623157e308)) return SSIM_ERR_VALUE;
  if (misaligned(norm, 4) || misaligned(workspace, 8)) return SSIM_ERR_SHAPE;
  std::vector<ClipRun> runs;
  int64_t total = 0, bytes = 0;  // elements, bytes read and written
  for (int64_t k = 0; k < count; ++k) {
    const ssim_clip_item& it = items[k];
    if (it.n < 0) return SSIM_ERR_SHAPE;
    if (it.n == 0) continue;
    if (!known_dtype(it.dtype)) return SSIM_ERR_DTYPE;
    if (!it.grad || (scales && !it.out)) return SSIM_ERR_NULL;
    const int eb = elem_bytes(it.dtype);
    if (misaligned(it.grad, eb) || (scales && misaligned(it.out, eb))) return SSIM_ERR_SHAPE;
    if (it.n > kMaxBytes / eb || (total += it.n) > kMaxBytes) return SSIM_ERR_OVERFLOW;
    bytes += 2 * it.n * eb;
    void* out = scales ? it.out : nullptr;
    if (!runs.empty()) {
      ClipRun& r = runs.back();
      if (r.dtype == it.dtype && follows(r.grad, r.n, eb, it.grad) &&
          (!scales || follows(r.out, r.n, eb, out))) {
        r.n += it.n;
        continue;
      }
    }
    runs.push_back({it.grad, out, it.n, 0, it.dtype});
  }
  std::vector<Span> spans;
  spans.reserve(2 * runs.size() + 2);
  for (const ClipRun& r : runs) {
    const size_t bytes = (size_t)r.n * elem_bytes(r.dtype);
    if (scales) add_span(spans, r.out, bytes, true);
    if (r.grad != r.out) add_span(spans, r.grad, bytes, false);
  }
  add_span(spans, norm, 4, true);
  add_span(spans, workspace, sizeof(Scratch), true);
  if (spans_clash(spans)) return SSIM_ERR_ALIAS;

  int rc = check_current_device();
  if (rc != SSIM_OK) return rc;

  SmallClipArgs small;
  if (scales && !runs.empty() &&
      fits_small(runs, [](const ClipRun& r) { return r.dtype; }, 16 / elem_bytes(runs[0].dtype),
                 &small.table)) {
    const int grid = (int)((small.table.first[kSmallRuns] + kSmallThreads - 1) / kSmallThreads);
    bool in_place = false;
    for (const ClipRun& r : runs) in_place |= r.grad == r.out;
    if (grid == 1 || !in_place) {
      small.max_norm = max_norm;
      small.norm = norm;
      const void* kernel = runs[0].dtype == SSIM_DTYPE_F32   ? (const void*)ssim_clip_small_kernel<F32>
                           : runs[0].dtype == SSIM_DTYPE_F16 ? (const void*)ssim_clip_small_kernel<F16>
                                                             : (const void*)ssim_clip_small_kernel<BF16>;
      return launch_kernel(kernel, grid, &small, stream, kSmallThreads);
    }
  }

  Scratch* scratch = static_cast<Scratch*>(workspace);
  std::vector<NormRun> norm_runs;
  norm_runs.reserve(runs.size());
  for (const ClipRun& r : runs) norm_runs.push_back({r.grad, r.n, 0, r.dtype});
  StepArgs none;
  memset(&none, 0, sizeof(none));
  const int U = clip_vectors(bytes);
  std::vector<Launch<ClipRun>> launches;
  if (scales &&
      !plan(runs, kClipRuns,
            [&](const ClipRun& r) { return (int64_t)(16 / elem_bytes(r.dtype)) * kThreads * U; },
            launches))
    return SSIM_ERR_OVERFLOW;
  int partials = 0;
  rc = launch_norm(norm_runs, bytes, scratch, none, &partials, stream);
  if (rc != SSIM_OK) return rc;
  if (launches.empty()) return launch_norm_only(scratch, partials, norm, stream);
  auto launch = [&](auto& a, const void* const (&kernels)[3], size_t k) {
    const auto& l = launches[k];
    a.count = (int)(l.end - l.begin);
    memcpy(a.run, &runs[l.begin], a.count * sizeof(ClipRun));
    a.chunks = l.chunks;
    a.partials = partials;
    a.max_norm = max_norm;
    a.norm = k == 0 ? norm : nullptr;
    a.scratch = scratch;
    return launch_kernel(kernels[U == 1 ? 0 : U == kClipStreamU ? 1 : 2], grid_for(l.chunks), &a,
                         stream);
  };
  if (runs.size() <= kFewRuns && launches.size() == 1) {
    ClipArgs<kFewRuns> a;
    return launch(a, kClipFew, 0);
  }
  // (the last tensors first: see the kernel)
  for (size_t k = launches.size(); k-- > 0;) {
    ClipArgs<kClipRuns> a;
    rc = launch(a, kClipMany, k);
    if (rc != SSIM_OK) return rc;
  }
  return SSIM_OK;
}

template <class TG, class TP>
const void* small_of(bool master) {
  return master ? (const void*)ssim_adamw_small_kernel<TG, TP, true>
                : (const void*)ssim_adamw_small_kernel<TG, TP, false>;
}
const void* adamw_small_kernel(const AdamRun& r) {
  const bool wide = r.grad_dtype == SSIM_DTYPE_F32, master = r.master != nullptr;
  switch (r.param_dtype) {
    case SSIM_DTYPE_F16: return wide ? small_of<F32, F16>(master) : small_of<F16, F16>(master);
    case SSIM_DTYPE_BF16: return wide ? small_of<F32, BF16>(master) : small_of<BF16, BF16>(master);
    default: return small_of<F32, F32>(master);
  }
}

int adamw_impl(const ssim_adamw_item* items, int64_t count, const ssim_adamw_options* o,
               int64_t* step, float* norm, void* workspace, void* stream) {
  if (count < 0) return SSIM_ERR_SHAPE;
  if ((count > 0 && !items) || !o || !step || !workspace) return SSIM_ERR_NULL;
  const double kMax = 1.7976931348623157e308;
  const bool clips = !(o->max_norm > kMax);  // (NaN: refused below)
  if (!(o->max_norm >= 0.0) || !(o->beta1 >= 0.0 && o->beta1 < 1.0) ||
      !(o->beta2 >= 0.0 && o->beta2 < 1.0) || !(o->eps >= 0.0 && o->eps <= kMax) ||
      !(o->weight_decay >= 0.0 && o->weight_decay <= kMax) ||
      (!o->lr_device && !(o->lr >= 0.0 && o->lr <= kMax)))
    return SSIM_ERR_VALUE;
  if (clips && !norm) return SSIM_ERR_NULL;
  if (misaligned(step, 8) || misaligned(norm, 4) || misaligned(workspace, 8) ||
      misaligned(o->lr_device, 4))
    return SSIM_ERR_SHAPE;
  std::vector<AdamRun> runs;
  int64_t total = 0, bytes = 0, grad_bytes = 0;
  for (int64_t k = 0; k < count; ++k) {
    const ssim_adamw_item& it = items[k];
    if (it.n < 0) return SSIM_ERR_SHAPE;
    if (it.n == 0) continue;
    if (!known_dtype(it.param_dtype) || !known_dtype(it.grad_dtype) ||
        (it.grad_dtype != it.param_dtype && it.grad_dtype != SSIM_DTYPE_F32))
      return SSIM_ERR_DTYPE;
    if (!it.grad || !it.param || !it.exp_avg || !it.exp_avg_sq) return SSIM_ERR_NULL;
    const int gb = elem_bytes(it.grad_dtype), pb = elem_bytes(it.param_dtype);
    if (misaligned(it.grad, gb) || misaligned(it.param, pb) || misaligned(it.exp_avg, 4) ||
        misaligned(it.exp_avg_sq, 4) || misaligned(it.master, 4))
      return SSIM_ERR_SHAPE;
    if (it.n > kMaxBytes / 4 || (total += it.n) > kMaxBytes) return SSIM_ERR_OVERFLOW;
    grad_bytes += it.n * gb;
    bytes += it.n * (gb + pb + 16 + (it.master ? 8 : pb));
    if (!runs.empty()) {
      AdamRun& r = runs.back();
      if (r.grad_dtype == it.grad_dtype && r.param_dtype == it.param_dtype &&
          follows(r.grad, r.n, gb, it.grad) && follows(r.param, r.n, pb, it.param) &&
          follows(r.m, r.n, 4, it.exp_avg) && follows(r.v, r.n, 4, it.exp_avg_sq) &&
          (r.master ? follows(r.master, r.n, 4, it.master) : !it.master)) {
        r.n += it.n;
        continue;
      }
    }
    runs.push_back({it.grad, it.param, it.exp_avg, it.exp_avg_sq, it.master, it.n, 0,
                    (int16_t)it.grad_dtype, (int16_t)it.param_dtype});
  }
  std::vector<Span> spans;
  spans.reserve(5 * runs.size() + 4);
  for (const AdamRun& r : runs) add_span(spans, r.grad, (size_t)r.n * elem_bytes(r.grad_dtype), false);
  for (const AdamRun& r : runs) add_span(spans, r.param, (size_t)r.n * elem_bytes(r.param_dtype), true);
  for (const AdamRun& r : runs) add_span(spans, r.m, (size_t)r.n * 4, true);
  for (const AdamRun& r : runs) add_span(spans, r.v, (size_t)r.n * 4, true);
  for (const AdamRun& r : runs) add_span(spans, r.master, (size_t)r.n * 4, true);
  add_span(spans, step, 16, true);
  add_span(spans, norm, 4, true);
  add_span(spans, o->lr_device, 4, false);
  add_span(spans, workspace, sizeof(Scratch), true);
  if (spans_clash(spans)) return SSIM_ERR_ALIAS;

  int rc = check_current_device();
  if (rc != SSIM_OK) return rc;

  const StepArgs st = {step, o->lr_device, o->lr, o->beta1, o->beta2, o->weight_decay};
  SmallAdamArgs small;
  // (a type of both, and whether there are masters)
  auto type_of = [](const AdamRun& r) {
    return r.grad_dtype | r.param_dtype << 4 | (r.master ? 256 : 0);
  };
  if (fits_small(runs, type_of, kAdamV, &small.table)) {
    small.max_norm = o->max_norm;
    small.norm = norm;
    small.step = st;
    small.beta1 = (float)o->beta1;
    small.one_minus_beta1 = (float)(1.0 - o->beta1);
    small.beta2 = (float)o->beta2;
    small.one_minus_beta2 = (float)(1.0 - o->beta2);
    small.eps = (float)o->eps;
    return launch_kernel(adamw_small_kernel(runs[0]),
                         (int)((small.table.first[kSmallRuns] + kSmallShare - 1) / kSmallShare),
                         &small, stream, kSmallThreads);
  }

  Scratch* scratch = static_cast<Scratch*>(workspace);
  const bool streams = bytes > kAdamStreamBytes;
  const int U = streams ? kAdamStreamU : 1;
  std::vector<Launch<AdamRun>> launches;
  if (!plan(runs, kAdamRuns, [&](const AdamRun&) { return (int64_t)kThreads * kAdamV * U; }, launches))
    return SSIM_ERR_OVERFLOW;
  std::vector<NormRun> norm_runs;
  if (norm) {
    norm_runs.reserve(runs.size());
    for (const AdamRun& r : runs) norm_runs.push_back({r.grad, r.n, 0, r.grad_dtype});
  }
  int partials = 0;  // (without a norm the first launch forms the scalars only)
  rc = launch_norm(norm_runs, 2 * grad_bytes, scratch, st, &partials, stream);
  if (rc != SSIM_OK) return rc;
  if (launches.empty()) return norm ? launch_norm_only(scratch, partials, norm, stream) : SSIM_OK;
  auto launch = [&](auto& a, const void* const (&kernels)[2], size_t k) {
    const auto& l = launches[k];
    a.count = (int)(l.end - l.begin);
    memcpy(a.run, &runs[l.begin], a.count * sizeof(AdamRun));
    a.chunks = l.chunks;
    a.partials = norm ? partials : 0;
    a.max_norm = o->max_norm;
    a.norm = k == 0 ? norm : nullptr;
    a.scratch = scratch;
    a.beta1 = (float)o->beta1;
    a.one_minus_beta1 = (float)(1.0 - o->beta1);
    a.beta2 = (float)o->beta2;
    a.one_minus_beta2 = (float)(1.0 - o->beta2);
    a.eps = (float)o->eps;
    return launch_kernel(kernels[streams], grid_for(l.chunks), &a, stream);
  };
  if (runs.size() <= kFewRuns && launches.size() == 1) {
    AdamArgs<kFewRuns> a;
    return launch(a, kAdamFew, 0);
  }
  for (size_t k = launches.size(); k-- > 0;) {
    AdamArgs<kAdamRuns> a;
    rc = launch(a, kAdamMany, k);
    if (rc != SSIM_OK) return rc;
  }
  return SSIM_OK;
}

}  // namespace

extern "C" {

size_t ssim_update_workspace_bytes(void) { return sizeof(Scratch); }

int ssim_clip_grads(const ssim_clip_item* items, int64_t count, double max_norm, float* norm,
                    void* workspace, void* stream) try {
  return clip_impl(items, count, true, max_norm, norm, workspace, stream);
} catch (...) {
  return SSIM_ERR_OVERFLOW;  // host memory for the table
}

int ssim_grad_norm(const ssim_clip_item* items, int64_t count, float* norm, void* workspace,
                   void* stream) try {
  return clip_impl(items, count, false, 0.0, norm, workspace, stream);
} catch (...) {
  return SSIM_ERR_OVERFLOW;
}

int ssim_adamw_step(const ssim_adamw_item* items, int64_t count, const ssim_adamw_options* options,
                    int64_t* step, float* norm, void* workspace, void* stream) try {
  return adamw_impl(items, count, options, step, norm, workspace, stream);
} catch (...) {
  return SSIM_ERR_OVERFLOW;
}

}  // extern "C"
