// train_common.hpp -- what the training operators' kernels and their host
// side share: element types, wide loads and stores, reductions, and the
// checks of pointers and device.

#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include "ssim_train_amd.h"

namespace ssim_train {

constexpr int kWave = 64;

// ---- element types
using F32 = float;
using F16 = _Float16;
using BF16 = __bf16;

// N elements of T as one value.  Tensors start at any element (packed buckets,
// rows of odd width), so the vectors promise the alignment of an element only;
// global loads and stores of gfx950 take such addresses at full width.
template <class T, int N>
struct Pack {
  typedef T Vec __attribute__((ext_vector_type(N)));
  typedef T Loose __attribute__((ext_vector_type(N), aligned(sizeof(T))));
  typedef float Wide __attribute__((ext_vector_type(N)));
};
template <class T, int N>
using Vec = typename Pack<T, N>::Vec;
template <int N>
using Wide = typename Pack<float, N>::Wide;

template <class T, int N>
__device__ __forceinline__ Vec<T, N> load(const T* p) {
  return *reinterpret_cast<const typename Pack<T, N>::Loose*>(p);
}
template <class T, int N>
__device__ __forceinline__ void store(T* p, Vec<T, N> v) {
  *reinterpret_cast<typename Pack<T, N>::Loose*>(p) = v;
}
template <class T, int N>
__device__ __forceinline__ Vec<T, N> load_once(const T* p) {  // not read again soon
  return __builtin_nontemporal_load(reinterpret_cast<const typename Pack<T, N>::Loose*>(p));
}
template <class T, int N>
__device__ __forceinline__ void store_once(T* p, Vec<T, N> v) {
  __builtin_nontemporal_store(v, reinterpret_cast<typename Pack<T, N>::Loose*>(p));
}
template <bool kOnce, class T, int N>
__device__ __forceinline__ Vec<T, N> load_as(const T* p) {
  if constexpr (kOnce) return load_once<T, N>(p);
  else return load<T, N>(p);
}
template <bool kOnce, class T, int N>
__device__ __forceinline__ void store_as(T* p, Vec<T, N> v) {
  if constexpr (kOnce) store_once<T, N>(p, v);
  else store<T, N>(p, v);
}
template <class T, int N>
__device__ __forceinline__ Wide<N> widen(Vec<T, N> v) {
  return __builtin_convertvector(v, typename Pack<T, N>::Wide);
}
template <class T, int N>
__device__ __forceinline__ Vec<T, N> narrow(Wide<N> v) {  // to nearest even
  return __builtin_convertvector(v, typename Pack<T, N>::Vec);
}

// ---- reductions: every lane gets the sum, in an order that does not change
// A value from the lane that kControl names, 0 where kRows leaves a row of 16
// lanes out (data-parallel primitives: within the vector unit, where a
// shuffle goes through the LDS at several times the latency).
template <int kControl, int kRows>
__device__ __forceinline__ float lane_move(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kControl, kRows, 0xf, false));
}
template <int kControl, int kRows>
__device__ __forceinline__ double lane_move(double v) {
  struct Words {
    int lo, hi;
  } w = __builtin_bit_cast(Words, v);
  w.lo = __builtin_amdgcn_update_dpp(0, w.lo, kControl, kRows, 0xf, false);
  w.hi = __builtin_amdgcn_update_dpp(0, w.hi, kControl, kRows, 0xf, false);
  return __builtin_bit_cast(double, w);
}
__device__ __forceinline__ float last_lane(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), kWave - 1));
}
__device__ __forceinline__ double last_lane(double v) {
  struct Words {
    int lo, hi;
  } w = __builtin_bit_cast(Words, v);
  w.lo = __builtin_amdgcn_readlane(w.lo, kWave - 1);
  w.hi = __builtin_amdgcn_readlane(w.hi, kWave - 1);
  return __builtin_bit_cast(double, w);
}
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
  v += lane_move<0xB1, 0xf>(v);   // the neighbour, of each two lanes
  v += lane_move<0x4E, 0xf>(v);   // the other two, of four
  v += lane_move<0x141, 0xf>(v);  // the mirror image, of eight
  v += lane_move<0x140, 0xf>(v);  // of sixteen
  v += lane_move<0x142, 0xa>(v);  // rows 1 and 3: the last lane of the row before
  v += lane_move<0x143, 0xc>(v);  // rows 2 and 3: lane 31
  return last_lane(v);
}

// The sum of each kLanes lanes beside each other, of 8, 16, 32 or the wave's 64.
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (kLanes == kWave) return wave_sum(v);
  v += lane_move<0xB1, 0xf>(v);
  v += lane_move<0x4E, 0xf>(v);
  v += lane_move<0x141, 0xf>(v);
  if constexpr (kLanes >= 16) v += lane_move<0x140, 0xf>(v);
  if constexpr (kLanes == 32)  // the lane 16 away
    v += __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, v), 0x401F));
  return v;
}

// ---- host side
inline int elem_bytes(int dtype) { return dtype == SSIM_DTYPE_F32 ? 4 : 2; }
inline bool known_dtype(int dtype) {
  return dtype == SSIM_DTYPE_F32 || dtype == SSIM_DTYPE_F16 || dtype == SSIM_DTYPE_BF16;
}
inline bool misaligned(const void* p, int bytes) { return ((uintptr_t)p % (uintptr_t)bytes) != 0; }
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t pa = (uintptr_t)a, pb = (uintptr_t)b;
  return pa < pb + nb && pb < pa + na;
}
// SSIM_OK if the current device is a gfx950
int check_current_device();

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kCUs = 256;  // of an MI355X; workspaces' sizes must not need a device query

struct Array {
  const void* p;
  size_t bytes;
  int align;
};
// alignment of all, and no output over an input or another output
inline int check_arrays(const Array* ins, int n_in, const Array* outs, int n_out) {
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

// Elements from the first of a tensor [batch][tokens][heads][dim] to its last; 0: there
// are none, -1: 2^58 or more.
inline int64_t span(const int64_t* stride, int64_t batch, int64_t tokens, int64_t heads, int64_t dim) {
  constexpr int64_t kMost = (int64_t)1 << 56;
  const int64_t sizes[3] = {batch, tokens, heads};
  int64_t sum = dim;
  for (int k = 0; k < 3; ++k) {
    if (sizes[k] < 1) return 0;
    if (sizes[k] > 1 && stride[k] > kMost / (sizes[k] - 1)) return -1;
    sum += (sizes[k] - 1) * stride[k];
  }
  return sum;
}

template <class Params>
int launch(const void* kernel, dim3 grid, int threads, Params& params, void* stream) {
  void* args[] = {&params};
  if (hipLaunchKernel(kernel, grid, dim3(threads), args, 0, static_cast<hipStream_t>(stream)) !=
      hipSuccess) {
    (void)hipGetLastError();
    return SSIM_ERR_HIP;
  }
  return SSIM_OK;
}

}  // namespace ssim_train
