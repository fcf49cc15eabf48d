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
template <class T, int N>
__device__ __forceinline__ Wide<N> widen(Vec<T, N> v) {
  return __builtin_convertvector(v, typename Pack<T, N>::Wide);
}
template <class T, int N>
__device__ __forceinline__ Vec<T, N> narrow(Wide<N> v) {  // to nearest even
  return __builtin_convertvector(v, typename Pack<T, N>::Vec);
}

// ---- reductions: every lane gets the sum, in an order that does not change
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int m = kWave / 2; m > 0; m >>= 1) v += __shfl_xor(v, m, kWave);
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
// SSIM_OK if the current device is a gfx950; *cus: its compute units
int current_device(int* cus);

}  // namespace ssim_train
