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

}  // namespace ssim_train
