// mma.hpp -- what the kernels built on matrix products share: 32 x 32 tiles of
// fp32 sums, operands from LDS, and loads from memory straight to LDS.
//
// Operands are moved in chunks of 16 bytes (8 elements of a half type, 4 of
// fp32).  An instruction's lane holds row (lane % 32) of its operand and, of the
// axis that is summed over, a chunk of its own half (h = lane / 32): a step sums
// over two chunks, the first half's and the second's.  Which element of the
// axis stands where in the two chunks is free as long as both operands agree:
//   - rows that are contiguous along the axis are read as they lie;
//   - an operand that comes out of another product has, in the 16 registers of
//     a lane, rows 8 (r / 4) + 4 h + r % 4; so a step takes these rows of the
//     other operand, which for half types LDS gives transposed.

#pragma once

#include "train_common.hpp"

namespace ssim_train {

typedef unsigned Chunk __attribute__((ext_vector_type(4)));
typedef float Sums __attribute__((ext_vector_type(16)));  // of a 32 x 32 tile, a lane's
typedef short Quad __attribute__((ext_vector_type(4)));

template <class T>
constexpr int kPerChunk = 16 / (int)sizeof(T);
template <class T>
constexpr int kPerStep = 2 * kPerChunk<T>;

// fp16 ends at 65504 and loses bits below 2^-14, so what is rounded to it between two
// products is taken times a power of two, which the second's sums are divided by.
template <class T>
constexpr bool kScaled = __is_same(T, F16);

// c += a b over one step
template <class T>
__device__ __forceinline__ void multiply(Sums& c, Chunk a, Chunk b) {
  if constexpr (sizeof(T) == 4) {
    const Vec<float, 4> x = __builtin_bit_cast(Vec<float, 4>, a), y = __builtin_bit_cast(Vec<float, 4>, b);
#pragma unroll
    for (int k = 0; k < 4; ++k) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[k], y[k], c, 0, 0, 0);
  } else if constexpr (__is_same(T, F16)) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(Vec<F16, 8>, a),
                                               __builtin_bit_cast(Vec<F16, 8>, b), c, 0, 0, 0);
  } else {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(Vec<BF16, 8>, a),
                                                __builtin_bit_cast(Vec<BF16, 8>, b), c, 0, 0, 0);
  }
}

// Registers 8 s .. of a tile as the other product's operand: its step s for half
// types, the chunks 2 s and 2 s + 1 (steps of their own) for fp32.  For half types
// the sums are rounded to the type, to nearest even: fp32's instructions take 16 times
// as long.  It is one rounding of the terms beside the result's own (bf16, gradients of
// attention: 2.4e-3 of the norm, with all between in fp32 1.7e-3).
template <class T>
__device__ __forceinline__ Chunk operand_of(const Sums& c, int first) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(Chunk, Vec<float, 4>{c[first], c[first + 1], c[first + 2], c[first + 3]});
  } else {
    Wide<8> w;
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = c[first + k];
    return __builtin_bit_cast(Chunk, narrow<T, 8>(w));
  }
}

// ---- tiles in LDS: rows of kRow bytes (192 or a power of two, 64 or more), whose
// chunks are permuted within 256 bytes by the row's number: neither 16 rows'
// chunks of one column (read as they lie) nor 64 bytes of each of 4 rows (read
// transposed) meet in a bank.  (Rows of 192 and 64 bytes begin 64 apart by themselves.)
template <int kRow>
__device__ __forceinline__ int swizzle(int row) {
  if constexpr (kRow == 128) return ((row >> 1 & 1) << 2) | (row >> 2 & 3);
  else if constexpr (kRow == 192 || kRow == 64) return row >> 2 & 3;
  else return ((row & 3) << 2) | (row >> 2 & 3);
}
// an offset `bytes` along a row from `offset`, in the first chunks of its row; only where rows begin at multiples of
// 256 bytes are the higher bits permuted, too
template <int kRow>
__device__ __forceinline__ int along_row(int offset, int bytes) {
  if constexpr (kRow == 192 || kRow == 64) return (offset ^ (bytes & 63)) + (bytes & ~63);
  else return offset ^ bytes;
}
template <int kRow>
__device__ __forceinline__ int place(int row, int chunk) {  // byte offset of a chunk
  return row * kRow + ((chunk ^ swizzle<kRow>(row)) << 4);
}

typedef __attribute__((address_space(3))) char Lds;

__device__ __forceinline__ Chunk lds_chunk(const Lds* p, int at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) Chunk*>(p + at);
}

// Where a lane reads: its offsets in a tile (at a multiple of 256 or kRow), of which the
// other reads' are an exclusive or and a constant away.  Left to itself the compiler
// keeps each of them in a register through a loop; fresh() makes it form them
// anew, one instruction each.
__device__ __forceinline__ int fresh(int offset) {
  asm("" : "+v"(offset));
  return offset;
}
// rows as they lie: row lane % 32, chunk 2 t + h
template <int kRow>
__device__ __forceinline__ int along_offset() {
  const int lane = threadIdx.x & (kWave - 1);
  return place<kRow>(lane & 31, lane >> 5);
}
template <int kRow>
__device__ __forceinline__ Chunk lds_along(const Lds* tile, int offset, int row, int t) {
  return lds_chunk(tile, along_row<kRow>(offset, t << 5) + row * kRow);
}

// The operand whose rows are columns of the tile: lane's column 32 block +
// lane % 32, and a step's rows from `row` on (half types: 16; fp32: 8; `row` a
// multiple of them), in the order in which operand_of's step holds them or, kPlain,
// in that of a row read as it lies.
template <class T, int kRow, bool kPlain = false>
__device__ __forceinline__ int across_offset() {
  const int lane = threadIdx.x & (kWave - 1), h = lane >> 5;
  if constexpr (sizeof(T) == 4) return place<kRow>(4 * h, (lane & 31) >> 2) + ((lane & 3) << 2);
  // each 16 lanes read 4 rows of 16 columns and get a column's 4 values each
  const int i = lane & 15;
  return place<kRow>((kPlain ? 8 : 4) * h + (i >> 2), (lane >> 4 & 1) * 2 + (i >> 1 & 1)) + ((i & 1) << 3);
}
template <class T, int kRow, bool kPlain = false>
__device__ __forceinline__ Chunk lds_across(const Lds* tile, int offset, int row, int block) {
  if constexpr (sizeof(T) == 4) {
    Vec<float, 4> v;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int turned = (kRow == 128 ? k >> 1 : k) << 6;
      const int at = (offset ^ (block << 7) ^ turned ^ ((row >> 3 & 1) << 5)) + (row + k) * kRow;
      v[k] = *reinterpret_cast<const __attribute__((address_space(3))) float*>(tile + at);
    }
    return __builtin_bit_cast(Chunk, v);
  } else {
    typedef __attribute__((address_space(3))) Quad* At;
    constexpr int kTurned = kPlain ? 1 << 4 : 1 << 5, kNext = kPlain ? 4 : 8;
    const int at = along_row<kRow>(offset, block << 6);
    union {
      Quad q[2];
      Chunk c;
    } u;
    u.q[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((At)(tile + at + row * kRow));
    u.q[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((At)(tile + along_row<kRow>(offset ^ kTurned, block << 6) + (row + kNext) * kRow));
    return u.c;
  }
}

// matrix instructions of a product of two operands
template <class T>
constexpr int kInstructions = sizeof(T) == 4 ? 4 : 1;

// ---- order of instructions.  Left alone the compiler reads an operand from LDS just
// before the instruction that needs it and waits.  These lines, behind a sequence of
// products in the same basic block, ask for kAhead products' reads before the first
// and for each product's reads kAhead products early.
// Two stretches, of N products (kEach instructions and R reads) each; N1 may be 0.
template <int kAhead, int kEach, int N0, int R0, int N1 = 0, int R1 = 0>
__device__ __forceinline__ void read_ahead() {
  constexpr int kLdsRead = 0x100, kMatrix = 0x8;
#pragma unroll
  for (int i = -kAhead; i < N0 + N1; ++i) {
    if (i >= 0) __builtin_amdgcn_sched_group_barrier(kMatrix, kEach, 0);
    if (i + kAhead < N0) {
      if constexpr (R0 > 0) __builtin_amdgcn_sched_group_barrier(kLdsRead, R0, 0);
    } else if (i + kAhead < N0 + N1) {
      if constexpr (R1 > 0) __builtin_amdgcn_sched_group_barrier(kLdsRead, R1, 0);
    }
  }
}

// ... and here, for R reads spread between N instructions that do not need them.
template <int R, int N>
__device__ __forceinline__ void read_between() {
  constexpr int kLdsRead = 0x100, kMatrix = 0x8, kEach = (R + N - 1) / N;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(kMatrix, 1, 0);
    if (i * kEach < R) __builtin_amdgcn_sched_group_barrier(kLdsRead, kEach, 0);
  }
}

// ---- memory to LDS, without registers between: 64 lanes' chunks go to 1024
// bytes at `to` (the same for the wave), lane after lane.  A chunk past the
// descriptor's bytes arrives as zeros.  In asm, since the compiler waits for its own
// form of these loads before any read of the LDS; it does not count them:
// landed_for_all() waits.  (m0 is written here; nothing else in these kernels uses it.
// The wait between is for a descriptor that the vector unit has just written.)
typedef unsigned Descriptor __attribute__((ext_vector_type(4)));

// of `bytes` (< 2^32, counted in whole chunks) from p on, which is the same for the wave
__device__ __forceinline__ Descriptor describe(const void* p, uint32_t bytes) {
  const uint64_t at = (uint64_t)p;
  Descriptor d;
  d[0] = __builtin_amdgcn_readfirstlane((uint32_t)at);
  d[1] = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32) & 0xffffu);
  d[2] = __builtin_amdgcn_readfirstlane(bytes);
  d[3] = 0x00020000;
  return d;
}
constexpr uint32_t kNowhere = 0xfffffff0u;  // an offset past any descriptor's bytes

__device__ __forceinline__ void load_to_lds(Descriptor from, uint32_t offset, uint32_t to) {
  asm volatile(
      "s_mov_b32 m0, %0\n"
      "s_nop 4\n"
      "buffer_load_dwordx4 %1, %2, 0 offen lds"
      :
      : "s"(to), "v"(offset), "s"(from)
      : "memory");
}
// ... and 64 lanes' words to 256 bytes
__device__ __forceinline__ void load_words_to_lds(Descriptor from, uint32_t offset, uint32_t to) {
  asm volatile(
      "s_mov_b32 m0, %0\n"
      "s_nop 4\n"
      "buffer_load_dword %1, %2, 0 offen lds"
      :
      : "s"(to), "v"(offset), "s"(from)
      : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const Lds* p) { return (uint32_t)(uintptr_t)p; }

// All waves' LDS reads are done, and of their loads to LDS all but the last kLater
// have landed.
template <int kLater = 0>
__device__ __forceinline__ void landed_for_all() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kLater) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A lane's v and that of the lane 32 away, in this order on the lower lanes and
// the other way on the upper ones: for sums and maxima over both.  (In asm: two
// registers that hold the same value are the instruction's two operands.)
struct Halves {
  float a, b;
};
__device__ __forceinline__ Halves both_halves(float v) {
  Halves t = {v, v};
  asm volatile(
      "s_nop 1\n"
      "v_permlane32_swap_b32 %0, %1\n"
      "s_nop 1"
      : "+v"(t.a), "+v"(t.b));
  return t;
}
__device__ __forceinline__ float halves_sum(float v) {
  const Halves t = both_halves(v);
  return t.a + t.b;
}
__device__ __forceinline__ float halves_max(float v) {
  const Halves t = both_halves(v);
  return fmaxf(t.a, t.b);
}

}  // namespace ssim_train
