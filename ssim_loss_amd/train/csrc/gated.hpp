// gated.hpp -- kernels of the gated layer:
//   g = x Wg^T + bg,  u = x Wu^T + bu,  h = act(g) u
//   dg = dh u act'(g),  du = dh act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  db = sums over rows
//
// Three products of one kernel's kind.  A workgroup forms a tile of the result,
// of which a lane has four neighbouring elements of a row at a time: the weights
// are the left operand.  Both operands go from memory straight to LDS, two tiles
// (of the smallest size three) in turn, 128 bytes of the axis that is summed over in
// each.  The forward's left tile is half Wg's and half Wu's rows, so a wave has g and u
// of the same elements in its registers and neither has to be written for the product.
// The bound is the matrix instructions and the clock under them (1.75 to 1.8 GHz): 16384 x 4096 x 10944 bf16, dx
// 1.27 PFLOP/s, dW 1.13, forward 1.11 with g and u written (a library product 1.32).

#pragma once

#include "mma.hpp"

namespace ssim_train {

struct GatedParams {
  const void* x;        // [rows][x_pitch]
  const void* w[2];     // gate, up: [hidden][w_pitch]
  const void* bias[2];  // [hidden] or NULL
  int64_t rows;
  int64_t x_pitch, w_pitch, h_pitch;  // elements; of g, u, dg and du: h_pitch
  int width, hidden, act;
  int width_ext;        // width, or x_pitch where x and w are copies padded with zeros
  void* out;            // [rows][hidden]
  float* saved[2];      // g, u: [rows][h_pitch], or NULL
  // backward
  const void* d_out;    // [rows][hidden]
  void* d[2];           // dg, du: [rows][h_pitch], zeros behind hidden
  float* part_bias;     // [blocks of rows][2][hidden] or NULL
  float* tops;          // fp16: of each workgroup of gated_tops, the largest finite |dg| and |du|; NULL: not wanted
  int* range;           // ... and the power of two that dg and du are kept times.  NULL: 0
  int top_count;
  int row_blocks;
  int rows_of_block;
  void* dx;             // [rows][width]
  void* dw[2];          // [hidden][width]
  void* db[2];
  // Of the products (Product; two gradients may be one launch's, that of x first):
  // tiles; parts of the summed axis, and where their sums go, [splits][rows of the
  // result][width]
  int m_tiles[3], n_tiles[3], splits[3];
  float* part[3];
  int x_blocks;
  // copies of x and the weights
  const void* from[3];
  void* to[3];
};

// act(g), and act'(g)
template <class T>
__device__ __forceinline__ float exp_of(float v) {
  if constexpr (sizeof(T) == 4) return expf(v);
  else return __expf(v);
}
template <class T>
__device__ __forceinline__ float quotient_of(float a, float b) {
  if constexpr (sizeof(T) == 4) return a / b;
  else return a * __builtin_amdgcn_rcpf(b);
}
// The normal distribution's share below g.  For half types exp(x^2) erfc(x) = t P(t),
// t = 1 / (1 + 0.44 x), with P fitted to 1.9e-7 of the value over x = 0 .. 10 (5e-7
// evaluated in fp32), a third of the library function's instructions (4100 x 1153
// x 2997 fp16: 108, so 98 us).
template <class T>
__device__ __forceinline__ float normal_share(float g) {
  if constexpr (sizeof(T) == 4) return 0.5f * erfcf(g * -0.70710678118654752f);
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(g), 0.44f * 0.70710678118654752f, 1.0f));
  float v = 0.07122284919023514f;
  v = fmaf(v, t, -0.2779455780982971f);
  v = fmaf(v, t, 0.29668352007865906f);
  v = fmaf(v, t, -0.02017728053033352f);
  v = fmaf(v, t, 0.21581058204174042f);
  v = fmaf(v, t, 0.2173140048980713f);
  v = fmaf(v, t, 0.2488711178302765f);
  v = fmaf(v, t, 0.24822095036506653f);
  const float half = 0.5f * t * v * __expf(-0.5f * g * g);
  return g > 0.0f ? 1.0f - half : half;
}
template <class T>
__device__ __forceinline__ float act_of(float g, int act) {
  if (act == SSIM_ACT_GELU) return g * normal_share<T>(g);
  return quotient_of<T>(act == SSIM_ACT_SILU ? g : 1.0f, 1.0f + exp_of<T>(-g));
}
template <class T>
__device__ __forceinline__ void act_slope(float g, int act, float& a, float& slope) {
  if (act == SSIM_ACT_GELU) {
    const float phi = normal_share<T>(g);
    a = g * phi;
    slope = fmaf(g * 0.39894228040143268f, exp_of<T>(-0.5f * g * g), phi);
    return;
  }
  // sigma(g) and sigma(-g), each without cancellation
  const float e = exp_of<T>(-fabsf(g));
  const float big = quotient_of<T>(1.0f, 1.0f + e), small = e * big;
  const float s = g >= 0.0f ? big : g < 0.0f ? small : g, r = g >= 0.0f ? small : big;
  if (act == SSIM_ACT_SILU) {
    a = g * s;
    slope = s * fmaf(g, r, 1.0f);
  } else {
    a = s;
    slope = s * r;
  }
}

enum Product { kForward, kGradX, kGradW };

constexpr int kDepthBytes = 128;  // of the summed axis, by which the host counts

// A product's tiles: BM x BN blocks of 32 x 32 to a wave, WM x WN waves, kDepthOf
// bytes of the summed axis at a time, kStages of them in LDS.
template <class T, int BM, int BN, int WM, int WN, int kDepthOf, int kStages_>
struct ProductShape {
  static constexpr int kThreads = WM * WN * kWave;
  static constexpr int kM = BM * WM * 32, kN = BN * WN * 32;
  static constexpr int kRow = kDepthOf;
  static constexpr int kDepth = kDepthOf / (int)sizeof(T);
  static constexpr int kSteps = kDepth / kPerStep<T>;
  static constexpr int kStages = kStages_;
  static constexpr int kABytes = kM * kDepthOf, kBBytes = kN * kDepthOf, kBytes = kABytes + kBBytes;
  static constexpr int kLoads = kBytes / (kThreads * 16);  // a wave's, of a stage
};

// An operand's tile whose rows are contiguous along the summed axis: kRows rows of
// kRow bytes.  `from` is the first row's first byte of the tile; `chunks` are left of
// the axis.
template <int kRows, int kRow, int kThreads>
__device__ __forceinline__ void fetch_along(const char* from, int64_t pitch, int64_t rows, int chunks, uint32_t to) {
  constexpr int kChunks = kRow / 16, kAtOnce = kThreads / kChunks;
  static_assert(kRows % kAtOnce == 0, "whole instructions");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int count = chunks <= 0 ? 0 : (int)(rows < kRows ? rows : kRows);
  const Descriptor d =
      describe(from, count <= 0 ? 0u : (uint32_t)(count - 1) * (uint32_t)pitch + (uint32_t)min(chunks, kChunks) * 16u);
#pragma unroll
  for (int j = 0; j < kRows / kAtOnce; ++j) {
    const int r = threadIdx.x / kChunks + j * kAtOnce;
    const int chunk = (threadIdx.x % kChunks) ^ swizzle<kRow>(r);
    const uint32_t offset = chunk < chunks ? (uint32_t)r * (uint32_t)pitch + (uint32_t)chunk * 16u : kNowhere;
    load_to_lds(d, offset, to + (uint32_t)(j * kThreads * 16 + wave * 1024));
  }
}
// An operand's tile whose rows lie along the other axis: kDepth rows of kRow bytes;
// `chunks` are left of such a row, `rows` of the summed axis.
template <int kDepth, int kRow, int kThreads>
__device__ __forceinline__ void fetch_across(const char* from, int64_t pitch, int64_t rows, int64_t chunks, uint32_t to) {
  constexpr int kChunks = kRow / 16, kAtOnce = kThreads / kChunks;
  static_assert(kAtOnce >= 1 && kDepth % kAtOnce == 0, "whole instructions");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int count = (int)(rows < kDepth ? rows : kDepth), left = (int)(chunks < kChunks ? chunks : kChunks);
  const Descriptor d = describe(from, count <= 0 || left <= 0 ? 0u : (uint32_t)(count - 1) * (uint32_t)pitch + (uint32_t)left * 16u);
#pragma unroll
  for (int j = 0; j < kDepth / kAtOnce; ++j) {
    const int r = threadIdx.x / kChunks + j * kAtOnce;
    const int chunk = (threadIdx.x % kChunks) ^ swizzle<kRow>(r);
    const uint32_t offset = chunk < left ? (uint32_t)r * (uint32_t)pitch + (uint32_t)chunk * 16u : kNowhere;
    load_to_lds(d, offset, to + (uint32_t)(j * kThreads * 16 + wave * 1024));
  }
}

// The workgroup's tile.  Ids go round the XCDs; each XCD takes a run of tiles that
// go down four rows of tiles at a time, so that its cache holds their operands (eight: 2% longer).
struct TileAt {
  int m, n;
};
__device__ __forceinline__ TileAt tile_at(unsigned block, int m_tiles, int n_tiles) {
  constexpr unsigned kGroup = 4;
  const unsigned total = (unsigned)m_tiles * n_tiles, per = (total + 7) / 8, rest = total - (per - 1) * 8;
  const unsigned xcd = block & 7, j = block >> 3;
  // (the first `rest` XCDs have a tile more where 8 does not divide the tiles)
  const unsigned id = xcd < rest ? xcd * per + j : rest * per + (xcd - rest) * (per - 1) + j;
  const unsigned of_group = kGroup * m_tiles, group = id / of_group, in = id - group * of_group;
  const unsigned rows = min(kGroup, n_tiles - group * kGroup);
  return {(int)(in / rows), (int)(group * kGroup + in % rows)};
}

// A wave's block of a result, kRows x kColumns, to memory: through its own part of
// the LDS, so that neighbouring lanes have a row's neighbouring chunks.  Straight
// from the registers each store would touch 32 rows with 16 bytes of each
// (16384 x 4096 x 10944 bf16, with g and u in bf16: 3419 us, so 2680).
// In: value(i, j, k), the four columns 32 i + 8 k + 4 h of row 32 j + lane % 32.
template <class T, int MB, int NB, class Value>
__device__ __forceinline__ void store_block(Lds* region, T* out, int64_t pitch, int64_t row0, int64_t column0,
                                            int64_t rows, int64_t columns, Value value) {
  constexpr int kRow = MB * 32 * 4 < 128 ? 128 : MB * 32 * 4;  // bytes, of fp32
  static_assert(MB == 1 || MB == 2, "a power of two");
  const int lane = threadIdx.x & (kWave - 1), h = lane >> 5;
  typedef __attribute__((address_space(3))) Wide<4>* At;
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *(At)(region + place<kRow>(32 * j + (lane & 31), 8 * i + 2 * k + h)) = value(i, j, k);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // (a wave's own)
  constexpr int V = kPerChunk<T>;
  constexpr int kLanes = MB * 32 / V;  // to a row
  constexpr int kAtOnce = kWave / kLanes;
#pragma unroll
  for (int r = 0; r < NB * 32; r += kAtOnce) {
    const int row = r + lane / kLanes, column = lane % kLanes * V;
    Wide<V> v;
#pragma unroll
    for (int q = 0; q < V / 4; ++q) {
      const Wide<4> w = *(At)(region + place<kRow>(row, column / 4 + q));
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * q + e] = w[e];
    }
    if (row0 + row >= rows) continue;
    T* to = out + (row0 + row) * pitch + column0 + column;
    const Vec<T, V> n = narrow<T, V>(v);
    if (column0 + column + V <= columns) {
      store<T, V>(to, n);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (column0 + column + e < columns) to[e] = n[e];
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}
// Four neighbouring elements of a row, those of them that it has.
template <class T>
__device__ __forceinline__ void store_four(T* row, int64_t column, int64_t width, Wide<4> v) {
  const Vec<T, 4> n = narrow<T, 4>(v);
  if (column + 4 <= width) {
    store<T, 4>(row + column, n);
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (column + k < width) row[column + k] = n[k];
}

template <class T, int kProduct, int BM, int BN, int WM, int WN, int kDepthOf, int kStages>
__device__ __forceinline__ void product_tile(const GatedParams& p, unsigned block, char* lds_) {
  using Shape = ProductShape<T, BM, BN, WM, WN, kDepthOf, kStages>;
  Lds* lds = (Lds*)lds_;
  const uint32_t lds_at = lds_address(lds);
  const int splits = p.splits[kProduct], n_tiles = p.n_tiles[kProduct];
  const int split = kProduct == kForward ? 0 : block % splits;
  const TileAt at = tile_at(kProduct == kForward ? block : block / splits, p.m_tiles[kProduct], n_tiles);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x & (kWave - 1);
  const int wm = wave % WM, wn = wave / WM, h = lane >> 5;
  constexpr int kBytes = (int)sizeof(T);
  constexpr int kHalfM = Shape::kM / 2;  // of the forward: columns of the result in a tile

  // how many tiles of the summed axis there are
  const int64_t depth = kProduct == kForward ? p.width_ext : kProduct == kGradX ? p.h_pitch : p.rows;
  const int once = (int)((depth + Shape::kDepth - 1) / Shape::kDepth);
  const int whole = kProduct == kGradX ? 2 * once : once, each = (whole + splits - 1) / splits;
  const int begin = kProduct == kForward ? 0 : min(split * each, whole);
  const int end = kProduct == kForward ? whole : min(begin + each, whole);
  const int n_half = n_tiles / 2;  // gradients of weights: gate's tiles, then up's
  const int which = kProduct == kGradW ? (at.n >= n_half) : 0;
  if (kProduct == kGradW && !p.dw[which]) return;
  const int64_t m0 = (int64_t)at.m * (kProduct == kForward ? kHalfM : Shape::kM);
  const int64_t n0 = (int64_t)(kProduct == kGradW ? at.n - which * n_half : at.n) * Shape::kN;

  auto fetch = [&](int t) {
    // (none past the end: their loads are counted all the same)
    const uint32_t a_to = lds_at + ((t - begin) % kStages) * Shape::kBytes, b_to = a_to + Shape::kABytes;
    const bool there = t < end;
    if constexpr (kProduct == kForward) {
      const int64_t k = (int64_t)t * Shape::kDepth;
      const int chunks = there ? (int)((p.width_ext - k) / kPerChunk<T>) : 0;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        fetch_along<kHalfM, Shape::kRow, Shape::kThreads>((const char*)p.w[i] + (m0 * p.w_pitch + k) * kBytes, p.w_pitch * kBytes,
                                             p.hidden - m0, chunks, a_to + i * (kHalfM * Shape::kRow));
      fetch_along<Shape::kN, Shape::kRow, Shape::kThreads>((const char*)p.x + (n0 * p.x_pitch + k) * kBytes, p.x_pitch * kBytes,
                                              p.rows - n0, chunks, b_to);
    } else if constexpr (kProduct == kGradX) {
      const int i = t >= once;
      const int64_t k = (int64_t)(t - i * once) * Shape::kDepth;
      fetch_across<Shape::kDepth, Shape::kM * kBytes, Shape::kThreads>((const char*)p.w[i] + (k * p.w_pitch + m0) * kBytes, p.w_pitch * kBytes,
                                                  there ? p.hidden - k : 0, (p.width_ext - m0 + kPerChunk<T> - 1) / kPerChunk<T>, a_to);
      fetch_along<Shape::kN, Shape::kRow, Shape::kThreads>((const char*)p.d[i] + (n0 * p.h_pitch + k) * kBytes, p.h_pitch * kBytes,
                                              p.rows - n0, there ? (int)((p.h_pitch - k) / kPerChunk<T>) : 0, b_to);
    } else {
      const int64_t k = (int64_t)t * Shape::kDepth;
      fetch_across<Shape::kDepth, Shape::kM * kBytes, Shape::kThreads>((const char*)p.x + (k * p.x_pitch + m0) * kBytes, p.x_pitch * kBytes,
                                                  there ? p.rows - k : 0, (p.width_ext - m0 + kPerChunk<T> - 1) / kPerChunk<T>, a_to);
      fetch_across<Shape::kDepth, Shape::kN * kBytes, Shape::kThreads>((const char*)p.d[which] + (k * p.h_pitch + n0) * kBytes,
                                                  p.h_pitch * kBytes, there ? p.rows - k : 0, (p.h_pitch - n0) / kPerChunk<T>, b_to);
    }
  };

  Sums c[BM][BN] = {};
  // the blocks' first rows (or columns) in the tiles; the forward's are g's, then u's
  auto a_block = [&](int i) {
    if constexpr (kProduct == kForward) return i < BM / 2 ? wm * (BM / 2) + i : kHalfM / 32 + wm * (BM / 2) + i - BM / 2;
    else return wm * BM + i;
  };
  const int a_at = kProduct == kForward ? along_offset<Shape::kRow>() : across_offset<T, Shape::kM * kBytes, true>();
  const int b_at = kProduct == kGradW ? across_offset<T, Shape::kN * kBytes, true>() : along_offset<Shape::kRow>();
  // A step's operands are read while the one before is multiplied, the next tile's first
  // with this tile's last: its buffer is free once all waves have read that.
  // 16384 x 4096 x 10944 bf16, with each step's read before its own products 2815 us
  // forward, 2550 and 2715 the gradients, so 2580, 2290 and 2590.  (Four waves of twice
  // the block each read less, but nothing runs beside a wave that waits: 3080, 2430, 2830.
  // 64 bytes of depth in four buffers: 2830, 2550, 2740.)
  Chunk a[2][BM], b[2][BN];
  auto take = [&](int which_, int t, int s) {
    const Lds* a_tile = lds + ((t - begin) % kStages) * Shape::kBytes;
    const Lds* b_tile = a_tile + Shape::kABytes;
#pragma unroll
    for (int i = 0; i < BM; ++i) {
      if constexpr (kProduct == kForward)
        a[which_][i] = lds_along<Shape::kRow>(a_tile, a_at, 32 * a_block(i), s);
      else
        a[which_][i] = lds_across<T, Shape::kM * kBytes, true>(a_tile, a_at, s * kPerStep<T>, a_block(i));
    }
#pragma unroll
    for (int i = 0; i < BN; ++i) {
      if constexpr (kProduct == kGradW)
        b[which_][i] = lds_across<T, Shape::kN * kBytes, true>(b_tile, b_at, s * kPerStep<T>, wn * BN + i);
      else
        b[which_][i] = lds_along<Shape::kRow>(b_tile, b_at, 32 * (wn * BN + i), s);
    }
  };
  static_assert(Shape::kSteps % 2 == 0, "the next tile's first step goes where this one's did");
  if (begin < end) {
#pragma unroll
    for (int t = 0; t < kStages; ++t) fetch(begin + t);
    landed_for_all<(kStages - 1) * Shape::kLoads>();
    take(0, begin, 0);
  }
  for (int t = begin; t < end; ++t) {
#pragma unroll
    for (int s = 0; s < Shape::kSteps; ++s) {
      if (s + 1 < Shape::kSteps) {
        take((s + 1) % 2, t, s + 1);
      } else {
        landed_for_all<(kStages - 2) * Shape::kLoads>();
        fetch(t + kStages);
        take(0, t + 1, 0);
      }
#pragma unroll
      for (int i = 0; i < BM; ++i)
#pragma unroll
        for (int j = 0; j < BN; ++j) multiply<T>(c[i][j], a[s % 2][i], b[s % 2][j]);
      // (2680 without; across rows a read is two, and the gradients were slower with it)
      if constexpr (kProduct == kForward) read_between<BM + BN, BM * BN * kInstructions<T>>();
    }
  }

  landed_for_all();  // the tiles' place is the waves' own now
  Lds* region = lds + wave * (kStages * Shape::kBytes / (WM * WN));
  const int64_t row0 = n0 + 32 * wn * BN;
  if constexpr (kProduct == kForward) {
    constexpr int MB = BM / 2;
    const int64_t column0 = m0 + 32 * wm * MB;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t column = column0 + 32 * i + 8 * k + 4 * h + e;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const float bias = p.bias[w] && column < p.hidden ? (float)static_cast<const T*>(p.bias[w])[column] : 0.0f;
#pragma unroll
            for (int j = 0; j < BN; ++j) c[i + w * MB][j][4 * k + e] += bias;
          }
        }
    if (p.saved[0]) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
        store_block<float, MB, BN>(region, p.saved[w], p.h_pitch, row0, column0, p.rows, p.h_pitch, [&](int i, int j, int k) {
          const Sums& s = c[i + w * MB][j];
          return Wide<4>{s[4 * k], s[4 * k + 1], s[4 * k + 2], s[4 * k + 3]};
        });
    }
    store_block<T, MB, BN>(region, static_cast<T*>(p.out), p.hidden, row0, column0, p.rows, p.hidden, [&](int i, int j, int k) {
      Wide<4> v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act_of<T>(c[i][j][4 * k + e], p.act) * c[i + MB][j][4 * k + e];
      return v;
    });
  } else {
    const int64_t rows = kProduct == kGradX ? p.rows : p.hidden;
    constexpr int MB = BM < 2 ? 1 : 2;  // at once
    const float down = kScaled<T> && p.range ? ldexpf(1.0f, -*p.range) : 1.0f;
#pragma unroll
    for (int i0 = 0; i0 < BM; i0 += MB) {
      const int64_t column0 = m0 + 32 * (wm * BM + i0);
      auto value = [&](int i, int j, int k) {
        const Sums& s = c[i0 + i][j];
        const Wide<4> v = {s[4 * k], s[4 * k + 1], s[4 * k + 2], s[4 * k + 3]};
        return kScaled<T> ? v * down : v;
      };
      if (splits > 1) {
        float* to = p.part[kProduct] + ((int64_t)split * (kProduct == kGradW ? 2 : 1) + which) * rows * p.width;
        store_block<float, MB, BN>(region, to, p.width, row0, column0, rows, p.width, value);
      } else {
        T* to = static_cast<T*>(kProduct == kGradX ? p.dx : p.dw[which]);
        store_block<T, MB, BN>(region, to, p.width, row0, column0, rows, p.width, value);
      }
    }
  }
}

template <class T, int kProduct, int BM, int BN, int WM, int WN, int kDepthOf, int kStages>
__global__ void __launch_bounds__(WM* WN* kWave, WM* WN == 4 ? 2 : 1) gated_product(const GatedParams p) {
  __shared__ __attribute__((aligned(1024))) char lds[kStages * ProductShape<T, BM, BN, WM, WN, kDepthOf, kStages>::kBytes];
  product_tile<T, kProduct, BM, BN, WM, WN, kDepthOf, kStages>(p, blockIdx.x, lds);
}
// Both gradients' small tiles in one launch: neither fills the GPU for long.
template <class T>
__global__ void __launch_bounds__(256, 2) gated_both(const GatedParams p) {
  __shared__ __attribute__((aligned(1024))) char lds[3 * ProductShape<T, 1, 1, 2, 2, 128, 3>::kBytes];
  if ((int)blockIdx.x < p.x_blocks) product_tile<T, kGradX, 1, 1, 2, 2, 128, 3>(p, blockIdx.x, lds);
  else product_tile<T, kGradW, 1, 1, 2, 2, 128, 3>(p, blockIdx.x - p.x_blocks, lds);
}

// `splits` parts of n elements, `step` apart, together.
template <class T>
__device__ __forceinline__ void join_parts(const float* part, T* to, int64_t n, int64_t step, int splits) {
  for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; at < n; at += (int64_t)gridDim.x * 256 * 4) {
    const float* from = part + at;
    if (at + 4 <= n) {
      Wide<4> sum = load<float, 4>(from);
#pragma unroll 4
      for (int s = 1; s < splits; ++s) sum += load<float, 4>(from + s * step);
      store<T, 4>(to + at, narrow<T, 4>(sum));
    } else {
      for (int k = 0; at + k < n; ++k) {
        float sum = from[k];
        for (int s = 1; s < splits; ++s) sum += from[s * step + k];
        to[at + k] = (T)sum;
      }
    }
  }
}
// The blocks' sums of a bias together: 64 columns at a time, a quarter of the blocks
// to each wave.
template <class T>
__device__ __forceinline__ void bias_sums(const GatedParams& p, int i) {
  __shared__ double sums[4][kWave];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
  for (int64_t first = (int64_t)blockIdx.x * kWave; first < p.hidden; first += (int64_t)gridDim.x * kWave) {
    const int64_t column = first + lane;
    double sum = 0.0;
    if (column < p.hidden) {
#pragma unroll 8
      for (int b = wave; b < p.row_blocks; b += 4) sum += p.part_bias[((int64_t)b * 2 + i) * p.hidden + column];
    }
    sums[wave][lane] = sum;
    __syncthreads();
    if (wave == 0 && column < p.hidden)
      static_cast<T*>(p.db[i])[column] = (T)(float)(((sums[0][lane] + sums[1][lane]) + sums[2][lane]) + sums[3][lane]);
    __syncthreads();
  }
}
// What is left of the gradients, blockIdx.y: the parts of dx, dWg, dWu; the biases.
template <class T>
__global__ void __launch_bounds__(256) gated_finish(const GatedParams p) {
  const int64_t x = p.rows * p.width, w = (int64_t)p.hidden * p.width;
  const int what = blockIdx.y;
  if (what == 0) {
    if (p.dx && p.splits[kGradX] > 1) join_parts<T>(p.part[kGradX], static_cast<T*>(p.dx), x, x, p.splits[kGradX]);
  } else if (what <= 2) {
    const int i = what - 1;
    if (p.dw[i] && p.splits[kGradW] > 1)
      join_parts<T>(p.part[kGradW] + i * w, static_cast<T*>(p.dw[i]), w, 2 * w, p.splits[kGradW]);
  } else if (p.db[what - 3]) {
    bias_sums<T>(p, what - 3);
  }
}

// dg and du of a workgroup's rows and columns: take(place, dg, du).  A thread has a vector
// of columns; 64 of them beside each other, four rows at a time.
template <class T, class Take>
__device__ __forceinline__ void each_slope(const GatedParams& p, int64_t column, Take take) {
  constexpr int V = kPerChunk<T>;
  const int64_t first = (int64_t)blockIdx.y * p.rows_of_block;
  const int64_t end = first + p.rows_of_block < p.rows ? first + p.rows_of_block : p.rows;
  if (column >= p.h_pitch) return;
  for (int64_t row = first + threadIdx.x / kWave; row < end; row += 4) {
    const int64_t at = row * p.h_pitch + column;
    const Wide<V> g = load_once<float, V>(p.saved[0] + at), u = load_once<float, V>(p.saved[1] + at);
    const T* d_row = static_cast<const T*>(p.d_out) + row * p.hidden;
    Wide<V> d = {};
    if (column + V <= p.hidden) d = widen<T, V>(load<T, V>(d_row + column));
    else
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (column + k < p.hidden) d[k] = (float)d_row[column + k];
    Wide<V> dg, du;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float a, slope;
      act_slope<T>(g[k], p.act, a, slope);
      const bool in = column + k < p.hidden;
      dg[k] = in ? d[k] * u[k] * slope : 0.0f;
      du[k] = in ? d[k] * a : 0.0f;
    }
    take(at, dg, du);
  }
}

// The largest number of a workgroup's threads, none of them below 0, for all of them.
__device__ __forceinline__ float largest_of(float v) {
  __shared__ float most[4];
  for (int step = 1; step < kWave; step *= 2) v = fmaxf(v, __shfl_xor(v, step));
  if ((threadIdx.x & (kWave - 1)) == 0) most[threadIdx.x / kWave] = v;
  __syncthreads();
  return fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
}

// The largest |dg| and |du| of a workgroup's share, by which fp16's are brought into its range: left
// as they are, gradients scaled by 2^16 overflow, and of those of 10^-6 dw is 2% off.  What is not finite is
// left out.  A read of g, u and d_out more, the memory's bound: forward and gradients of 16384 x 4096 x 10944
// fp16 8340, so 8720 us, 4100 x 1153 x 2997 322, so 348.  (A bound by the norms of rows would need x and the
// weights alone, but may be far too large.)
template <class T>
__global__ void __launch_bounds__(256) gated_tops(const GatedParams p) {
  constexpr int V = kPerChunk<T>;
  const int64_t column = ((int64_t)blockIdx.x * kWave + (threadIdx.x & (kWave - 1))) * V;
  float top = 0.0f;
  each_slope<T>(p, column, [&](int64_t, Wide<V> dg, Wide<V> du) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float a = fabsf(dg[k]), b = fabsf(du[k]);
      if (a < INFINITY) top = fmaxf(top, a);
      if (b < INFINITY) top = fmaxf(top, b);
    }
  });
  top = largest_of(top);
  if (threadIdx.x == 0) p.tops[blockIdx.y * gridDim.x + blockIdx.x] = top;
}

// dg and du, rounded to the type as the products' operands (bf16: gradients 2.3e-3 of the
// norm, with fp32 operands, whose instructions take 16 times as long, 1.7e-3), and what they
// add up to over a block of rows, unrounded.
template <class T>
__global__ void __launch_bounds__(256) gated_slopes(const GatedParams p) {
  constexpr int V = kPerChunk<T>;
  __shared__ float sums[3][2][kWave * V];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
  const int64_t column = ((int64_t)blockIdx.x * kWave + lane) * V;
  float up = 1.0f;
  if constexpr (kScaled<T>) {
    if (p.tops) {
      float top = 0.0f;
      for (int k = threadIdx.x; k < p.top_count; k += 256) top = fmaxf(top, p.tops[k]);
      top = largest_of(top);
      // (top < 2^exponent: the largest is kept below 2^15)
      const int range = top > 0.0f ? min(15 - __builtin_amdgcn_frexp_expf(top), 100) : 0;
      up = ldexpf(1.0f, range);
      if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.range = range;
    }
  }
  Wide<V> total[2] = {};
  each_slope<T>(p, column, [&](int64_t at, Wide<V> dg, Wide<V> du) {
    total[0] += dg;
    total[1] += du;
    if constexpr (kScaled<T>) {
      dg *= up;
      du *= up;
    }
    store<T, V>(static_cast<T*>(p.d[0]) + at, narrow<T, V>(dg));
    store<T, V>(static_cast<T*>(p.d[1]) + at, narrow<T, V>(du));
  });
  if (!p.part_bias) return;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (wave > 0) sums[wave - 1][i][k * kWave + lane] = total[i][k];
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float s = ((total[i][k] + sums[0][i][k * kWave + lane]) + sums[1][i][k * kWave + lane]) + sums[2][i][k * kWave + lane];
      if (column + k < p.hidden) p.part_bias[((int64_t)blockIdx.y * 2 + i) * p.hidden + column + k] = s;
    }
}

// Rows of `width` elements to rows of width_ext, zeros behind them.
template <class T>
__global__ void __launch_bounds__(256) gated_copy(const GatedParams p) {
  constexpr int V = kPerChunk<T>;
  const int64_t chunks = p.width_ext / V, rows = blockIdx.y ? p.hidden : p.rows;
  for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < rows * chunks; id += (int64_t)gridDim.x * 256) {
    const int64_t row = id / chunks, column = (id - row * chunks) * V;
    const T* from = static_cast<const T*>(p.from[blockIdx.y]) + row * p.width;
    Vec<T, V> v = {};
    if (column + V <= p.width) v = load<T, V>(from + column);
    else
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (column + k < p.width) v[k] = from[column + k];
    store<T, V>(static_cast<T*>(p.to[blockIdx.y]) + row * p.width_ext + column, v);
  }
}

// ---- few rows: the weights go by once, from memory straight to the matrix
// instruction (16 rows of weights, 16 of x); four waves share the summed axis.  The bound
// is the memory: 1 x 4096 x 10944 bf16, 179 MB in 37.8 us, 4.8 TB/s.
typedef float Sums4 __attribute__((ext_vector_type(4)));
template <class T>
__device__ __forceinline__ void multiply16(Sums4& c, Chunk a, Chunk b) {
  if constexpr (sizeof(T) == 4) {
    const Vec<float, 4> x = __builtin_bit_cast(Vec<float, 4>, a), y = __builtin_bit_cast(Vec<float, 4>, b);
#pragma unroll
    for (int k = 0; k < 4; ++k) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[k], y[k], c, 0, 0, 0);
  } else if constexpr (__is_same(T, F16)) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(Vec<F16, 8>, a), __builtin_bit_cast(Vec<F16, 8>, b), c, 0, 0, 0);
  } else {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(Vec<BF16, 8>, a), __builtin_bit_cast(Vec<BF16, 8>, b), c, 0, 0, 0);
  }
}
// The chunk of a row at `column`; zeros behind its end, the last one with one load.
// (rows have a chunk's elements or more)
template <class T>
__device__ __forceinline__ Chunk chunk_of_row(const T* row, int column, int width) {
  constexpr int V = kPerChunk<T>;
  const int start = min(column, width - V);
  Chunk c = __builtin_bit_cast(Chunk, load<T, V>(row + start));
  if (column > start) {  // elements that belong to the chunk before go
    const int shift = min(column - start, V) * (int)sizeof(T) * 8;  // bits, to 128
    unsigned __int128 bits = __builtin_bit_cast(unsigned __int128, c);
    bits = shift >= 128 ? 0 : bits >> shift;
    c = __builtin_bit_cast(Chunk, bits);
  }
  return c;
}

constexpr int kFewUnroll = 4;

template <class T, int NB>
__global__ void __launch_bounds__(256) gated_few_rows(const GatedParams p) {
  __shared__ Sums4 joined[3][2][NB][kWave];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
  const int group = lane >> 4;
  const int m0 = blockIdx.x * 16;
  const int w_row = min(m0 + (lane & 15), p.hidden - 1);
  const T* gate = static_cast<const T*>(p.w[0]) + (int64_t)w_row * p.w_pitch;
  const T* up = static_cast<const T*>(p.w[1]) + (int64_t)w_row * p.w_pitch;
  const T* x[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
    x[j] = static_cast<const T*>(p.x) + min((int64_t)(16 * j + (lane & 15)), p.rows - 1) * p.x_pitch;
  constexpr int kStep = 4 * kPerChunk<T>;  // elements that an instruction (fp32: four) sums over
  constexpr int kAtOnce = kStep * kFewUnroll;
  Sums4 c[2][NB] = {};
  for (int k0 = wave * kAtOnce; k0 < p.width; k0 += 4 * kAtOnce) {
    Chunk a[2][kFewUnroll];
#pragma unroll
    for (int s = 0; s < kFewUnroll; ++s) {
      const int k = k0 + s * kStep + group * kPerChunk<T>;
      a[0][s] = chunk_of_row<T>(gate, k, p.width);
      a[1][s] = chunk_of_row<T>(up, k, p.width);
    }
#pragma unroll
    for (int s = 0; s < kFewUnroll; ++s) {
      const int k = k0 + s * kStep + group * kPerChunk<T>;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const Chunk b = chunk_of_row<T>(x[j], k, p.width);
        multiply16<T>(c[0][j], a[0][s], b);
        multiply16<T>(c[1][j], a[1][s], b);
      }
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) joined[wave - 1][i][j][lane] = c[i][j];
  }
  __syncthreads();
  if (wave > 0) return;
  const int column = m0 + 4 * group;
  if (column >= p.h_pitch) return;
#pragma unroll
  for (int j = 0; j < NB; ++j) {
#pragma unroll
    for (int i = 0; i < 2; ++i) c[i][j] = ((c[i][j] + joined[0][i][j][lane]) + joined[1][i][j][lane]) + joined[2][i][j][lane];
    const int64_t row = 16 * j + (lane & 15);
    if (row >= p.rows) continue;
    Wide<4> g, u, v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = column + e < p.hidden;
      g[e] = c[0][j][e] + (p.bias[0] && in ? (float)static_cast<const T*>(p.bias[0])[column + e] : 0.0f);
      u[e] = c[1][j][e] + (p.bias[1] && in ? (float)static_cast<const T*>(p.bias[1])[column + e] : 0.0f);
      v[e] = act_of<T>(g[e], p.act) * u[e];
    }
    store_four<T>(static_cast<T*>(p.out) + row * p.hidden, column, p.hidden, v);
    if (p.saved[0]) {
      store<float, 4>(p.saved[0] + row * p.h_pitch + column, g);
      store<float, 4>(p.saved[1] + row * p.h_pitch + column, u);
    }
  }
}

// ---- kernels of a type
struct GatedTable {
  const void* product[3][3];  // [Product][tiles of 64, 128, 256 rows]
  const void* few[3];         // 16, 32, 64 rows
  const void* tops;           // NULL: not needed
  const void* slopes;
  const void* both;
  const void* finish;
  const void* copy;
};
template <class T>
GatedTable make_gated_table() {
  GatedTable t;
  t.product[kForward][0] = (const void*)gated_product<T, kForward, 2, 1, 2, 2, 128, 3>;
  t.product[kForward][1] = (const void*)gated_product<T, kForward, 2, 2, 2, 2, 128, 2>;
  t.product[kForward][2] = (const void*)gated_product<T, kForward, 4, 2, 2, 4, 128, 2>;
  t.product[kGradX][0] = (const void*)gated_product<T, kGradX, 1, 1, 2, 2, 128, 3>;
  t.product[kGradX][1] = (const void*)gated_product<T, kGradX, 2, 2, 2, 2, 128, 2>;
  t.product[kGradX][2] = (const void*)gated_product<T, kGradX, 4, 2, 2, 4, 128, 2>;
  t.product[kGradW][0] = (const void*)gated_product<T, kGradW, 1, 1, 2, 2, 128, 3>;
  t.product[kGradW][1] = (const void*)gated_product<T, kGradW, 2, 2, 2, 2, 128, 2>;
  t.product[kGradW][2] = (const void*)gated_product<T, kGradW, 4, 2, 2, 4, 128, 2>;
  t.few[0] = (const void*)gated_few_rows<T, 1>;
  t.few[1] = (const void*)gated_few_rows<T, 2>;
  t.few[2] = (const void*)gated_few_rows<T, 4>;
  t.tops = nullptr;
  if constexpr (kScaled<T>) t.tops = (const void*)gated_tops<T>;
  t.slopes = (const void*)gated_slopes<T>;
  t.both = (const void*)gated_both<T>;
  t.finish = (const void*)gated_finish<T>;
  t.copy = (const void*)gated_copy<T>;
  return t;
}
const GatedTable& gated_table_f32();
const GatedTable& gated_table_f16();
const GatedTable& gated_table_bf16();

}  // namespace ssim_train
