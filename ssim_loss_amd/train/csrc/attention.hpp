// attention.hpp -- kernels of softmax attention and its gradients:
//   s_ij = q_i . k_j     p_ij = exp(scale s_ij - lse_i)     o_i = sum_j p_ij v_j
//   ds_ij = p_ij (do_i . v_j - do_i . o_i)
//   dq_i = scale sum_j ds_ij k_j     dk_j = scale sum_i ds_ij q_i     dv_j = sum_i p_ij do_i
// over the keys j that row i sees; a row that sees none gives zeros.
//
// Scores and probabilities never reach memory.  A wave holds 32 rows' queries (or,
// for the gradients of keys and values, 32 keys) in registers as one operand and
// streams the other side through LDS.  A product's result comes out with one of
// its rows to a lane, so the row's maximum and sum need but one exchange, and is
// the next product's operand as it stands (mma.hpp).

#pragma once

#include "mma.hpp"

namespace ssim_train {

constexpr int kAttentionThreads = 256;
constexpr int kRowsOfWave = 32;

struct Strided {
  const char* p;
  int64_t batch, head;  // bytes
  uint32_t token;
};

struct AttentionParams {
  Strided q, k, v;
  const int* q_length;  // NULL: q_tokens
  const int* k_length;
  int q_tokens, k_tokens, heads, kv_heads, group, dim, batch;
  int causal, spread;  // spread: (batch, key head) pairs are dealt out over the XCDs
  int tiles, splits;   // of rows (or keys); parts of the keys that workgroups of their own take
  float scale2;        // scale log2(e), not 0: of a masked score it is a factor
  float scale;         // scale 2^scale_power is the scale, of which fp32 would hold few bits below 2^-126
  int scale_power;
  void* out;           // [batch][q_tokens][heads][dim]
  void* rest;          // as out: what out's rounding left, rounded itself; NULL: not wanted, or fp32
  float* lse;          // [batch][heads][q_tokens], log2 of the row's sum; +inf: no keys.  NULL: not wanted
  float* part_out;     // [splits][batch][heads][q_tokens][dim], each part's own softmax
  float* part_lse;     // [splits][batch][heads][q_tokens]; -inf: no keys
  // backward
  const void* o;       // as out and rest
  const void* o_rest;
  const void* d_out;
  float* delta;        // [batch][heads][q_tokens]
  int kv_tiles, q_blocks;  // where one launch has both gradients: that of the queries first
  float* norms;        // fp16: [batch][kv_heads][kNormParts][2], largest |do_i| and |v_j|
  void* dq;
  void* dk;
  void* dv;
};

// Of a kernel for elements T and heads of at most 32 DB elements.
template <class T, int DB>
struct HeadShape {
  static constexpr int kBytes = DB * 32 * (int)sizeof(T);
  // In LDS.  (192 where 256 left room for two workgroups to a CU, not three: 4 x 1025 x
  // 16 x 72 fp16 54.8, so 46.4 us.)
  static constexpr int kRow = kBytes <= 128 ? 128 : kBytes == 192 ? 192 : kBytes <= 256 ? 256 : 512;
  static constexpr int kSteps = DB * 32 / kPerStep<T>;
};
// a block of 32 rows as an operand: so many steps, of so many registers of a tile
template <class T>
constexpr int kAcrossSteps = 32 / kPerStep<T>;
template <class T>
constexpr int kAcrossRegs = kPerStep<T> / 2;
// reads of an operand across rows
template <class T>
constexpr int kAcrossReads = sizeof(T) == 4 ? 4 : 2;
constexpr int kAhead = 4;

// The workgroup's (batch, key head) and its item among theirs.  Ids go round the
// XCDs (id % 8); where the pairs can be dealt out evenly, a pair's keys stay in one
// XCD's cache.
struct Where {
  int b, kvh, item;
};
template <bool kItemsFirst = false>
__device__ __forceinline__ Where where(const AttentionParams& p, unsigned id, int items) {
  const unsigned step = p.spread ? 8 : 1, j = id / step;
  if (kItemsFirst && p.causal) {
    const unsigned pairs = (unsigned)(p.batch * p.kv_heads) / step, pair = j % pairs * step + id % step;
    return {(int)(pair / p.kv_heads), (int)(pair % p.kv_heads), (int)(j / pairs)};
  }
  const unsigned pair = j / items * step + id % step;
  return {(int)(pair / p.kv_heads), (int)(pair % p.kv_heads), (int)(j % items)};
}

// kTile rows of memory, from `from` on, to a tile in LDS; rows from `rows` on and
// chunks from `chunks` on arrive as zeros.
template <int kRow, int kTile, int kThreads = kAttentionThreads>
__device__ __forceinline__ void fetch_tile(const char* from, uint32_t stride, int rows, int chunks, uint32_t to) {
  constexpr int kChunksOfRow = kRow / 16;
  static_assert(kTile * kChunksOfRow % kThreads == 0, "whole instructions");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t size = rows <= 0 ? 0u : (uint32_t)(min(rows, kTile) - 1) * stride + (uint32_t)chunks * 16u;
  const Descriptor d = describe(from, size);
#pragma unroll
  for (int j = 0; j < kTile * kChunksOfRow / kThreads; ++j) {
    const int slot = j * kThreads + threadIdx.x, r = slot / kChunksOfRow;
    const int chunk = (slot % kChunksOfRow) ^ swizzle<kRow>(r);
    const uint32_t offset = chunk < chunks ? (uint32_t)r * stride + (uint32_t)chunk * 16u : kNowhere;
    load_to_lds(d, offset, to + (uint32_t)(j * kThreads * 16 + wave * (kWave * 16)));
  }
}
template <int kRow, int kTile, int kThreads>
constexpr int kLoadsOfTile = kTile * kRow / (kThreads * 16);  // a wave's

// A lane's chunks of its row: 2 t + h; zeros past the row's chunks and where it is
// not live (`row` can be read all the same).
template <class T, int DB>
__device__ __forceinline__ void load_row(const char* row, bool live, int chunks, Chunk (&to)[HeadShape<T, DB>::kSteps]) {
  const int h = threadIdx.x >> 5 & 1;
#pragma unroll
  for (int t = 0; t < HeadShape<T, DB>::kSteps; ++t) {
    const int c = 2 * t + h;
    to[t] = *reinterpret_cast<const Chunk*>(row + (c < chunks ? c : 0) * 16);
    if (!live || c >= chunks) to[t] = Chunk{0, 0, 0, 0};
  }
}

// s = rows `row` .. row + 31 of the tile times the lane's row
template <class T, int DB>
__device__ __forceinline__ Sums along(const Lds* tile, int offset, int row, const Chunk (&mine)[HeadShape<T, DB>::kSteps]) {
  Sums s = {};
#pragma unroll
  for (int t = 0; t < HeadShape<T, DB>::kSteps; ++t)
    multiply<T>(s, lds_along<HeadShape<T, DB>::kRow>(tile, offset, row, t), mine[t]);
  return s;
}
// ... where the lane's row is row `other` + lane % 32 of another tile
template <class T, int DB>
__device__ __forceinline__ Sums along_both(const Lds* tile, const Lds* others, int offset, int row, int other) {
  constexpr int kRow = HeadShape<T, DB>::kRow;
  Sums s = {};
#pragma unroll
  for (int t = 0; t < HeadShape<T, DB>::kSteps; ++t)
    multiply<T>(s, lds_along<kRow>(tile, offset, row, t), lds_along<kRow>(others, offset, other, t));
  return s;
}
// to[block] += (columns of the tile's rows `row` .. row + 31) times w
template <class T, int DB>
__device__ __forceinline__ void across(Sums (&to)[DB], const Lds* tile, int offset, int row, const Sums& w) {
#pragma unroll
  for (int t = 0; t < kAcrossSteps<T>; ++t) {
    const Chunk b = operand_of<T>(w, t * kAcrossRegs<T>);
#pragma unroll
    for (int d = 0; d < DB; ++d)
      multiply<T>(to[d], lds_across<T, HeadShape<T, DB>::kRow>(tile, offset, row + t * kPerStep<T>, d), b);
  }
}
// the row of a tile's register r
__device__ __forceinline__ int row_of(int r) { return 8 * (r >> 2) + 4 * (int)(threadIdx.x >> 5 & 1) + (r & 3); }

// Four elements of a result and, where it is wanted, what their rounding leaves: the
// backward's delta_i = do_i . o_i is the difference of numbers that may be far
// larger than ds_ij / p_ij, and with o_i rounded to bf16 a third of dq's error came of
// it (4 x 4096 x 16 x 128: 2.6e-3 of the norm to 2.4e-3).
template <class T>
__device__ __forceinline__ void store_with_rest(T* to, T* rest, Wide<4> v) {
  const Vec<T, 4> n = narrow<T, 4>(v);
  store<T, 4>(to, n);
  if constexpr (sizeof(T) == 2)
    if (rest) store<T, 4>(rest, narrow<T, 4>(v - widen<T, 4>(n)));
}
// v times factor 2^power
template <int N>
__device__ __forceinline__ Wide<N> times(Wide<N> v, float factor, int power) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = __builtin_amdgcn_ldexpf(v[k] * factor, power);
  return v;
}
// A lane's row of the result, of which it holds the columns row_of() of each block,
// times factor 2^power.
template <class T, int DB>
__device__ __forceinline__ void store_row(T* row, const Sums (&v)[DB], float factor, int dim, T* rest = nullptr,
                                          int power = 0) {
  const int h = threadIdx.x >> 5 & 1;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int column = 32 * d + 8 * k + 4 * h;
      Wide<4> w;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = v[d][4 * k + e];
      if (column < dim) store_with_rest<T>(row + column, rest ? rest + column : nullptr, times<4>(w, factor, power));
    }
}

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// What is subtracted from the scaled scores of a row whose largest score is `top`.  It is rounded, by up
// to 2^-24 of itself, and 2 to that is in all of the row's probabilities: 2^64 below 2^31, 2^8 below 2^28
// (fp16).  A row past that is NaN, not one that has lost its keys; one as far below 0 gives zeros, as one of
// minus infinity does.
// fp16's probabilities are kept times 2^7, the most that its largest number leaves where they may be 2^8:
// of 2^17 keys with 2^-26 of the largest weight each, 2^-9 of the result, nothing was left without.
constexpr float kSlackBelow = 0x1p23f;  // further out a score's own step is 1 and more
template <class T>
__device__ __forceinline__ float base_of(const AttentionParams& p, float top) {
  constexpr float kMost = kScaled<T> ? 0x1p28f : 0x1p31f;
  const float base = top * p.scale2;
  if (top == -INFINITY) return 0.0f;
  if (kScaled<T> && fabsf(base) < kSlackBelow) return base - 7.0f;
  return base < kMost ? fmaxf(base, -kMost) : NAN;
}

// What rows see: of sequence b the first q_length queries, the first k_length
// keys; with causal order the last query sees the last key.
struct Seen {
  int q_length, k_length, shift;  // query i sees keys up to i + shift
};
__device__ __forceinline__ Seen seen_of(const AttentionParams& p, int b) {
  Seen s;
  s.q_length = p.q_length ? min(max(p.q_length[b], 0), p.q_tokens) : p.q_tokens;
  s.k_length = p.k_length ? min(max(p.k_length[b], 0), p.k_tokens) : p.k_tokens;
  s.shift = p.causal ? s.k_length - s.q_length : s.k_length;
  return s;
}
// the last key that query i sees; < 0: none
__device__ __forceinline__ int last_key(const Seen& s, int i) {
  return i < s.q_length ? min(s.k_length - 1, i + s.shift) : -1;
}
// ... and the last whose score matters: a row that sees one key gives it all, whatever its
// score, and has no gradient, where do . v - do . o would leave its roundings.  (Such rows
// come first of those that see any: the comparisons are made wherever they are.)
__device__ __forceinline__ int last_with_slope(const Seen& s, int i) {
  const int last = last_key(s, i);
  return last == 0 ? -1 : last;
}
// Of the rows from `first` to `end`, all of a group's heads a token: the last key that
// each of them sees (past it scores are compared), and the last that any does (past it
// there is nothing to do).
struct Reach {
  int open, any;
};
__device__ __forceinline__ Reach reach_of(const AttentionParams& p, const Seen& seen, int first, int end) {
  if (first >= end) return {-1, -1};
  const int last = (end - 1) / p.group;
  return {last < seen.q_length ? last_key(seen, first / p.group) : -1,
          first / p.group < seen.q_length ? last_key(seen, min(last, seen.q_length - 1)) : -1};
}

// ---- four waves' sums of the same 32 rows together, through the LDS
template <int DB>
struct JoinShape {
  static constexpr int kPitch = DB * 32 + 4;  // floats of a row
  static constexpr int kBytes = 4 * 32 * kPitch * 4;
};
// A wave's own; landed_for_all() comes before and after.
template <int DB>
__device__ __forceinline__ void give_to_join(char* lds, const Sums (&v)[DB]) {
  const int wave = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
  store_row<float, DB>((float*)lds + (wave * 32 + (lane & 31)) * JoinShape<DB>::kPitch, v, 1.0f, DB * 32);
}
// The sums of row lane % 32, four columns at a time: take(column, sum).
template <int DB, class Take>
__device__ __forceinline__ void take_joined(const char* lds, int dim, Take take) {
  const int row = threadIdx.x & 31;
#pragma unroll
  for (int c = 4 * (threadIdx.x >> 5); c < DB * 32; c += 32) {
    if (c >= dim) break;
    const float* from = (const float*)lds + row * JoinShape<DB>::kPitch + c;
    Wide<4> sum = {};
#pragma unroll
    for (int w = 0; w < 4; ++w) sum += load<float, 4>(from + w * 32 * JoinShape<DB>::kPitch);
    take(c, sum);
  }
}

// ---------------------------------------------------------------- forward
// NW waves.  KW of them share rows and take keys in turn: 1, a wave has 32 rows of
// its own; 4, all have the same 32 (few rows, many keys).
// The bound is the matrix instructions (56% of the cycles), and the exponentials where they
// run beside none: 1 x 16384 x 16 x 128 bf16 1870 to 2000 us, 1.10 to 1.18 PFLOP/s at 1.9 to
// 2.0 GHz (1650 without the softmax).  One token against 8 x 8193 keys, 32 (8) heads of 128: the
// memory, 44 to 48 us, 3.9 to 4.2 TB/s, and 4 for the join.
//
// Tiles of keys are loaded kBuffers - 1 ahead.  Eight waves with four buffers, one
// workgroup to a CU, ask the caches for half of what two workgroups of four waves do
// and wait less for it (heads of 97 to 128 in a half type with rows enough:
// 16384 x 16 x 128 bf16 2044, so 1948 us).
template <class T, int DB, int KW, int NW>
struct ForwardShape {
  static constexpr int kThreads = NW * kWave;
  static constexpr int kKeys = KW == 1 ? 64 : 128;  // of a tile
  static constexpr int kBlocks = KW == 1 ? 2 : 1;   // of 32 keys, a wave's
  static constexpr int kRows = NW / KW * 32;        // of the workgroup
  static constexpr int kTileBytes = kKeys * HeadShape<T, DB>::kRow;
  static constexpr int kRoom = NW == 8 || KW == 4 || sizeof(T) == 4 ? 128 << 10 : DB > 2 ? 64 << 10 : 48 << 10;
  static constexpr int kBuffers = kRoom / (2 * kTileBytes) > 4 ? 4 : kRoom / (2 * kTileBytes);
  static constexpr int kLoads = 2 * kLoadsOfTile<HeadShape<T, DB>::kRow, kKeys, kThreads>;
  static constexpr int kJoin = KW == 1 ? 0 : JoinShape<DB>::kBytes;
  static constexpr int kTiles = 2 * kBuffers * kTileBytes;
  static constexpr int kLds = kTiles > kJoin ? kTiles : kJoin;
};

template <class T, int DB, int KW, int NW>
__global__ void __launch_bounds__(NW* kWave, (sizeof(T) == 2 && KW == 1) ? 2 : 1)
attention_forward(const AttentionParams p) {
  using Shape = ForwardShape<T, DB, KW, NW>;
  using Head = HeadShape<T, DB>;
  __shared__ __attribute__((aligned(1024))) char lds_[Shape::kLds];
  __shared__ float joined[2][4][32];
  Lds* lds = (Lds*)lds_;
  const uint32_t lds_at = lds_address(lds);
  const Where at = where(p, blockIdx.x, p.tiles * p.splits);
  if (at.b >= p.batch) return;
  // (the last rows see most: first)
  const int tile = p.tiles - 1 - at.item / p.splits, split = at.item % p.splits;
  const Seen seen = seen_of(p, at.b);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x & (kWave - 1);
  const int chunks = p.dim / kPerChunk<T>;

  const int rows = p.q_tokens * p.group;
  const int first_row = tile * Shape::kRows;
  const int row_ = first_row + (KW == 1 ? wave * kRowsOfWave : 0) + (lane & 31);
  const bool there = row_ < rows;
  const int row = there ? row_ : 0;
  const int token = row / p.group, head = at.kvh * p.group + row % p.group;
  const int last = there ? last_key(seen, token) : -1;
  Chunk q[Head::kSteps];
  load_row<T, DB>(p.q.p + at.b * p.q.batch + (int64_t)token * p.q.token + head * p.q.head,
                  there && token < seen.q_length, chunks, q);

  // the keys of the workgroup: those that its last row sees, and of them its share
  const int keys = reach_of(p, seen, first_row, min(first_row + Shape::kRows, rows)).any + 1;
  const int key_tiles = (keys + Shape::kKeys - 1) / Shape::kKeys;
  const int each = (key_tiles + p.splits - 1) / p.splits;
  const int begin = min(split * each, key_tiles), end = min(begin + each, key_tiles);
  const int wave_row = first_row + (KW == 1 ? wave * kRowsOfWave : 0);
  const Reach reach = reach_of(p, seen, wave_row, min(wave_row + kRowsOfWave, rows));

  const char* k_from = p.k.p + at.b * p.k.batch + at.kvh * p.k.head;
  const char* v_from = p.v.p + at.b * p.v.batch + at.kvh * p.v.head;
  auto fetch = [&](int t) {  // (none past the end: their loads are counted all the same)
    const int key = t * Shape::kKeys, left = t < end ? seen.k_length - key : 0;
    const uint32_t to = lds_at + ((t - begin) % Shape::kBuffers) * 2 * Shape::kTileBytes;
    fetch_tile<Head::kRow, Shape::kKeys, Shape::kThreads>(k_from + (int64_t)key * p.k.token, p.k.token, left, chunks, to);
    fetch_tile<Head::kRow, Shape::kKeys, Shape::kThreads>(v_from + (int64_t)key * p.v.token, p.v.token, left, chunks,
                                                          to + Shape::kTileBytes);
  };

  const int along_at = along_offset<Head::kRow>(), across_at = across_offset<T, Head::kRow>();
  Sums o[DB] = {};
  // The row's reference, a maximum so far: p = exp2(scale2 s - base).  It is raised, and
  // the sums with it, only where scores pass it by 2^8 in p, which the types and the
  // sums hold: in a long row seldom, where a larger maximum comes with every other tile.
  float m = -INFINITY, base = 0.0f, limit = -INFINITY;
  const float slack = 8.0f / fmaxf(p.scale2, 0x1p-100f);  // (finite: of -infinity and it the limit is -infinity)
  float l = 0.0f;  // the sum of this lane's half
  constexpr int kEarly = Shape::kBuffers > 1 ? Shape::kBuffers - 1 : 1;
  if (begin < end) {
#pragma unroll
    for (int t = 0; t < kEarly; ++t) fetch(begin + t);
  }
  for (int t = begin; t < end; ++t) {
    landed_for_all<(kEarly - 1) * Shape::kLoads>();
    if constexpr (Shape::kBuffers > 1) fetch(t + kEarly);
    const Lds* k_tile = lds + ((t - begin) % Shape::kBuffers) * 2 * Shape::kTileBytes;
    const Lds* v_tile = k_tile + Shape::kTileBytes;
    const int in_tile = KW == 1 ? 0 : wave * 32;
    const int key = t * Shape::kKeys + in_tile;
    if (key <= reach.any) {
      Sums s[Shape::kBlocks];
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int b = 0; b < Shape::kBlocks; ++b) s[b] = along<T, DB>(k_tile, fresh(along_at), in_tile + 32 * b, q);
      read_ahead<kAhead, kInstructions<T>, Shape::kBlocks * Head::kSteps, 1>();
      __builtin_amdgcn_s_setprio(0);
      if (key + 32 * Shape::kBlocks - 1 > reach.open) {
#pragma unroll
        for (int b = 0; b < Shape::kBlocks; ++b)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            s[b][r] = key + 32 * b + row_of(r) > last ? -INFINITY : s[b][r];
      }
      float top = -INFINITY;
#pragma unroll
      for (int b = 0; b < Shape::kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, s[b][r]);
      top = halves_max(top);
      if (__any(top > limit)) {
        const float before = m == -INFINITY ? -INFINITY : base;
        m = fmaxf(m, top);
        base = base_of<T>(p, m);
        limit = m + (fabsf(base) < kSlackBelow ? slack : 0.0f);
        const float less = exp2_fast(before - base);
        l *= less;
#pragma unroll
        for (int d = 0; d < DB; ++d) o[d] *= less;
      }
#pragma unroll
      for (int b = 0; b < Shape::kBlocks; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[b][r] = exp2_fast(fmaf(s[b][r], p.scale2, -base));
          l += s[b][r];
        }
#pragma unroll
      for (int b = 0; b < Shape::kBlocks; ++b) across<T, DB>(o, v_tile, fresh(across_at), in_tile + 32 * b, s[b]);
      read_ahead<kAhead, kInstructions<T>, Shape::kBlocks * DB * kAcrossSteps<T>, kAcrossReads<T>>();
    }
    if constexpr (Shape::kBuffers == 1) {
      landed_for_all();
      fetch(t + 1);
    }
  }
  landed_for_all();  // what was fetched past the end, too
  l = halves_sum(l);

  if constexpr (KW == 4) {  // the waves' results together
    if (lane < 32) joined[0][wave][lane] = m;
    landed_for_all();
    float top = joined[0][0][lane & 31];
#pragma unroll
    for (int w = 1; w < 4; ++w) top = fmaxf(top, joined[0][w][lane & 31]);
    const float before = m == -INFINITY ? -INFINITY : base;
    base = base_of<T>(p, top);
    const float less = exp2_fast(before - base);
    l *= less;
    if (lane < 32) joined[1][wave][lane] = l;
#pragma unroll
    for (int d = 0; d < DB; ++d) o[d] *= less;
    give_to_join<DB>(lds_, o);
    landed_for_all();
    l = joined[1][0][lane & 31] + joined[1][1][lane & 31] + joined[1][2][lane & 31] + joined[1][3][lane & 31];
  }

  const float inverse = l > 0.0f || l != l ? 1.0f / l : 0.0f;
  const float lse = l > 0.0f || l != l ? base + __builtin_amdgcn_logf(l) : -INFINITY;
  const int64_t stat = ((int64_t)at.b * p.heads + head) * p.q_tokens + token;
  const int64_t part = (int64_t)split * p.batch * p.heads * p.q_tokens;
  const bool whole = p.splits == 1;
  if (there && lane < 32 && (KW == 1 || wave == 0)) {
    if (!whole) p.part_lse[part + stat] = lse;
    else if (p.lse) p.lse[stat] = lse == -INFINITY ? INFINITY : lse;
  }
  const int64_t dense = (((int64_t)at.b * p.q_tokens + token) * p.heads + head) * p.dim;
  T* out = static_cast<T*>(p.out) + dense;
  T* rest = p.rest ? static_cast<T*>(p.rest) + dense : nullptr;
  float* part_out = p.part_out + (part + stat) * p.dim;
  if constexpr (KW == 1) {
    if (!there) return;
    if (whole) store_row<T, DB>(out, o, inverse, p.dim, rest);
    else store_row<float, DB>(part_out, o, inverse, p.dim);
  } else {
    if (!there) return;
    take_joined<DB>(lds_, p.dim, [&](int c, Wide<4> sum) {
      sum *= inverse;
      if (whole) store_with_rest<T>(out + c, rest ? rest + c : nullptr, sum);
      else store<float, 4>(part_out + c, sum);
    });
  }
}

// The parts of the keys together: a wave to a row.
template <class T>
__global__ void __launch_bounds__(kAttentionThreads) attention_join(const AttentionParams p) {
  const int64_t rows = (int64_t)p.batch * p.heads * p.q_tokens;
  const int64_t row = (int64_t)blockIdx.x * (kAttentionThreads / kWave) + threadIdx.x / kWave;  // (b, head, token)
  const int lane = threadIdx.x & (kWave - 1);
  if (row >= rows) return;
  float top = -INFINITY;
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, p.part_lse[s * rows + row]);
  const float base = top == -INFINITY ? 0.0f : top;
  const int64_t token = row % p.q_tokens, head = row / p.q_tokens % p.heads, b = row / p.q_tokens / p.heads;
  const int64_t dense = ((b * p.q_tokens + token) * p.heads + head) * p.dim;
  float weights = 0.0f;
  const int column = 4 * (lane & 31), half = lane >> 5;  // each half of the wave takes every second part
  Wide<4> sum = {};
  for (int s = half; s < p.splits; s += 2) {
    const float w = exp2_fast(p.part_lse[s * rows + row] - base);
    weights += w;
    if (column < p.dim) sum += w * load<float, 4>(p.part_out + (s * rows + row) * p.dim + column);
  }
  weights = halves_sum(weights);
#pragma unroll
  for (int k = 0; k < 4; ++k) sum[k] = halves_sum(sum[k]);
  const float inverse = weights > 0.0f || weights != weights ? 1.0f / weights : 0.0f;
  if (half == 0 && column < p.dim)
    store_with_rest<T>(static_cast<T*>(p.out) + dense + column,
                       p.rest ? static_cast<T*>(p.rest) + dense + column : nullptr, sum * inverse);
  if (p.lse && lane == 0) p.lse[row] = weights > 0.0f || weights != weights ? base + __builtin_amdgcn_logf(weights) : INFINITY;
}

// ---------------------------------------------------------------- the range of fp16
// A long row's ds_ij are far smaller than fp16's normal numbers, and where the
// gradients are scaled up they may pass its largest.  So they are rounded times
// 2^e, with |ds_ij| <= 2 max |do_i| max |v_j| kept below 2^15; the products are
// divided again in fp32.
constexpr int kNormParts = 16;

// Each of kNormParts workgroups of a (batch, key head) takes a part of its rows and
// keys, 16 lanes to one.
template <class T>
__global__ void __launch_bounds__(kAttentionThreads) attention_norms(const AttentionParams p) {
  __shared__ float most[2][kAttentionThreads / kWave];
  const int part = blockIdx.x % kNormParts;
  const unsigned pair = blockIdx.x / kNormParts;
  const int b = pair / p.kv_heads, kvh = pair % p.kv_heads;
  const Seen seen = seen_of(p, b);
  const int group = threadIdx.x / 16, chunk = threadIdx.x % 16, chunks = p.dim / kPerChunk<T>;
  auto square = [&](const char* row) {
    float s = 0.0f;
    if (chunk < chunks) {
      const Wide<8> v = widen<T, 8>(load<T, 8>(reinterpret_cast<const T*>(row) + chunk * 8));
#pragma unroll
      for (int k = 0; k < 8; ++k) s = fmaf(v[k], v[k], s);
    }
    return lanes_sum<16>(s);
  };
  float top[2] = {0.0f, 0.0f};
  const int rows = seen.q_length * p.group;
  for (int r = part * 16 + group; r < rows; r += 16 * kNormParts) {
    const int64_t at = (((int64_t)b * p.q_tokens + r / p.group) * p.heads + kvh * p.group + r % p.group) * p.dim;
    top[0] = fmaxf(top[0], square(static_cast<const char*>(p.d_out) + at * (int64_t)sizeof(T)));
  }
  for (int j = part * 16 + group; j < seen.k_length; j += 16 * kNormParts)
    top[1] = fmaxf(top[1], square(p.v.p + b * p.v.batch + kvh * p.v.head + (int64_t)j * p.v.token));
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    for (int step = 16; step < kWave; step *= 2) top[k] = fmaxf(top[k], __shfl_xor(top[k], step));
    if ((threadIdx.x & (kWave - 1)) == 0) most[k][threadIdx.x / kWave] = top[k];
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    const float* m = most[threadIdx.x];
    p.norms[blockIdx.x * 2 + threadIdx.x] = sqrtf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
  }
}
// e, for all lanes of the wave
template <class T>
__device__ __forceinline__ int range_of(const AttentionParams& p, const Where& at) {
  if constexpr (!kScaled<T>) return 0;
  const float* from = p.norms + ((int64_t)at.b * p.kv_heads + at.kvh) * kNormParts * 2 + 2 * (threadIdx.x % kNormParts);
  float a = from[0], b = from[1];
  for (int step = 1; step < kNormParts; step *= 2) {
    a = fmaxf(a, __shfl_xor(a, step));
    b = fmaxf(b, __shfl_xor(b, step));
  }
  const float most = a * b;
  if (!(most > 0.0f && most < 0x1p120f)) return 0;
  return min(13 - __builtin_amdgcn_frexp_expf(most), 100);  // most < 2^exponent
}

// ---------------------------------------------------------------- gradient of the queries
// As the forward: a wave has 32 rows, the keys go by.  It forms delta_i = do_i . o_i
// and leaves it for the other kernel.  Three products; the bound is the chain of scores,
// exponentials and products in each wave, beside which only the SIMD's other wave runs: matrix
// instructions take 35% of the cycles (the forward's 30, the keys' and values' gradients', of four
// products, 31).  4 x 4096 x 16 (8) x 128 bf16, causal, sequences of different lengths: 251 us, the
// forward 190, the keys' and values' gradients 371.
template <class T, int DB, int KW, int NW>
struct QueriesShape {
  static constexpr int kThreads = NW * kWave;
  static constexpr int kKeys = KW == 1 ? 64 : 128;
  static constexpr int kRows = NW / KW * 32;
  static constexpr int kTileBytes = kKeys * HeadShape<T, DB>::kRow;
  static constexpr int kRoom = NW == 8 || KW == 4 || sizeof(T) == 4 ? 128 << 10 : DB > 2 ? 64 << 10 : 48 << 10;
  static constexpr int kBuffers = kRoom / (2 * kTileBytes) > 4 ? 4 : kRoom / (2 * kTileBytes);
  static constexpr int kLoads = 2 * kLoadsOfTile<HeadShape<T, DB>::kRow, kKeys, kThreads>;
  static constexpr int kJoin = KW == 1 ? 0 : JoinShape<DB>::kBytes;
  static constexpr int kTiles = 2 * kBuffers * kTileBytes;
  static constexpr int kLds = kTiles > kJoin ? kTiles : kJoin;
};

// kDelta: it forms delta and leaves it; else delta is there.
template <class T, int DB, int KW, int NW, bool kDelta>
__device__ __forceinline__ void grad_q_tile(const AttentionParams& p, unsigned block, char* lds_) {
  using Shape = QueriesShape<T, DB, KW, NW>;
  using Head = HeadShape<T, DB>;
  Lds* lds = (Lds*)lds_;
  const uint32_t lds_at = lds_address(lds);
  const Where at = where(p, block, p.tiles);
  if (at.b >= p.batch) return;
  const int tile = p.tiles - 1 - at.item;
  const Seen seen = seen_of(p, at.b);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x & (kWave - 1);
  const int chunks = p.dim / kPerChunk<T>;
  const int rows = p.q_tokens * p.group;
  const int first_row = tile * Shape::kRows;
  const int row_of_wave = first_row + (KW == 1 ? wave * kRowsOfWave : 0);
  const int row_ = row_of_wave + (lane & 31);
  const bool there = row_ < rows;
  const int row = there ? row_ : 0;
  const int token = row / p.group, head = at.kvh * p.group + row % p.group;
  const bool live = there && token < seen.q_length;
  const int last = there ? last_with_slope(seen, token) : -1;
  const int64_t dense = (((int64_t)at.b * p.q_tokens + token) * p.heads + head) * p.dim;
  const int64_t stat = ((int64_t)at.b * p.heads + head) * p.q_tokens + token;

  Chunk q[Head::kSteps], d_out[Head::kSteps];
  load_row<T, DB>(p.q.p + at.b * p.q.batch + (int64_t)token * p.q.token + head * p.q.head, live, chunks, q);
  load_row<T, DB>((const char*)p.d_out + dense * (int64_t)sizeof(T), live, chunks, d_out);
  float delta = 0.0f;
  if constexpr (!kDelta) {
    if (there) delta = p.delta[stat];
  } else {
    constexpr int N = kPerChunk<T>;
    constexpr bool kRest = sizeof(T) == 2;
    Chunk o[Head::kSteps], o_rest[kRest ? Head::kSteps : 1];
    load_row<T, DB>((const char*)p.o + dense * (int64_t)sizeof(T), live, chunks, o);
    if constexpr (kRest) load_row<T, DB>((const char*)p.o_rest + dense * (int64_t)sizeof(T), live, chunks, o_rest);
#pragma unroll
    for (int t = 0; t < Head::kSteps; ++t) {
      Wide<N> a = widen<T, N>(__builtin_bit_cast(Vec<T, N>, o[t]));
      if constexpr (kRest) a += widen<T, N>(__builtin_bit_cast(Vec<T, N>, o_rest[t]));
      const Wide<N> b = widen<T, N>(__builtin_bit_cast(Vec<T, N>, d_out[t]));
#pragma unroll
      for (int k = 0; k < N; ++k) delta = fmaf(a[k], b[k], delta);
    }
    delta = halves_sum(delta);
  }
  if (kDelta && there && lane < 32 && (KW == 1 || wave == 0)) p.delta[stat] = delta;
  const float lse = there ? p.lse[stat] : INFINITY;
  const int range = range_of<T>(p, at);
  const float up = ldexpf(1.0f, range);

  const int keys = reach_of(p, seen, first_row, min(first_row + Shape::kRows, rows)).any + 1;
  const int end = (keys + Shape::kKeys - 1) / Shape::kKeys;
  const Reach reach = reach_of(p, seen, row_of_wave, min(row_of_wave + kRowsOfWave, rows));

  const char* k_from = p.k.p + at.b * p.k.batch + at.kvh * p.k.head;
  const char* v_from = p.v.p + at.b * p.v.batch + at.kvh * p.v.head;
  auto fetch = [&](int t) {
    const int key = t * Shape::kKeys, left = t < end ? seen.k_length - key : 0;
    const uint32_t to = lds_at + (t % Shape::kBuffers) * 2 * Shape::kTileBytes;
    fetch_tile<Head::kRow, Shape::kKeys, Shape::kThreads>(k_from + (int64_t)key * p.k.token, p.k.token, left, chunks, to);
    fetch_tile<Head::kRow, Shape::kKeys, Shape::kThreads>(v_from + (int64_t)key * p.v.token, p.v.token, left, chunks,
                                                          to + Shape::kTileBytes);
  };
  const int along_at = along_offset<Head::kRow>(), across_at = across_offset<T, Head::kRow>();
  Sums dq[DB] = {};
  constexpr int kEarly = Shape::kBuffers > 1 ? Shape::kBuffers - 1 : 1;
  if (end > 0) {
#pragma unroll
    for (int t = 0; t < kEarly; ++t) fetch(t);
  }
  for (int t = 0; t < end; ++t) {
    landed_for_all<(kEarly - 1) * Shape::kLoads>();
    if constexpr (Shape::kBuffers > 1) fetch(t + kEarly);
    const Lds* k_tile = lds + (t % Shape::kBuffers) * 2 * Shape::kTileBytes;
    const Lds* v_tile = k_tile + Shape::kTileBytes;
#pragma unroll
    for (int b = 0; b < (KW == 1 ? Shape::kKeys / 32 : 1); ++b) {
      const int in_tile = KW == 1 ? 32 * b : 32 * wave;
      const int key = t * Shape::kKeys + in_tile;
      if (key > reach.any) continue;
      Sums s = along<T, DB>(k_tile, fresh(along_at), in_tile, q);
      const Sums dp = along<T, DB>(v_tile, fresh(along_at), in_tile, d_out);
      read_ahead<kAhead, kInstructions<T>, 2 * Head::kSteps, 1>();
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[r] = exp2_fast(fmaf(s[r], p.scale2, -lse)) * (dp[r] - delta);
        if constexpr (kScaled<T>) s[r] *= up;
      }
      if (key + 31 > reach.open) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          s[r] = key + row_of(r) > last ? 0.0f : s[r];
      }
      across<T, DB>(dq, k_tile, fresh(across_at), in_tile, s);
      read_ahead<kAhead, kInstructions<T>, DB * kAcrossSteps<T>, kAcrossReads<T>>();
    }
    if constexpr (Shape::kBuffers == 1) {
      landed_for_all();
      fetch(t + 1);
    }
  }
  landed_for_all();  // what was fetched past the end, too
  T* to = static_cast<T*>(p.dq) + dense;
  const int power = p.scale_power - range;
  if constexpr (KW == 1) {
    if (there && p.dq) store_row<T, DB>(to, dq, p.scale, p.dim, nullptr, power);
  } else {
    give_to_join<DB>(lds_, dq);
    landed_for_all();
    if (there && p.dq)
      take_joined<DB>(lds_, p.dim, [&](int c, Wide<4> sum) { store<T, 4>(to + c, narrow<T, 4>(times<4>(sum, p.scale, power))); });
  }
}

template <class T, int DB, int KW, int NW>
__global__ void __launch_bounds__(NW* kWave, sizeof(T) == 2 && KW == 1 ? 2 : 1) attention_grad_q(const AttentionParams p) {
  __shared__ __attribute__((aligned(1024))) char lds[QueriesShape<T, DB, KW, NW>::kLds];
  grad_q_tile<T, DB, KW, NW, true>(p, blockIdx.x, lds);
}

// delta alone, 16 lanes to a row.
template <class T>
__global__ void __launch_bounds__(kAttentionThreads) attention_delta(const AttentionParams p) {
  const int64_t rows = (int64_t)p.batch * p.q_tokens * p.heads;
  const int64_t row = (int64_t)blockIdx.x * (kAttentionThreads / 16) + threadIdx.x / 16;  // (b, token, head)
  if (row >= rows) return;
  constexpr int N = 128 / 16;  // elements of a lane
  const int column = (int)(threadIdx.x % 16) * N;
  const int64_t head = row % p.heads, token = row / p.heads % p.q_tokens, b = row / p.heads / p.q_tokens;
  float delta = 0.0f;
  if (column < p.dim && (int)token < seen_of(p, (int)b).q_length) {
    const int64_t at = row * p.dim + column;
    const Wide<N> d = widen<T, N>(load<T, N>(static_cast<const T*>(p.d_out) + at));
    Wide<N> o = widen<T, N>(load<T, N>(static_cast<const T*>(p.o) + at));
    if constexpr (sizeof(T) == 2) o += widen<T, N>(load<T, N>(static_cast<const T*>(p.o_rest) + at));
#pragma unroll
    for (int k = 0; k < N; ++k) delta = fmaf(o[k], d[k], delta);
  }
  delta = lanes_sum<16>(delta);
  if (threadIdx.x % 16 == 0) p.delta[(b * p.heads + head) * p.q_tokens + token] = delta;
}

// ---------------------------------------------------------------- gradients of the keys and values
// A wave has 32 keys; the rows of all heads that share them go by, head after
// head, in one order: no atomics, the same bits every time.
// KW: 4, all waves have the same 32 keys and take the rows in turn.
template <class T, int DB, int KW, int NW>
struct KeysShape {
  static constexpr int kThreads = NW * kWave;
  static constexpr int kKeys = NW / KW * 32;
  // Of half types' widest heads the values are read from LDS each time: with them
  // in registers as well, 224 of 256 are taken and each read from LDS is waited for
  // (4 x 4096 x 16 x 128 bf16: 489, so 431 us).
  static constexpr bool kValuesInLds = sizeof(T) == 2 && DB == 4 && KW == 1;
  static constexpr int kRows =
      KW == 4 ? 128 : !kValuesInLds && 64 * HeadShape<T, DB>::kRow <= 16 << 10 ? 64 : 32;  // of a tile
  static constexpr int kTileBytes = kRows * HeadShape<T, DB>::kRow;
  static constexpr int kValueBytes = kValuesInLds ? kKeys * HeadShape<T, DB>::kRow : 0;
  static constexpr int kRoom = (NW == 8 || KW == 4 ? 128 << 10 : sizeof(T) == 4 || DB > 2 ? 64 << 10 : 48 << 10) - kValueBytes;
  static constexpr int kBuffers = kRoom / (2 * kTileBytes) > 4 ? 4 : kRoom / (2 * kTileBytes);
  static constexpr int kLoads = 2 * kLoadsOfTile<HeadShape<T, DB>::kRow, kRows, kThreads> + 1;
  static constexpr int kStats = kRows < kWave ? kWave : kRows;  // rows that there is room for
  static constexpr int kJoin = KW == 1 ? 0 : JoinShape<DB>::kBytes;
  static constexpr int kTiles = 2 * kBuffers * kTileBytes + kValueBytes;
  static constexpr int kLds = kTiles > kJoin ? kTiles : kJoin;
};
// The probabilities of fp16 are rounded times 2^14: at most 1, most of a long row's
// would be subnormal.
template <class T>
constexpr int kLift = kScaled<T> ? 14 : 0;

template <class T, int DB, int KW, int NW>
__device__ __forceinline__ void grad_kv_tile(const AttentionParams& p, unsigned block, int tiles, char* lds_) {
  using Shape = KeysShape<T, DB, KW, NW>;
  using Head = HeadShape<T, DB>;
  __shared__ __attribute__((aligned(16))) float stats[Shape::kBuffers][2][Shape::kStats];  // [lse, delta][row of the tile]
  Lds* lds = (Lds*)lds_;
  __shared__ float nowhere[kWave];
  const uint32_t lds_at = lds_address(lds), stats_at = lds_address((Lds*)&stats[0][0][0]);
  const uint32_t nowhere_at = lds_address((Lds*)nowhere);
  const Where at = where<true>(p, block, tiles);
  if (at.b >= p.batch) return;
  const Seen seen = seen_of(p, at.b);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x & (kWave - 1);
  const int chunks = p.dim / kPerChunk<T>;
  const int first_key = at.item * Shape::kKeys;
  const int wave_key = first_key + (KW == 1 ? wave * 32 : 0), key = wave_key + (lane & 31);
  const bool live = key < seen.k_length;
  const int key_read = min(key, p.k_tokens - 1);
  Chunk k[Head::kSteps], v[Shape::kValuesInLds ? 1 : Head::kSteps];
  load_row<T, DB>(p.k.p + at.b * p.k.batch + at.kvh * p.k.head + (int64_t)key_read * p.k.token, live, chunks, k);
  const char* v_from = p.v.p + at.b * p.v.batch + at.kvh * p.v.head;
  const Lds* v_tile = lds + 2 * Shape::kBuffers * Shape::kTileBytes;
  if constexpr (!Shape::kValuesInLds)
    load_row<T, DB>(v_from + (int64_t)key_read * p.v.token, live, chunks, v);

  const int range = range_of<T>(p, at);
  const float up = ldexpf(1.0f, range - kLift<T>);
  // tiles of tokens, the first that sees a key of the workgroup's
  const int first_token = max(0, first_key - seen.shift);
  const int begin = p.causal ? first_token / Shape::kRows : 0;
  const int end = first_key < seen.k_length ? (seen.q_length + Shape::kRows - 1) / Shape::kRows : 0;
  const int per_head = max(end - begin, 0), total = per_head * p.group;
  const uint32_t dense_stride = (uint32_t)(p.heads * p.dim) * sizeof(T);
  int next = 0, next_head = at.kvh * p.group, next_tile = begin;  // what fetch takes
  auto fetch = [&]() {
    const int head = min(next_head, p.heads - 1), token = next_tile * Shape::kRows, buffer = next % Shape::kBuffers;
    const int count = next < total ? seen.q_length - token : 0;
    ++next;
    if (++next_tile == end) {
      next_tile = begin;
      ++next_head;
    }
    const uint32_t to = lds_at + buffer * 2 * Shape::kTileBytes;
    fetch_tile<Head::kRow, Shape::kRows, Shape::kThreads>(
        p.q.p + at.b * p.q.batch + head * p.q.head + (int64_t)token * p.q.token, p.q.token, count, chunks, to);
    fetch_tile<Head::kRow, Shape::kRows, Shape::kThreads>(
        (const char*)p.d_out + (((int64_t)at.b * p.q_tokens + token) * p.heads + head) * p.dim * (int64_t)sizeof(T),
        dense_stride, count, chunks, to + Shape::kTileBytes);
    // 64 rows' statistics to a wave, lse or delta.  (Rows that are not there arrive as zeros, and their queries and
    // gradients with them; waves that have none load nothing, since loads are counted alike.)
    const int64_t stat = ((int64_t)at.b * p.heads + head) * p.q_tokens + token;
    const int which = wave & 1, first = (wave >> 1) * kWave, some = first < Shape::kStats ? min(count, Shape::kRows) - first : 0;
    load_words_to_lds(describe((which ? p.delta : p.lse) + stat + first, some <= 0 ? 0 : 4 * min(some, kWave)),
                      4 * (threadIdx.x & (kWave - 1)),
                      first < Shape::kStats ? stats_at + ((buffer * 2 + which) * Shape::kStats + first) * 4 : nowhere_at);
  };
  const int along_at = along_offset<Head::kRow>(), across_at = across_offset<T, Head::kRow>();
  Sums dk[DB] = {}, dv[DB] = {};
  constexpr int kEarly = Shape::kBuffers > 1 ? Shape::kBuffers - 1 : 1;
  if (total > 0) {
    if constexpr (Shape::kValuesInLds)
      fetch_tile<Head::kRow, Shape::kKeys, Shape::kThreads>(v_from + (int64_t)first_key * p.v.token, p.v.token,
                                                            seen.k_length - first_key, chunks,
                                                            lds_at + 2 * Shape::kBuffers * Shape::kTileBytes);
#pragma unroll
    for (int t = 0; t < kEarly; ++t) fetch();
  }
  for (int n = 0, now = begin; n < total; ++n) {
    landed_for_all<(kEarly - 1) * Shape::kLoads>();
    if constexpr (Shape::kBuffers > 1) fetch();
    const int buffer = n % Shape::kBuffers;
    const Lds* q_tile = lds + buffer * 2 * Shape::kTileBytes;
    const Lds* d_tile = q_tile + Shape::kTileBytes;
    const int token = now * Shape::kRows;
    if (++now == end) now = begin;
#pragma unroll
    for (int b = 0; b < (KW == 1 ? Shape::kRows / 32 : 1); ++b) {
      const int in_tile = KW == 1 ? 32 * b : 32 * wave;
      // (of rows that see no key of the wave's there is nothing to add)
      if (last_key(seen, min(token + in_tile + 31, seen.q_length - 1)) < wave_key) continue;
      Sums s = along<T, DB>(q_tile, fresh(along_at), in_tile, k);
      Sums ds;
      if constexpr (Shape::kValuesInLds) ds = along_both<T, DB>(d_tile, v_tile, fresh(along_at), in_tile, wave * 32);
      else ds = along<T, DB>(d_tile, fresh(along_at), in_tile, v);
      read_ahead<kAhead, kInstructions<T>, Head::kSteps, 1, Head::kSteps, Shape::kValuesInLds ? 2 : 1>();
      __builtin_amdgcn_sched_barrier(0);  // (the statistics' reads are none of these)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int first = in_tile + row_of(4 * j);
        const Vec<float, 4> lse = *reinterpret_cast<const Vec<float, 4>*>(&stats[buffer][0][first]);
        const Vec<float, 4> delta = *reinterpret_cast<const Vec<float, 4>*>(&stats[buffer][1][first]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 4 * j + e;
          s[r] = exp2_fast(fmaf(s[r], p.scale2, (float)kLift<T> - lse[e]));
          ds[r] = s[r] * (ds[r] - delta[e]);
          if constexpr (kScaled<T>) ds[r] *= up;
        }
      }
      if (last_key(seen, token + in_tile) < wave_key + 31 || token + in_tile + 31 >= seen.q_length) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[r] = key > last_key(seen, token + in_tile + row_of(r)) ? 0.0f : s[r];
          ds[r] = key > last_with_slope(seen, token + in_tile + row_of(r)) ? 0.0f : ds[r];
        }
      }
      across<T, DB>(dv, d_tile, fresh(across_at), in_tile, s);
      across<T, DB>(dk, q_tile, fresh(across_at), in_tile, ds);
      read_ahead<kAhead, kInstructions<T>, 2 * DB * kAcrossSteps<T>, kAcrossReads<T>>();
    }
    if constexpr (Shape::kBuffers == 1) {
      landed_for_all();
      fetch();
    }
  }
  landed_for_all();  // what was fetched past the end, too
  const int64_t dense = (((int64_t)at.b * p.k_tokens + key_read) * p.kv_heads + at.kvh) * p.dim;
  T *to_k = p.dk ? static_cast<T*>(p.dk) + dense : nullptr, *to_v = p.dv ? static_cast<T*>(p.dv) + dense : nullptr;
  const int power = p.scale_power - range;
  const float v_factor = ldexpf(1.0f, -kLift<T>);
  const bool there = key < p.k_tokens;
  if constexpr (KW == 1) {
    if (there && to_k) store_row<T, DB>(to_k, dk, p.scale, p.dim, nullptr, power);
    if (there && to_v) store_row<T, DB>(to_v, dv, v_factor, p.dim);
  } else {
    give_to_join<DB>(lds_, dk);
    landed_for_all();
    if (there && to_k)
      take_joined<DB>(lds_, p.dim, [&](int c, Wide<4> sum) { store<T, 4>(to_k + c, narrow<T, 4>(times<4>(sum, p.scale, power))); });
    landed_for_all();
    give_to_join<DB>(lds_, dv);
    landed_for_all();
    if (there && to_v)
      take_joined<DB>(lds_, p.dim, [&](int c, Wide<4> sum) { store<T, 4>(to_v + c, narrow<T, 4>(sum * v_factor)); });
  }
}

template <class T, int DB, int KW, int NW>
__global__ void __launch_bounds__(NW* kWave, sizeof(T) == 2 && KW == 1 ? 2 : 1) attention_grad_kv(const AttentionParams p) {
  __shared__ __attribute__((aligned(1024))) char lds[KeysShape<T, DB, KW, NW>::kLds];
  grad_kv_tile<T, DB, KW, NW>(p, blockIdx.x, p.tiles, lds);
}

// Both in one launch, behind attention_delta's, where neither fills the GPU (2 x 257 x
// 6 x 64 fp32: 19.1 and 20.8 us one after the other, so 22.9 and 3.0 of delta's).
template <class T, int DB>
__global__ void __launch_bounds__(kAttentionThreads, 1) attention_grads(const AttentionParams p) {
  using Q = QueriesShape<T, DB, 4, 4>;
  using K = KeysShape<T, DB, 4, 4>;
  __shared__ __attribute__((aligned(1024))) char lds[Q::kLds > K::kLds ? Q::kLds : K::kLds];
  if ((int)blockIdx.x < p.q_blocks) grad_q_tile<T, DB, 4, 4, false>(p, blockIdx.x, lds);
  else grad_kv_tile<T, DB, 4, 4>(p, blockIdx.x - p.q_blocks, p.kv_tiles, lds);
}

// ---------------------------------------------------------------- kernels of a type
struct AttentionTable {
  // [blocks of 32 elements - 1][0: four waves of 32 rows (or keys) each, 1: eight, 2: four that share 32].  NULL:
  // there is none.
  const void* forward[4][3];
  const void* grad_q[4][3];
  const void* grad_kv[4][3];
  const void* grads[4];
  const void* delta;
  const void* join;
  const void* norms;  // NULL: not needed
};
template <class T, int DB>
void fill_attention_table(AttentionTable& t) {
  constexpr int k = DB - 1;
  t.forward[k][0] = (const void*)attention_forward<T, DB, 1, 4>;
  t.forward[k][2] = (const void*)attention_forward<T, DB, 4, 4>;
  t.grad_q[k][0] = (const void*)attention_grad_q<T, DB, 1, 4>;
  t.grad_q[k][2] = (const void*)attention_grad_q<T, DB, 4, 4>;
  t.grad_kv[k][0] = (const void*)attention_grad_kv<T, DB, 1, 4>;
  t.grad_kv[k][2] = (const void*)attention_grad_kv<T, DB, 4, 4>;
  t.grads[k] = (const void*)attention_grads<T, DB>;
  t.forward[k][1] = t.grad_q[k][1] = t.grad_kv[k][1] = nullptr;
  if constexpr (sizeof(T) == 2 && DB == 4) {
    t.forward[k][1] = (const void*)attention_forward<T, DB, 1, 8>;
    t.grad_q[k][1] = (const void*)attention_grad_q<T, DB, 1, 8>;
    t.grad_kv[k][1] = (const void*)attention_grad_kv<T, DB, 1, 8>;
  }
}
template <class T>
AttentionTable make_attention_table() {
  AttentionTable t;
  fill_attention_table<T, 1>(t);
  fill_attention_table<T, 2>(t);
  fill_attention_table<T, 3>(t);
  fill_attention_table<T, 4>(t);
  t.join = (const void*)attention_join<T>;
  t.delta = (const void*)attention_delta<T>;
  t.norms = nullptr;
  if constexpr (kScaled<T>) t.norms = (const void*)attention_norms<T>;
  return t;
}
const AttentionTable& attention_table_f32();
const AttentionTable& attention_table_f16();
const AttentionTable& attention_table_bf16();

}  // namespace ssim_train
