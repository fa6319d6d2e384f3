// What the attention kernels share: the ragged tiling, tiles of rows in LDS, and the fragments of
// the 32x32x16 matrix instruction.
//
// Rows.  There is no mask inside an item, so the G query heads that share a key head are simply
// G times as many rows of that head: packed row r of item b and key head j is token
// q_offsets[b] + r / G, head j G + r % G.  Grouped heads, single tokens and long sequences are
// then one problem [rows, d] x [keys, d] for each (item, key head), and the gradients of a shared
// key head come out summed over its query heads.
//
// Tiles without a plan.  A grid over blocks of B packed rows of ragged items needs no prefix sum:
// item b owns the slots floor(s / B) + b .. floor(e / B) + b, with s, e its first and past-the-end
// packed rows, of which the first ceil((e - s) / B) hold its tiles and the rest (at most one)
// exit.  The starts rise strictly with b, so a slot finds its item by binary search, and there are
// floor(total / B) + items slots, which the host knows.
//
// Products.  Every kernel keeps its own rows as the columns of the accumulator, so a lane holds 16
// scores of one own row: element i of the tile of rows 0 .. 31 is row 8 (i / 4) + 4 (lane / 32) +
// i % 4.  Those 16 values, converted, are the B operand of the next product as they lie: the
// contraction takes rows in the order (lane half, element), and the A operand is read from LDS in
// that same order.  No score crosses lanes except for the maximum and sum of two halves.
#pragma once

#include "device_common.h"
#include "internal.h"
#include "sparse_transformer.h"

namespace submconv {

// Eight contraction values of a lane: lane l holds row (or column) l % 32, values 8 (l / 32) + j.
template <DT D> struct Frag { uint4 v[Elem<D>::kSize / 2]; };

template <DT D> __device__ __forceinline__ f32x16_t mma(const Frag<D>& a, const Frag<D>& b, f32x16_t c) {
  if constexpr (D == DT::F32) {
    // The same 16 contraction steps as the 16-bit form, two at a time (one of each lane half).
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.v[i].x), __uint_as_float(b.v[i].x), c, 0, 0, 0);
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.v[i].y), __uint_as_float(b.v[i].y), c, 0, 0, 0);
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.v[i].z), __uint_as_float(b.v[i].z), c, 0, 0, 0);
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.v[i].w), __uint_as_float(b.v[i].w), c, 0, 0, 0);
    }
    return c;
  } else {
    return mfma32<D>(a.v[0], b.v[0], c);
  }
}

__device__ __forceinline__ f32x16_t zero16() {
  f32x16_t z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// Elements 8 s .. 8 s + 7 of a score tile as the contraction step s (of 2) of the next product.
template <DT D> __device__ __forceinline__ Frag<D> to_frag(const f32x16_t& p, int s) {
  Frag<D> f;
  if constexpr (D == DT::F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      f.v[i] = make_uint4(__float_as_uint(p[8 * s + 4 * i]), __float_as_uint(p[8 * s + 4 * i + 1]),
                          __float_as_uint(p[8 * s + 4 * i + 2]), __float_as_uint(p[8 * s + 4 * i + 3]));
  } else {
    const uint2 lo = pack4<D>(p[8 * s], p[8 * s + 1], p[8 * s + 2], p[8 * s + 3]);
    const uint2 hi = pack4<D>(p[8 * s + 4], p[8 * s + 5], p[8 * s + 6], p[8 * s + 7]);
    f.v[0] = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  return f;
}

// The two lanes that hold a column, l and l + 32, joined in both (one VALU instruction swaps the halves).
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// One tensor as the kernels see it.
template <DT D> struct Heads {
  typename Elem<D>::T* data;
  int64_t row, head;
};

template <DT D> __device__ __forceinline__ Heads<D> heads_of(const subm_heads_t& t) {
  return Heads<D>{static_cast<typename Elem<D>::T*>(t.data), t.row_stride, t.head_stride};
}

// The rows of one (item, key head): q-like tensors take G heads of a token as G rows.
struct RowMap {
  int64_t first;  // first token of the item
  int head0;      // first head
  int group;      // heads a token
  template <DT D> __device__ __forceinline__ typename Elem<D>::T* at(const Heads<D>& t, int row) const {
    const int tok = group == 1 ? row : row / group;
    const int h = group == 1 ? 0 : row - tok * group;
    return t.data + (first + tok) * t.row + (int64_t)(head0 + h) * t.head;
  }
  // index into a float [tokens, heads] array
  __device__ __forceinline__ int64_t stat(int row, int heads) const {
    const int tok = group == 1 ? row : row / group;
    return (first + tok) * heads + head0 + (row - tok * group);
  }
};

// The item of slot `slot` in a tiling by `block` packed rows of `offsets` (each token `group`
// rows), and the slot's tile in it.
__device__ __forceinline__ int find_item(const int64_t* offsets, int64_t total, int items, int group, int block,
                                         int64_t slot, int* tile) {
  const auto start = [&](int b) {
    const int64_t o = offsets[b];
    return (o < 0 ? 0 : o > total ? total : o) * group / block + b;
  };
  int lo = 0, hi = items - 1;  // the last item whose first slot is at or before `slot`
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (start(mid) <= slot) lo = mid;
    else hi = mid - 1;
  }
  const int64_t t = slot - start(lo);
  *tile = t < 0 ? INT32_MAX / block : (int)t;  // (only for offsets that do not rise: no such rows)
  return lo;
}

__device__ __forceinline__ void item_rows(const int64_t* offsets, int64_t total, int b, int64_t* first, int* count) {
  int64_t s = offsets[b], e = offsets[b + 1];
  s = s < 0 ? 0 : s > total ? total : s;
  e = e < s ? s : e > total ? total : e;
  *first = s;
  *count = (int)(e - s);
}

// ------------------------------------------------------------------------ parts of tiles
//
// Tiles do not fill the compute units evenly: few rows against many leave most of them idle, and a
// last round of tiles on a full machine takes as long as the others.  The tiles (slots of all
// heads, head by head) from `whole` on are therefore worked on in `parts` parts of their walked
// rows by workgroups of their own, which leave float32 sums, [tile - whole][part][rows of a tile], for
// a second kernel to join in order.  whole = 0: every tile.

struct Cut {
  int slots, whole, cut, parts;  // cut: tiles in parts
  // The order of the workgroups.  Tile by tile where each of the 8 XCDs, which take workgroups in
  // turn, then walks its own part of the rows; else part by part, so that those which walk the same
  // rows run together.  Tile by tile and part by part: 4 parts (7,813 tokens, 12 / 4 heads of 64,
  // forward and backward) 360 and 375 us, 16 (8 single tokens, 30,000 keys each, 16 / 4 heads of 128)
  // 87 and 90; 23 (300 queries, 12,000 keys, 4 heads of 64) 21.0 and 18.0, 6 (800 tokens, 8 heads of
  // 64, forward and backward) 45.0 and 42.4.
  bool by_tile;
};

// At 128 channels in 16 bits a half-empty last round runs at a higher clock, and parts must gain more
// than elsewhere.  16 heads of 128, bf16: 6,100 tokens, 128 of 384 tiles in 2 parts: 329 -> 304 us, 7,000
// tokens, 192 of 448 in 4: 395 -> 413; as large last rounds elsewhere, forward and backward: float32,
// 3,500 tokens, 16 heads of 64: 2.09 -> 1.91 ms, bf16, 10,500 tokens, 16 heads of 64: 2.28 -> 2.18 ms.
constexpr double kGain = 0.8, kGainAt128 = 0.65;

struct Share {
  int head, slot;
  int part;   // -1: the whole tile
  int place;  // of a part's sums
};

// Kernels for no tile, every tile and the last tiles in parts: a kernel with one way to its end needs
// fewer scalar registers.
constexpr int kNoCut = 0, kCutAll = 1, kCutLast = 2;

// (A division runs on the vector units: without this the addresses that follow from it would stay in
// vector registers.)
__device__ __forceinline__ int first_lane(uint32_t v) { return __builtin_amdgcn_readfirstlane((int)v); }

template <int CUT> __device__ __forceinline__ Share share_of(const Cut& c, uint32_t block) {
  if constexpr (CUT == kNoCut) return Share{(int)blockIdx.y, (int)blockIdx.x, -1, 0};
  const uint32_t whole = CUT == kCutAll ? 0u : (uint32_t)c.whole;
  uint32_t id = block;
  Share s{0, 0, -1, 0};
  if (CUT == kCutAll || block >= whole) {
    const uint32_t b = block - whole;
    const uint32_t d = c.by_tile ? c.parts : c.cut, t = first_lane(b / d), u = b - t * d;
    const uint32_t i = c.by_tile ? t : u;
    s.part = (int)(c.by_tile ? u : t);
    s.place = (int)(i * c.parts) + s.part;
    id = whole + i;
  }
  s.head = first_lane(id / (uint32_t)c.slots);
  s.slot = (int)(id - (uint32_t)s.head * c.slots);
  return s;
}

// Of the i-th tile in parts: its head and slot, and the place of its first part.
__device__ __forceinline__ Share tile_share(const Cut& c, int i) {
  const int id = c.whole + i, head = id / c.slots;
  return Share{head, id - head * c.slots, 0, i * c.parts};
}

// Part `part` of `steps` steps: its first, and how many (perhaps none).
__device__ __forceinline__ int part_steps(const Cut& c, int part, int* steps) {
  if (part < 0) return 0;
  const int share = (*steps + c.parts - 1) / c.parts, first = min(*steps, share * part);
  *steps = min(share, *steps - first);
  return first;
}

// Host.  `slots` * `kv_heads` tiles (`spare` of them perhaps empty) of on average `walked` rows, of which
// a part keeps at least `least`; `resident` workgroups fill the machine, `few` are wanted when there
// are less.  parts = 1: nothing to cut.  The last tiles, whole and in parts, bf16: 4,500 tokens, 16 heads
// of 128, 288 tiles: 240 and 174 us, with the backward pass 1,040 and 738; 24,576 tokens, 1,552 tiles:
// 2.35 and 2.23 ms; 9,000 tokens, 12 heads of 64, with the backward pass: 1,370 and 1,150 us; float32,
// 5,000 tokens, 8 heads of 64, with it: 2.95 and 1.91 ms.
inline Cut plan_cut(int64_t slots, int kv_heads, int64_t spare, int64_t walked, int least, int64_t resident, int64_t few,
                    double gain) {
  const int64_t tiles = slots * kv_heads;
  Cut c{(int)slots, (int)tiles, 0, 1, false};
  const int64_t most = walked / least;
  if (tiles < resident) {
    const int64_t want = few / tiles < most ? few / tiles : most;
    if (want >= 2) c = Cut{(int)slots, 0, (int)tiles, (int)want, want % 8 == 0 || 8 % want == 0};
    return c;
  }
  // The tiles past the last full round, in the number of parts whose rounds take least of a tile's
  // time, if that is less than `gain` of it and empty slots do not blur where a round ends.
  const int64_t rest = tiles % resident;
  if (rest == 0 || spare * 4 > resident || walked < 2048) return c;
  double best = gain;
  for (int64_t parts = 2; parts <= 16 && parts <= most; ++parts) {
    const double t = (double)((rest * parts + resident - 1) / resident) / parts + 0.01 * parts;
    if (t < best) {
      best = t;
      c = Cut{(int)slots, (int)(tiles - rest), (int)rest, (int)parts, parts % 8 == 0 || 8 % parts == 0};
    }
  }
  return c;
}

inline int64_t cut_places(const Cut& c) { return (int64_t)c.cut * c.parts; }
inline int64_t cut_blocks(const Cut& c) { return c.whole + cut_places(c); }

// ------------------------------------------------------------------------ tiles in LDS
//
// A tile is R rows of DP channels, row-major in 16-byte chunks, chunk c of row r at position
// c ^ swizzle(r).  LDS serves 256 bytes a clock, 16 lanes of a 16-byte read and 32 of an 8-byte
// transposing read: the former sit on 16 consecutive rows at one chunk, the latter on 4 rows of
// 64 bytes, and the swizzle puts either on 64 different banks.  Measured on this card with 8
// waves: 254 and 229 bytes a clock and compute unit at 128 channels, against 127 and 63 with the
// plain c ^ (r & 7).

//
// The kernels come for DC = 32, 64, 96 and 128 computed channels; tiles are DP = 64 or 128 wide
// (the channels past head_dim read zeros), and what a narrow head need not compute it skips.

constexpr int tile_width(int dc) { return dc <= 64 ? 64 : 128; }

template <DT D, int DP> constexpr int kRowChunks = DP * Elem<D>::kSize / 16;
template <DT D, int DP> constexpr int kRowBytes = DP * Elem<D>::kSize;

template <DT D, int DP> __device__ __forceinline__ int swizzle(int r) {
  // (float32: row r + 4 on the other 128 bytes)
  if constexpr (D == DT::F32) return ((r >> 2) & 1) << 3 | (r & 3) << 1 | ((r >> 3) & 1);
  else if constexpr (DP == 128) return (r & 3) << 2 | ((r >> 2) & 3);
  else return ((r >> 1) & 1) << 2 | ((r >> 2) & 3);  // (two rows in 256 bytes)
}

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) u32x4_t lds_u32x4_t;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
typedef __attribute__((address_space(3))) float lds_float_t;

// A lane's LDS addresses for the two ways to read tiles: rows of tiles that start at `row_base`
// and transposed columns of tiles that start at `col_base`, plus a constant for the tile and its
// rows r0 (swizzles repeat every 16 rows), which goes into the instruction while it is below 64 KB.
template <DT D, int DP> struct TileReader {
  static constexpr int kPer = Elem<D>::kSize / 2;  // chunks of 8 values
  uint32_t row[DP / 16 * kPer];
  uint32_t col[D == DT::F32 ? 16 : DP / 16];

  __device__ __forceinline__ TileReader(int lane, uint32_t row_base, uint32_t col_base) {
    const int r = lane & 31;
#pragma unroll
    for (int i = 0; i < DP / 16 * kPer; ++i) {
      const int c = (i / kPer * 2 + (lane >> 5)) * kPer + i % kPer;
      row[i] = row_base + r * kRowBytes<D, DP> + ((c ^ swizzle<D, DP>(r)) << 4);
    }
    if constexpr (D == DT::F32) {  // col[2 j + db % 2]: element j of channel block db
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = i >> 1, cc = (i & 1) * 32 + (lane & 31);
        const int rr = 8 * (j >> 2) + 4 * (lane >> 5) + (j & 3);
        col[i] = col_base + rr * kRowBytes<D, DP> + (((cc >> 2) ^ swizzle<D, DP>(rr)) << 4) + ((cc & 3) << 2);
      }
    } else {
      const int t = lane & 15;
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) {
        const int cc = i / 2 * 32 + ((lane >> 4) & 1) * 16 + (t & 3) * 4;
        const int rr = 8 * (i % 2) + 4 * (lane >> 5) + (t >> 2);
        col[i] = col_base + rr * kRowBytes<D, DP> + (((cc >> 3) ^ swizzle<D, DP>(rr)) << 4) + ((cc & 7) << 1);
      }
    }
  }

  // A operand of step kk (channels 16 kk .. 16 kk + 15) over tile rows r0 .. r0 + 31.
  __device__ __forceinline__ Frag<D> row_frag(int tile, int r0, int kk) const {
    Frag<D> f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const u32x4_t w = *(const lds_u32x4_t*)(uintptr_t)(row[kk * kPer + i] + (tile + r0 * kRowBytes<D, DP>));
      f.v[i] = make_uint4(w.x, w.y, w.z, w.w);
    }
    return f;
  }

  // A operand of the transposed tile: row = channel 32 db + lane % 32, contraction over tile rows
  // r0 + 8 (j / 4) + 4 (lane / 32) + j % 4 (r0 a multiple of 16), the order of to_frag.
  __device__ __forceinline__ Frag<D> column_frag(int tile, int r0, int db) const {
    Frag<D> f;
    if constexpr (D == DT::F32) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[j] = *(const lds_float_t*)(uintptr_t)(col[2 * j + db % 2] + (tile + r0 * kRowBytes<D, DP> + db / 2 * 256));
      f.v[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
      f.v[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
    } else {
      // The transposing read: 16 lanes hand in 4 rows of 16 channels (lane t: row t / 4, channels
      // 4 (t % 4) .. + 3) and lane t gets channel t of the 4 rows.
      uint2 half[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        half[i] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                (lds_s16x4_t*)(uintptr_t)(col[db * 2 + i] + (tile + r0 * kRowBytes<D, DP>))));
      f.v[0] = make_uint4(half[0].x, half[0].y, half[1].x, half[1].y);
    }
    return f;
  }
};

// Direct global-to-LDS loads of a tile of R rows by W waves: 1 KB an instruction, kLoads<..> of
// them a wave and tile, always that many (rows past the end and channels past head_dim read
// zeros), so that a wave can wait for a tile by counting.
template <DT D, int DP, int R, int W> constexpr int kLoads = R * kRowBytes<D, DP> / 1024 / W;

template <DT D, int DP, int R, int W> struct TileLoader {
  static constexpr int N = kLoads<D, DP, R, W>;
  static_assert(N >= 1 && N * W * 1024 == R * kRowBytes<D, DP>, "whole instructions");
  static constexpr int C = kRowChunks<D, DP>;
  static constexpr int kRowsPer = 64 / C;  // rows of an instruction
  uint32_t offset[N];  // of this lane, from the tile's first token
  int wave, lane;

  __device__ __forceinline__ int row(int n) const { return (n * W + wave) * kRowsPer + lane / C; }

  // Tiles of packed rows, `group` a token, that start `rem` rows into a token; keys: group 1.
  // magic: 65536 / group + 1 (exact for the r + rem < 2 * 128 + 32 that occur with group <= 128).
  __device__ __forceinline__ void place(const Heads<D>& t, int head_dim, int group, int rem, int magic) {
    constexpr int size = Elem<D>::kSize;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int r = row(n);
      const int c = (lane % C) ^ swizzle<D, DP>(r);
      const int tok = group == 1 ? r : ((r + rem) * magic) >> 16;
      const int h = group == 1 ? 0 : r + rem - tok * group;
      offset[n] = c * 16 < head_dim * size ? (uint32_t)((tok * (int)t.row + h * (int)t.head) * size + c * 16) : kOutOfRange;
    }
  }
  // `first`: the tile's first token; `left`: rows from the tile's first to the last there is (any
  // value; <= 0 reads nothing); `lds`: where the tile goes.
  __device__ __forceinline__ void load(const typename Elem<D>::T* first, int left, uint32_t lds) const {
    const i32x4_t rsrc = make_rsrc(first, kOutOfRange);
    lds = __builtin_amdgcn_readfirstlane(lds + wave * 1024);
    if (left >= R) {
#pragma unroll
      for (int n = 0; n < N; ++n) lds_dma16(rsrc, offset[n], lds + n * W * 1024);
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) lds_dma16(rsrc, row(n) < left ? offset[n] : kOutOfRange, lds + n * W * 1024);
    }
  }
};

// A lane's own row as the B operand of step kk, straight from global memory.
template <DT D>
__device__ __forceinline__ Frag<D> own_frag(const typename Elem<D>::T* row, bool there, int kk, int head_dim, int lane) {
  constexpr int kPer = Elem<D>::kSize / 2;
  constexpr int kVals = 16 / Elem<D>::kSize;
  Frag<D> f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = (kk * 2 + (lane >> 5)) * kPer + i;
    f.v[i] = there && c * kVals < head_dim ? *reinterpret_cast<const uint4*>(row + c * kVals) : make_uint4(0, 0, 0, 0);
  }
  return f;
}

// Four consecutive channels of an own row, rounded once.
template <DT D> __device__ __forceinline__ void store4(typename Elem<D>::T* p, float a, float b, float c, float d) {
  if constexpr (D == DT::F32) *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
  else *reinterpret_cast<uint2*>(p) = pack4<D>(a, b, c, d);
}

// Accumulator tiles [DC / 32] (row = channel, column = own row) to the row, times `f`.
template <DT D, int DC>
__device__ __forceinline__ void store_row(typename Elem<D>::T* row, const f32x16_t (&acc)[DC / 32], float f, int head_dim,
                                          int lane) {
#pragma unroll
  for (int db = 0; db < DC / 32; ++db)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int c = db * 32 + 8 * a + 4 * (lane >> 5);
      if (c < head_dim)
        store4<D>(row + c, acc[db][4 * a] * f, acc[db][4 * a + 1] * f, acc[db][4 * a + 2] * f, acc[db][4 * a + 3] * f);
    }
}

// Accumulators through LDS between the waves that hold the same own rows: the values of a lane 256
// bytes apart, so that a wave's accesses are contiguous.  `at`: this wave's area, DC / 32 * 4 KB.
template <int DC> __device__ __forceinline__ void put_acc(uint32_t at, const f32x16_t (&acc)[DC / 32], int lane) {
#pragma unroll
  for (int db = 0; db < DC / 32; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) *(lds_float_t*)(uintptr_t)(at + (db * 16 + i) * 256 + lane * 4) = acc[db][i];
}
template <int DC>
__device__ __forceinline__ void add_acc(uint32_t at, f32x16_t (&acc)[DC / 32], float mine, float theirs, int lane) {
#pragma unroll
  for (int db = 0; db < DC / 32; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float v = *(const lds_float_t*)(uintptr_t)(at + (db * 16 + i) * 256 + lane * 4);
      acc[db][i] = fmaf(v, theirs, acc[db][i] * mine);
    }
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Host: the checks that the forward and backward entry points share (attention.hip).
struct AttentionShape {
  int64_t nq, nk;
  const int64_t *q_offsets, *k_offsets;
  int items, heads, kv_heads, head_dim, dtype;
  float scale;
};
Status check_attention(const AttentionShape& s);
Status check_heads(const subm_heads_t* t, int64_t rows, int heads, const AttentionShape& s, bool written, const char* what);
Status check_forward(const subm_heads_t* q, const subm_heads_t* k, const subm_heads_t* v, const subm_heads_t* out,
                     const float* lse, const AttentionShape& s);
// (attention_backward.hip)
Status check_backward(const subm_heads_t* dout, const subm_heads_t* q, const subm_heads_t* k, const subm_heads_t* v,
                      const subm_heads_t* out, const float* lse, const subm_heads_t* dq, const subm_heads_t* dk,
                      const subm_heads_t* dv, const AttentionShape& s);

}  // namespace submconv
