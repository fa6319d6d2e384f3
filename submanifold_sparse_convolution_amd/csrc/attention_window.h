// What a row of a sliding window sees, and the tiles of keys or rows that this leaves.
//
// Query i of an item with nq queries and nk keys stands at key position p = i + nk - nq and sees key j if
// j <= p + right and (j >= p - left or j < sinks).  Both ends of the range rise with i, so those of a block
// of rows are its first row's first and its last row's last key.
#pragma once

#include "attention_common.h"
#include "row_lanes.h"

namespace submconv {

struct Window {
  int64_t left, right;  // at most kOpen, which is more than there are keys
  int sinks;
  const int64_t* k_lengths;  // keys of each item that are there, or null: all its rows
  bool runs;                 // most tiles walk as many keys: runs of them to each XCD (window_share)

  // How many keys an item with `rows` rows of keys has.
  __device__ __forceinline__ int keys(int item, int rows) const {
    if (k_lengths == nullptr) return rows;
    const int64_t n = k_lengths[item];
    return n < 0 ? 0 : n < rows ? (int)n : rows;
  }
  // Of position p: the first key (0 if the sinks reach it) and the last, -1 if there is none.
  __device__ __forceinline__ void range(int64_t p, int nk, int* lo, int* hi) const {
    const int64_t first = p - left, last = p + right;
    *lo = first <= sinks ? 0 : (int)(first < nk ? first : nk);
    *hi = last < 0 ? -1 : last < nk ? (int)last : nk - 1;
  }
  __device__ __forceinline__ bool sees(int64_t p, int j) const {
    return j <= p + right && (j >= p - left || j < sinks);
  }
  // The packed rows (`group` a token) that see key j of an item: *from .. *to - 1.
  __device__ __forceinline__ void rows(int j, bool sink, int nq, int shift, int group, int* from, int* to) const {
    const int64_t first = (int64_t)j - right - shift, past = (int64_t)j + left - shift + 1;
    *from = (int)(first < 0 ? 0 : first < nq ? first : nq) * group;
    *to = (sink ? nq : (int)(past < 0 ? 0 : past < nq ? past : nq)) * group;
  }
  // Host: keys of an item of `keys` that a block of `rows` tokens walks, at most.
  int64_t walked(int64_t keys, int64_t rows) const {
    const int64_t most = left + right + sinks + rows;
    return most < keys ? most : keys;
  }
  // Host: whether most tiles of items of `keys` walk the same number of keys, and heads are not grouped.
  bool in_runs(int64_t keys, int group) const { return group == 1 && (left + right) * 2 < keys; }
};

// ------------------------------------------------------------------ the item of a tile
//
// A workgroup of a window has little to do, and a chain of dependent loads before it (a search through the
// offsets, then the item's) is a good part of its time.  A wave therefore looks at 64 items at once, with
// everything of the item in flight at the same time.

struct Item {
  int index, tile;
  int64_t q0, k0;
  int nq, nk;
};

__device__ __forceinline__ int64_t lane_value64(int64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, lane), hi = __builtin_amdgcn_readlane((uint32_t)(v >> 32), lane);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// find_item and item_rows of slot `slot` in the tiling of the queries by `block` packed rows, in one; every lane of
// the wave calls it.
template <typename Args>
__device__ __forceinline__ Item find_rows(const Args& a, const Window& w, int group, int block, int64_t slot) {
  const int lane = threadIdx.x & 63;
  const auto start = [&](int64_t o, int b) { return (o < 0 ? 0 : o > a.nq ? a.nq : o) * group / block + b; };
  int first = 0, count = a.items;  // the item is one of first .. first + count - 1
  while (count > 64) {
    const int stride = (count + 63) / 64, at = lane * stride;
    const bool before = at < count && start(a.q_offsets[first + min(at, count - 1)], first + at) <= slot;
    const int n = max(1, (int)__popcll(__builtin_amdgcn_ballot_w64(before)));
    first += (n - 1) * stride;
    count = min(stride, count - (n - 1) * stride);
  }
  const int mine = first + min(lane, count - 1);
  const int64_t q_from = a.q_offsets[mine], q_to = a.q_offsets[mine + 1], k_from = a.k_offsets[mine], k_to = a.k_offsets[mine + 1];
  const int64_t there = w.k_lengths != nullptr ? w.k_lengths[mine] : INT64_MAX;
  const int64_t at = start(q_from, mine);
  const int n = max(1, (int)__popcll(__builtin_amdgcn_ballot_w64(lane < count && at <= slot)));
  const auto rows = [&](int64_t from, int64_t to, int64_t most, int64_t* first_row, int* number) {
    const int64_t s = lane_value64(from, n - 1), e = lane_value64(to, n - 1);
    *first_row = s < 0 ? 0 : s > most ? most : s;
    *number = (int)((e < *first_row ? *first_row : e > most ? most : e) - *first_row);
  };
  Item item;
  item.index = first + n - 1;
  const int64_t t = slot - lane_value64(at, n - 1);
  item.tile = t < 0 ? INT32_MAX / block : (int)t;  // (only for offsets that do not rise: no such rows)
  rows(q_from, q_to, a.nq, &item.q0, &item.nq);
  rows(k_from, k_to, a.nk, &item.k0, &item.nk);
  const int64_t most = lane_value64(there, n - 1);
  item.nk = most < 0 ? 0 : most < item.nk ? (int)most : item.nk;
  return item;
}

// Host: plan_cut for windows: all tiles in parts, or none (the last ones alone are never cut).  `resident`: workgroups
// that the machine holds.  Where most of an item is seen the longest tile takes twice the mean, and few tiles
// leave compute units that wait for it: then in at least four parts (three and six, which the XCDs do not share
// evenly, measured up to 30 % slower).  16,384 tokens, 8 / 2 heads of 128, causal, backward: 3.48 -> 1.81 ms; 9,000
// tokens, 6 heads of 64, forward 153 -> 120 us, backward 422 -> 384; with more tiles two share a unit, and
// the one left alone speeds up: 8,000 tokens, 8 heads of 128, forward 217 us whole and 231 in parts.
inline Cut plan_window_cut(const Window& w, int64_t slots, int kv_heads, int64_t keys, int64_t walked, int least,
                           int64_t resident, int64_t few) {
  constexpr int kUneven = 4;
  const int64_t tiles = slots * kv_heads;
  const bool uneven = (w.left + w.right) * 4 >= keys * 3;
  if (uneven && tiles * 4 <= resident * 3 && few < tiles * kUneven) few = tiles * kUneven;
  return plan_cut(slots, kv_heads, 0, walked, least, INT32_MAX, few, kGain);
}

// The workgroup's tile (or part of one).  Neighbouring tiles of a window walk nearly the same keys, while the XCDs
// take workgroups in turn and each has its own L2: every XCD gets a run of consecutive tiles, so that what
// one loads the next finds there (24,576 tokens, 16 heads of 128, 2,048 keys: 493 -> 437 us).  Not with grouped
// heads, whose tiles are that many times fewer tokens apart as it is (16,384 tokens, 8 / 2 heads: 150 us, 176 in
// runs).  Where tiles differ in length (an open end) each head's go from the last rows' on (`last_first`: an item's
// last rows walk the most keys, and those the same from the start on; 16,384 tokens, 8 / 2 heads of 128, causal:
// 673 -> 526 us); heads follow one another, and items from the last one on, whatever their lengths.
template <int CUT> __device__ __forceinline__ Share window_share(const Cut& c, const Window& w, bool last_first) {
  Share s = share_of<CUT>(c, blockIdx.x);
  if constexpr (CUT != kNoCut) return s;
  if (w.runs) {
    constexpr uint32_t kXcds = 8;
    const uint32_t block = blockIdx.x + gridDim.x * blockIdx.y, all = gridDim.x * gridDim.y;
    const uint32_t xcd = block % kXcds, each = all / kXcds, more = all % kXcds;
    const uint32_t id = xcd * each + min(xcd, more) + block / kXcds;
    s.head = first_lane(id / (uint32_t)c.slots);
    s.slot = (int)(id - (uint32_t)s.head * c.slots);
  } else if (last_first) {
    s.slot = c.slots - 1 - s.slot;
  }
  return s;
}

constexpr int64_t kOpen = int64_t(1) << 31;  // a window's end that no position reaches
constexpr int kMaxSinks = 128;

// Host (window_attention.hip).
Status check_window(int64_t left, int64_t right, int sinks, const int64_t* k_lengths, Window* w);

// The tiles of KEYS keys that a block of rows walks: the sinks, if the window does not reach them, and the
// window from its first key on.
template <int KEYS> struct KeyTiles {
  int sink_tiles, sink_end;  // keys 0 .. sink_end - 1
  int low, high;             // keys low .. high - 1
  int first, tiles;          // tiles first .. first + tiles - 1 of them all are this workgroup's

  __device__ __forceinline__ void place(const Window& w, int nk, int shift, int first_token, int last_token) {
    int unused, hi;
    w.range((int64_t)first_token + shift, nk, &low, &unused);
    w.range((int64_t)last_token + shift, nk, &unused, &hi);
    low = first_lane(low);  // (its token comes from a division)
    high = first_lane(hi) + 1;
    sink_end = low == 0 ? 0 : min(w.sinks, high);
    sink_tiles = (sink_end + KEYS - 1) / KEYS;
    first = 0;
    tiles = sink_tiles + max(0, (high - low + KEYS - 1) / KEYS);
  }
  __device__ __forceinline__ void cut(int from, int count) {
    first = from;
    tiles = count;
  }
  // Of tile t: its first key, and where its keys end (0 past the last tile).
  __device__ __forceinline__ int key(int t) const {
    t += first;
    return t < sink_tiles ? t * KEYS : low + (t - sink_tiles) * KEYS;
  }
  __device__ __forceinline__ int end(int t) const { return t >= tiles ? 0 : t + first < sink_tiles ? sink_end : high; }
};

// What a lane's own query row sees, and what all rows of its wave do.
struct RowView {
  int lo, hi, sinks;
  uint32_t span;         // the row sees lo .. lo + span (and the sinks)
  int wave_lo, wave_hi;  // every row of the wave sees these and what lies between (and the sinks up to wave_hi)
  int wave_low, wave_high;  // some row of the wave sees these, and none sees any before (but sinks) or after

  __device__ __forceinline__ void place(const Window& w, int nk, int shift, int token, int first_token, int last_token) {
    w.range((int64_t)token + shift, nk, &lo, &hi);
    w.range((int64_t)first_token + shift, nk, &wave_low, &wave_hi);
    w.range((int64_t)last_token + shift, nk, &wave_lo, &wave_high);
    wave_lo = first_lane(wave_lo);
    wave_hi = first_lane(wave_hi);
    wave_low = first_lane(wave_low);
    wave_high = first_lane(wave_high);
    sinks = w.sinks;
    if (hi < lo) lo = INT32_MAX;  // (sees no more than sinks)
    span = hi < lo ? 0u : (uint32_t)(hi - lo);
  }
  // Keys key .. key + n - 1, of which those from `end` on are not there.
  __device__ __forceinline__ bool sees_all(int key, int n, int end) const {
    return key + n <= end && key + n - 1 <= wave_hi && (key >= wave_lo || key + n <= sinks);
  }
  __device__ __forceinline__ bool sees_any(int key, int n, int end) const {
    return key < end && key <= wave_high && (key + n > wave_low || key < sinks);
  }
  // Calls hide(kb, i) for element i of each 32 keys' scores that the row does not see.
  template <int KB, typename Hide>
  __device__ __forceinline__ void mask(int key, int end, int lane, const Hide& hide) const {
    const int first = key + 4 * (lane >> 5);
    if (key < sinks || end <= key) {  // (a part's tiles may end before the window does)
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = first + kb * 32 + 8 * (i >> 2) + (i & 3);
          if (!(j < end && j <= hi && (j >= lo || j < sinks))) hide(kb, i);
        }
    } else {
      const uint32_t from = (uint32_t)first - (uint32_t)lo;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (from + (uint32_t)(kb * 32 + 8 * (i >> 2) + (i & 3)) > span) hide(kb, i);
    }
  }
};

// Which packed rows a lane's own key is seen by, and which all keys of its wave are.
struct KeyView {
  int from;
  uint32_t span;  // the key is seen by rows from .. from + span - 1
  int wave_from, wave_to;    // every key of the wave is seen by rows wave_from .. wave_to - 1,
  int wave_first, wave_end;  // some key by these and none by others

  __device__ __forceinline__ void place(const Window& w, bool sink, int nq, int shift, int group, int key, int first_key,
                                        int last_key) {
    int to;
    w.rows(key, sink, nq, shift, group, &from, &to);
    w.rows(first_key, sink, nq, shift, group, &wave_first, &wave_to);
    w.rows(last_key, sink, nq, shift, group, &wave_from, &wave_end);
    wave_from = first_lane(wave_from);
    wave_to = first_lane(wave_to);
    wave_first = first_lane(wave_first);
    wave_end = first_lane(wave_end);
    span = to > from ? (uint32_t)(to - from) : 0u;
  }
  __device__ __forceinline__ bool sees_all(int row, int n) const { return row >= wave_from && row + n <= wave_to; }
  __device__ __forceinline__ bool sees_any(int row, int n) const { return row < wave_end && row + n > wave_first; }
  // Calls hide(i) for element i of 32 rows' values that the key is not seen by.
  template <typename Hide> __device__ __forceinline__ void mask(int row, int lane, const Hide& hide) const {
    const uint32_t at = (uint32_t)(row + 4 * (lane >> 5)) - (uint32_t)from;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (at + (uint32_t)(8 * (i >> 2) + (i & 3)) >= span) hide(i);
  }
};

// ------------------------------------------------------------------ rows that are not finite
//
// A matrix product adds 0 times a hidden key's value, which is NaN where the value is not finite.  A row
// that ends so is computed again over what it sees alone, a wave a row, two channels a lane; but only if
// something hidden is not finite, and only until each of its channels that came out so is again: where inputs are
// full of NaN (a training run that has diverged) nearly every row ends so, and each walking all that it sees would
// take a thousand times as long as the products (8,192 tokens, 8 heads of 128, causal, backward: 0.8 ms finite, 3
// all NaN, 76 with one infinity in dout, beside which 128 keys are computed again).

// The kernel's arguments, read again: what only this rare work needs of them is not kept in registers.
template <typename A> __device__ __forceinline__ A fresh_args() {
  static_assert(sizeof(A) % 4 == 0, "whole words");
  uint64_t p = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  const auto* words = (const __attribute__((address_space(4))) uint32_t*)p;
  struct Words { uint32_t w[sizeof(A) / 4]; } all;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(A) / 4); ++i) all.w[i] = words[i];
  return __builtin_bit_cast(A, all);
}

// The lane's number, from nothing that has to be kept.
__device__ __forceinline__ int fresh_lane() {
  int m = -1;
  asm volatile("" : "+s"(m));
  return __builtin_amdgcn_mbcnt_hi(m, __builtin_amdgcn_mbcnt_lo(m, 0u));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

// The own rows (bits 0 .. 31) with a value that is not finite, of those that `may` be computed again.
template <int DC> __device__ __forceinline__ uint64_t odd_rows(const f32x16_t (&acc)[DC / 32], bool may) {
  float z = 0.f;
#pragma unroll
  for (int db = 0; db < DC / 32; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) z = fmaf(acc[db][i], 0.f, z);
  const uint64_t odd = __builtin_amdgcn_ballot_w64(may && !(z == 0.f));
  return (odd | odd >> 32) & 0xffffffffu;
}

template <DT D> __device__ __forceinline__ float2 row_pair(const typename Elem<D>::T* row, int head_dim, int lane) {
  if (2 * lane >= head_dim) return make_float2(0.f, 0.f);
  return make_float2(to_float<D>(row[2 * lane]), to_float<D>(row[2 * lane + 1]));
}
__device__ __forceinline__ float pair_dot(float2 x, float2 y) { return lanes_sum<64>(fmaf(x.x, y.x, x.y * y.y)); }
__device__ __forceinline__ void add_scaled(float2& o, float p, float2 x) { o = make_float2(fmaf(p, x.x, o.x), fmaf(p, x.y, o.y)); }

// A value that is not finite makes z NaN.
template <DT D> __device__ __forceinline__ void add_odd(float& z, const typename Elem<D>::T* row, int head_dim, int lane) {
  const float2 x = row_pair<D>(row, head_dim, lane);
  z = fmaf(x.x, 0.f, fmaf(x.y, 0.f, z));
}
// Whether a row of `rows` for the keys that position p does not see of those that a tile walks is not finite.
template <DT D, int KEYS>
__device__ __forceinline__ bool hidden_odd(const Window& w, const KeyTiles<KEYS>& walk, int64_t p, int nk,
                                           const typename Elem<D>::T* rows, int64_t stride, int head_dim, int lane) {
  int lo, hi;
  w.range(p, nk, &lo, &hi);
  float z = 0.f;
  const auto look = [&](int from, int to) {
#pragma unroll 1
    for (int j = from; j < to; ++j)
      if (!w.sees(p, j)) add_odd<D>(z, rows + j * stride, head_dim, lane);
  };
  look(walk.low, min(lo, walk.high));
  look(max(hi + 1, walk.low), walk.high);
  return __builtin_amdgcn_ballot_w64(!(z == 0.f)) != 0;
}

// A row of the accumulators of the lanes l and l + 32, two channels a lane.
template <int DC> __device__ __forceinline__ float2 take_row(const f32x16_t (&acc)[DC / 32], int l, int head_dim, int lane) {
  float2 o = make_float2(0.f, 0.f);
  asm volatile("" : "+v"(lane));  // (or the comparisons below are kept in registers over the rows)
#pragma unroll
  for (int db = 0; db < DC / 32; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int at = (db * 32 + 8 * (i >> 2) + (i & 3)) / 2;  // (and 2 lanes on, the upper half's)
      const float v = __shfl(acc[db][i], l + (lane == at ? 0 : 32), 64);
      if ((lane == at || lane == at + 2) && 2 * lane < head_dim) (i % 2 ? o.y : o.x) = v;
      __builtin_amdgcn_sched_barrier(0);
    }
  return o;
}
// Of a row that came out as `was`: whether a channel that was not finite still is.
__device__ __forceinline__ bool still_finite(float2 was, float2 o) {
  return __builtin_amdgcn_ballot_w64((!__builtin_isfinite(was.x) && __builtin_isfinite(o.x)) ||
                                     (!__builtin_isfinite(was.y) && __builtin_isfinite(o.y))) != 0;
}
__device__ __forceinline__ float2 mended(float2 was, float2 o) {
  return make_float2(__builtin_isfinite(was.x) ? was.x : o.x, __builtin_isfinite(was.y) ? was.y : o.y);
}

// A row in that form into the accumulators of the lanes l and l + 32.
template <int DC> __device__ __forceinline__ void put_row(f32x16_t (&acc)[DC / 32], float2 o, int l, int lane) {
  asm volatile("" : "+v"(lane));
#pragma unroll
  for (int db = 0; db < DC / 32; ++db)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int c = db * 32 + 8 * (i >> 2) + (i & 3);  // (and c + 4 in the upper half)
      const float v = __shfl(c % 2 ? o.y : o.x, c / 2 + 2 * (lane >> 5), 64);
      if ((lane & 31) == l) acc[db][i] = v;
      __builtin_amdgcn_sched_barrier(0);  // (one after the other: together they would need 64 registers more)
    }
}

}  // namespace submconv
