// Embedding lookup with a scale and its gradient (include/sparse_transformer.h).
//
//   out_i = c T[token_i],   dT_t = c sum_{i: token_i = t} dout_i
//
// Both are bound by HBM (no element is used twice, but those of rows that several tokens name), small
// calls by their launches.
//
// The gradient goes by the tokens in sorted order, ties by position, so every sum has one order and no
// atomics on values: (1) long lists are first split stably into buckets of consecutive table rows; (2) a
// workgroup a bucket sorts its tokens by counting, stores where each row's begin, and zeros the rows without
// any (a table of at most 1,024 rows has a bucket a row, and nothing is left to sort); (3) pieces of
// consecutive sorted positions, the same work for all whatever the tokens' frequencies, sum their rows of
// dout: a row of a few tokens is summed where it begins, one of more in several pieces leaves float32 sums a piece,
// (4) which are joined in order.
//
// Measured, gradient of 135,826 tokens, 1,024 channels, bf16, on the device: table of 65,536 rows, tokens evenly
// spread: 5 + 12 + 15 + 84 + 5 us (382 MB in (3): 4.5 TB/s); a twelfth of them one token, half of the rows without
// any: 5 + 12 + 42 + 86 + 8 (the first bucket's list, a third of all, and 72 MB of zeros beside it); table of 100 rows: 5 + 10 +
// 50 + 6 (5.3 TB/s).  4,099 tokens, 1,021 rows of 675 channels, float32: 10 + 8 + 4, all of it latency.  Lookup of 450
// tokens, 768 channels, f16: 3 us.
#include <algorithm>
#include <cmath>

#include "chunk.h"
#include "device_common.h"
#include "internal.h"
#include "row_lanes.h"
#include "sparse_transformer.h"

namespace submconv {
namespace {

// The table row of token i, or `rows` for a token outside the table.
__device__ __forceinline__ int token_row(const void* tokens, int wide, int64_t i, int rows) {
  const int64_t t = wide ? static_cast<const int64_t*>(tokens)[i] : static_cast<const int32_t*>(tokens)[i];
  return t >= 0 && t < rows ? (int)t : rows;
}

template <DT D, bool TAIL>
__global__ __launch_bounds__(256) void embedding_forward_kernel(const typename Elem<D>::T* __restrict__ table, int rows, int channels,
                                                                const void* __restrict__ tokens, int wide, int64_t n, float scale,
                                                                typename Elem<D>::T* __restrict__ out, int lanes) {
  constexpr int V = kChunk<D>, kFlight = 4;
  const int lane = threadIdx.x & (lanes - 1), step = 256 / lanes, chunks = (channels + V - 1) / V;
  for (int64_t i = (int64_t)blockIdx.x * step + threadIdx.x / lanes; i < n; i += (int64_t)gridDim.x * step) {
    const int row = token_row(tokens, wide, i, rows);
    const typename Elem<D>::T* src = table + (int64_t)(row < rows ? row : 0) * channels;
    const float c = row < rows ? scale : 0.f;
    for (int k0 = lane; k0 < chunks; k0 += kFlight * lanes) {
      float v[kFlight][V];
#pragma unroll
      for (int k = 0; k < kFlight; ++k) load_chunk<D, TAIL>(src, (k0 + k * lanes) * V, channels, v[k]);
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[k][j] = row < rows ? v[k][j] * c : 0.f;  // (row 0 may hold anything)
        store_chunk<D, TAIL>(out + i * channels, (k0 + k * lanes) * V, channels, v[k]);
      }
    }
  }
}

// ------------------------------------------------------------------------------ sorted tokens

constexpr int kMaxBuckets = 1024;
constexpr int kMaxSpan = 2048;  // rows of a bucket: five counters each stay below 64 KB of LDS
constexpr int kMaxTiles = 256;
constexpr int kSplitThreads = 1024;

struct Sort {
  const void* tokens;
  int wide, rows;
  int64_t n;
  int span_bits, buckets;  // buckets of 2^span_bits rows
  int tiles;               // 0: no split
  int64_t tile;            // tokens of a tile
  int32_t* counts;         // [tiles][buckets]
  int32_t* bucket;         // [buckets + 1] where each bucket begins in the split list
  int2* split;             // [n] positions and rows by bucket
  int32_t *order, *row;    // [n] positions and rows in sorted order
  int32_t* start;          // [rows + 1] first sorted position of each row
  int32_t* joins;          // how many rows are to be joined (set to 0 here)
};

// Lanes of the wave whose `v` (of `bits` bits) is this lane's, of those that are `valid`.
__device__ __forceinline__ uint64_t peers_of(uint32_t v, bool valid, int bits) {
  uint64_t m = __ballot(valid);
  for (int b = 0; b < bits; ++b) {
    const uint64_t with = __ballot((v >> b) & 1u);
    m &= ((v >> b) & 1u) ? with : ~with;
  }
  return m;
}

// LDS written by other lanes of this wave has arrived (a wave's LDS accesses stay in order).
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ int wave_scan(int v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o, 64);
    if (lane >= o) v += u;
  }
  return v;
}

// Exclusive prefix sum of x[0 .. count) in LDS, in place, by a workgroup of WAVES waves; returns the sum of
// all.  Every thread calls it.
template <int WAVES> __device__ __forceinline__ int block_scan(int32_t* x, int count, int32_t* slots) {
  const int per = (count + WAVES * 64 - 1) / (WAVES * 64), lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int first = min(count, (int)threadIdx.x * per), end = min(count, first + per);
  int sum = 0;
  for (int i = first; i < end; ++i) sum += x[i];
  const int incl = wave_scan(sum, lane);
  if (lane == 63) slots[w] = incl;
  __syncthreads();
  int run = incl - sum, all = 0;
#pragma unroll
  for (int k = 0; k < WAVES; ++k) {
    if (k < w) run += slots[k];
    all += slots[k];
  }
  for (int i = first; i < end; ++i) {
    const int v = x[i];
    x[i] = run;
    run += v;
  }
  __syncthreads();
  return all;
}

// A wave walks its own part of a list in order, so that equal values keep their order; `run` [values] in
// LDS holds the next place of each value.  item(i) is {value or -1, what}; the next 64 are on their way.
template <typename Get, typename Put>
__device__ __forceinline__ void place_in_order(int64_t first, int64_t end, int bits, int32_t* run, const Get& get, const Put& put) {
  const int lane = threadIdx.x & 63;
  int2 next = first + lane < end ? get(first + lane) : make_int2(-1, 0);
  for (int64_t i0 = first; i0 < end; i0 += 64) {
    const int2 x = next;
    next = i0 + 64 + lane < end ? get(i0 + 64 + lane) : make_int2(-1, 0);
    const uint64_t peers = peers_of((uint32_t)x.x, x.x >= 0, bits);
    const int rank = __popcll(peers & ((1ull << lane) - 1ull));
    if (x.x >= 0) put(run[x.x] + rank, x.x, x.y);
    wave_fence();
    if (x.x >= 0 && rank == 0) run[x.x] += __popcll(peers);
    wave_fence();
  }
}

template <int WAVES> __device__ __forceinline__ void wave_part(int64_t first, int64_t end, int64_t* a, int64_t* b) {
  const int w = threadIdx.x >> 6;
  const int64_t per = ((end - first + WAVES - 1) / WAVES + 63) / 64 * 64;
  *a = min(end, first + per * w);
  *b = min(end, *a + per);
}

template <DT D> __device__ __forceinline__ void zero_row(typename Elem<D>::T* out, int channels) {  // by a wave
  constexpr int V = kChunk<D>;
  const float zero[V] = {};
  for (int c = (threadIdx.x & 63) * V; c < channels; c += 64 * V) store_chunk<D>(out, c, channels, zero);
}

// Tokens of each bucket in each tile.
__global__ __launch_bounds__(kSplitThreads) void embedding_count_kernel(Sort s) {
  __shared__ int32_t s_count[kMaxBuckets];
  for (int b = threadIdx.x; b < s.buckets; b += kSplitThreads) s_count[b] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * s.tile, end = min(s.n, first + s.tile);
#pragma unroll 4
  for (int64_t i = first + threadIdx.x; i < end; i += kSplitThreads) {
    const int row = token_row(s.tokens, s.wide, i, s.rows);
    if (row < s.rows) atomicAdd(&s_count[row >> s.span_bits], 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < s.buckets; b += kSplitThreads) s.counts[(int64_t)blockIdx.x * s.buckets + b] = s_count[b];
}

// The stable split into buckets: each tile sums the tiles' counts before it by itself (at most 256 of
// them: one launch less than a prefix sum of its own).  Buckets of one row are the sorted list.
template <DT D>
__global__ __launch_bounds__(kSplitThreads) void embedding_split_kernel(Sort s, typename Elem<D>::T* __restrict__ dtable, int channels) {
  constexpr int W = kSplitThreads / 64;
  __shared__ int32_t s_start[kMaxBuckets];  // the bucket's tokens, then where it begins
  __shared__ int32_t s_run[W][kMaxBuckets];
  __shared__ int32_t s_slots[W];
  for (int b = threadIdx.x; b < s.buckets; b += kSplitThreads) {
    int all = 0, before = 0;
#pragma unroll 16
    for (int t = 0; t < s.tiles; ++t) {
      const int c = s.counts[(int64_t)t * s.buckets + b];
      all += c;
      before += t < (int)blockIdx.x ? c : 0;
    }
    s_start[b] = all;
    s_run[0][b] = before;
#pragma unroll
    for (int w = 1; w < W; ++w) s_run[w][b] = 0;
  }
  __syncthreads();
  const int all = block_scan<W>(s_start, s.buckets, s_slots);
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const bool rows = s.span_bits == 0;  // (buckets are rows)
  if (blockIdx.x == 0) {
    int32_t* out = rows ? s.start : s.bucket;
    for (int b = threadIdx.x; b < s.buckets; b += kSplitThreads) out[b] = s_start[b];
    if (threadIdx.x == 0) {
      out[s.buckets] = all;
      *s.joins = 0;
    }
  }
  const int64_t first = blockIdx.x * s.tile, end = min(s.n, first + s.tile);
  int64_t a, b;
  wave_part<W>(first, end, &a, &b);
  if (w + 1 < W)  // what the next wave's places start behind
    for (int64_t i = a + lane; i < b; i += 64) {
      const int row = token_row(s.tokens, s.wide, i, s.rows);
      if (row < s.rows) atomicAdd(&s_run[w + 1][row >> s.span_bits], 1);
    }
  __syncthreads();
  for (int v = threadIdx.x; v < s.buckets; v += kSplitThreads) {
    int run = s_start[v];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      run += s_run[k][v];
      s_run[k][v] = run;
    }
  }
  __syncthreads();
  int bits = 0;
  while ((1 << bits) < s.buckets) ++bits;
  place_in_order(
      a, b, bits, s_run[w],
      [&](int64_t i) {
        const int row = token_row(s.tokens, s.wide, i, s.rows);
        // (the position in 31 bits is all that is kept of i; the row is read again where it is stored)
        return make_int2(row < s.rows ? row >> s.span_bits : -1, (int)i);
      },
      [&](int place, int v, int i) {
        if (rows) {
          s.order[place] = i;
          s.row[place] = v;
        } else {
          s.split[place] = make_int2(i, token_row(s.tokens, s.wide, i, s.rows));
        }
      });
  if (rows)
    for (int r = blockIdx.x * W + w; r < s.rows; r += s.tiles * W)
      if ((r + 1 < s.buckets ? s_start[r + 1] : all) == s_start[r]) zero_row<D>(dtable + (int64_t)r * channels, channels);
}

// One bucket: its tokens sorted by row, where each row's begin, zeros for the rows without any.
template <DT D, int W>
__global__ __launch_bounds__(W * 64) void embedding_sort_kernel(Sort s, typename Elem<D>::T* __restrict__ dtable, int channels) {
  extern __shared__ int32_t s_mem[];  // [W][span] places of the waves, [span] counts
  __shared__ int32_t s_slots[W], s_base;
  const int span = 1 << s.span_bits, row0 = (int)blockIdx.x << s.span_bits;
  const int here = min(span, s.rows - row0);  // rows of this bucket
  int32_t* s_count = s_mem + W * span;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int r = threadIdx.x; r < (W + 1) * span; r += W * 64) s_mem[r] = 0;
  // the bucket's list, and the sorted position it begins at (of a whole list: counted below)
  int64_t first = 0, end = s.n;
  if (s.tiles > 0) {
    first = s.bucket[blockIdx.x];
    end = s.bucket[blockIdx.x + 1];
  }
  if (threadIdx.x == 0) {
    s_base = s.tiles > 0 ? (int)first : 0;
    if (blockIdx.x == 0) *s.joins = 0;
  }
  __syncthreads();
  const auto get = [&](int64_t i) {  // {row in the bucket (others: below 0 or from `here` on), position}
    if (s.tiles > 0) {
      const int2 x = s.split[i];
      return make_int2(x.y - row0, x.x);
    }
    return make_int2(token_row(s.tokens, s.wide, i, s.rows) - row0, (int)i);
  };
  int64_t a, b;
  wave_part<W>(first, end, &a, &b);
  int less = 0;
#pragma unroll 4
  for (int64_t i = a + lane; i < b; i += 64) {
    const int r = get(i).x;
    less += r < 0 ? 1 : 0;
    if (r >= 0 && r < here) atomicAdd(&s_mem[w * span + r], 1);
  }
  if (s.tiles == 0) {
    less = wave_scan(less, lane);
    if (lane == 63) atomicAdd(&s_base, less);
  }
  __syncthreads();
  const int base = s_base;
  for (int r = threadIdx.x; r < span; r += W * 64) {
    int sum = 0;
#pragma unroll
    for (int k = 0; k < W; ++k) sum += s_mem[k * span + r];
    s_count[r] = sum;
  }
  __syncthreads();
  const int all = block_scan<W>(s_count, span, s_slots);
  for (int r = threadIdx.x; r < span; r += W * 64) {
    int run = base + s_count[r];
    if (r < here) s.start[row0 + r] = run;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const int c = s_mem[k * span + r];
      s_mem[k * span + r] = run;
      run += c;
    }
  }
  if (row0 + here == s.rows && threadIdx.x == 0) s.start[s.rows] = base + all;
  for (int r = w; r < here; r += W)  // (on their way while the tokens are placed)
    if ((r + 1 < span ? s_count[r + 1] : all) == s_count[r]) zero_row<D>(dtable + (int64_t)(row0 + r) * channels, channels);
  __syncthreads();
  place_in_order(
      a, b, s.span_bits, s_mem + w * span,
      [&](int64_t i) {
        const int2 x = get(i);
        return make_int2(x.x >= 0 && x.x < here ? x.x : -1, x.y);
      },
      [&](int place, int r, int i) {
        s.order[place] = i;
        s.row[place] = row0 + r;
      });
}

// ------------------------------------------------------------------------------------ sums

struct Sums {
  const void* dout;
  void* dtable;
  const int32_t *order, *row, *start;
  float *head, *tail;  // [pieces][channels]: of a piece's first row, if it is long and began before; of its last, if long and it goes on
  int32_t* joins;      // long rows so far, then
  int2* join;          // (the piece they begin in, how many they lie in), in any order
  int rows, channels, piece;
  int shortest;  // rows of more tokens, in several pieces, are long
  float scale;
};

template <int V, bool TAIL> __device__ __forceinline__ void store_floats(float* p, int c0, int end, const float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const float part[4] = {v[i], v[i + 1], v[i + 2], v[i + 3]};
    store_chunk<DT::F32, TAIL>(p, c0 + i, end, part);
  }
}

// TPR lanes a piece (blockIdx.y: a slice of the channels), each with a chunk of V channels.
template <DT D, int TPR, bool TAIL>
__global__ __launch_bounds__(256) void embedding_piece_kernel(Sums a) {
  using T = typename Elem<D>::T;
  constexpr int V = kChunk<D>, kFlight = 8;
  const int lane = threadIdx.x % TPR;
  const int64_t id = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  const int64_t total = a.start[a.rows], first = id * a.piece, end = min(total, first + a.piece);
  if (first >= end) return;
  const int c0 = (blockIdx.y * TPR + lane) * V;
  const T* dout = static_cast<const T*>(a.dout);
  // The rows that begin here, to their ends, but of long ones what lies here.
  int cur = a.row[first];
  const int final = a.row[end - 1];
  const int cur_from = a.start[cur], cur_to = a.start[cur + 1], final_from = a.start[final], final_to = a.start[final + 1];
  const bool began = cur_from < first && cur_to - cur_from > a.shortest, goes_on = final_to > end && final_to - final_from > a.shortest;
  const int64_t from = cur_from < first && !began ? cur_to : first, to = goes_on ? end : final_to;
  if (goes_on && final_from >= first && lane == 0 && blockIdx.y == 0)
    a.join[atomicAdd(a.joins, 1)] = make_int2((int)id, (int)((final_to - 1) / a.piece - id + 1));
  if (from >= end) return;
  float acc[V] = {};
  bool head = began;  // (of the row that is being summed)
  const auto leave = [&](bool tail) {
    if (head || tail) {
      float* p = (head ? a.head : a.tail) + id * a.channels;
      store_floats<V, TAIL>(p, c0, a.channels, acc);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] *= a.scale;
      store_chunk<D, TAIL>(static_cast<T*>(a.dtable) + (int64_t)cur * a.channels, c0, a.channels, acc);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    head = false;
  };
  if (from > first) cur = a.row[from];
  for (int64_t p0 = from; p0 < to; p0 += kFlight) {
    Chunk<T, V> x[kFlight];
    int rows[kFlight], at[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int64_t p = min(p0 + k, to - 1);
      rows[k] = p0 + k < to ? a.row[p] : -1;
      at[k] = a.order[p];
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) x[k] = load_raw<D, TAIL>(dout + (int64_t)at[k] * a.channels, c0, a.channels);
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (rows[k] < 0) break;
      if (rows[k] != cur) {
        leave(false);
        cur = rows[k];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] += to_float<D>(x[k].v[j]);
    }
  }
  leave(goes_on);
}

// Long rows: groups of 64 lanes take an equal share of a row's pieces each, 4 channels a lane (blockIdx.y: a
// slice of 256 channels).
constexpr int kJoinGroups = 8;
template <DT D> __global__ __launch_bounds__(kJoinGroups * 64) void embedding_join_kernel(Sums a) {
  __shared__ float4 s_sum[kJoinGroups][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = (blockIdx.y * 64 + lane) * 4, count = *a.joins;
  for (int k = blockIdx.x; k < count; k += gridDim.x) {
    const int2 what = a.join[k];
    const int64_t id = what.x, pieces = what.y;  // at least two
    const int row = a.row[(id + 1) * a.piece - 1];
    const int64_t per = (pieces + kJoinGroups - 1) / kJoinGroups, from = min(pieces, per * w), to = min(pieces, from + per);
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kFlight = 8;
    for (int64_t p0 = from; p0 < to; p0 += kFlight) {
      float x[kFlight][4];
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int64_t p = min(p0 + i, to - 1);
        load_chunk<DT::F32>((p == 0 ? a.tail : a.head) + (id + p) * a.channels, c, p0 + i < to ? a.channels : 0, x[i]);
      }
#pragma unroll
      for (int i = 0; i < kFlight; ++i) sum = make_float4(sum.x + x[i][0], sum.y + x[i][1], sum.z + x[i][2], sum.w + x[i][3]);
    }
    __syncthreads();  // (the sums of the row before have been read)
    s_sum[w][lane] = sum;
    __syncthreads();
    if (w != 0) continue;
#pragma unroll
    for (int i = 1; i < kJoinGroups; ++i) {
      const float4 o = s_sum[i][lane];
      sum = make_float4(sum.x + o.x, sum.y + o.y, sum.z + o.z, sum.w + o.w);
    }
    const float f[4] = {sum.x * a.scale, sum.y * a.scale, sum.z * a.scale, sum.w * a.scale};
    typename Elem<D>::T* out = static_cast<typename Elem<D>::T*>(a.dtable) + (int64_t)row * a.channels;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < a.channels) out[c + j] = from_float<D>(f[j]);
  }
}

constexpr int kMaxRows = kMaxBuckets * kMaxSpan;

// Lists up to this many tokens are sorted without the split: every bucket reads the whole list (8,000 tokens, 65,536
// rows: 34 us for 42 with it; 16,000: 46 for 42).
constexpr int64_t kShortList = 8192;

template <DT D, int TPR, bool TAIL> void launch_lanes(const Sums& a, int64_t pieces, int chunks, hipStream_t stream) {
  constexpr int each = 256 / TPR;
  const dim3 grid((unsigned)((pieces + each - 1) / each), (chunks + TPR - 1) / TPR);
  embedding_piece_kernel<D, TPR, TAIL><<<grid, 256, 0, stream>>>(a);
}
template <DT D, bool TAIL> void launch_pieces(const Sums& a, int64_t pieces, hipStream_t stream) {
  const int chunks = (a.channels + kChunk<D> - 1) / kChunk<D>;
  if (chunks <= 8) launch_lanes<D, 8, TAIL>(a, pieces, chunks, stream);
  else if (chunks <= 16) launch_lanes<D, 16, TAIL>(a, pieces, chunks, stream);
  else if (chunks <= 32) launch_lanes<D, 32, TAIL>(a, pieces, chunks, stream);
  else launch_lanes<D, 64, TAIL>(a, pieces, chunks, stream);
}

template <DT D> Status backward(Sort s, Sums a, hipStream_t stream) {
  const bool whole = s.n <= kShortList;
  s.span_bits = 0;  // (a short list in about as many buckets as workgroups run at once)
  while (((int64_t)(whole ? 512 : kMaxBuckets) << s.span_bits) < s.rows && (1 << s.span_bits) < kMaxSpan) ++s.span_bits;
  s.buckets = ((s.rows - 1) >> s.span_bits) + 1;
  s.tiles = 0;
  if (!whole) {
    s.tile = 4096;
    while ((s.n + s.tile - 1) / s.tile > kMaxTiles) s.tile *= 2;
    s.tiles = (int)((s.n + s.tile - 1) / s.tile);
  }
  // Pieces of 64 positions where those are enough, of 8 at least (135,826 tokens, 100 rows of 1,024 channels, all four
  // steps: 70 us, with pieces of 32 76, of 16 89).
  a.piece = 8;
  while (s.n / a.piece > (a.piece < 64 ? 2048 : 65536)) a.piece *= 2;
  // Beside its own positions a piece sums a row that is not long to its end, and all wait for the piece with most: (3)
  // of the skewed list above takes 106 us where a row is long from a piece's 64 tokens on, 86 from 16.
  a.shortest = std::max(a.piece / 4, 8);
  const int64_t pieces = (s.n + a.piece - 1) / a.piece;

  int dev = 0;
  SUBM_HIP_TRY(hipGetDevice(&dev));
  const auto padded = [](size_t bytes) { return (bytes + 255) / 256 * 256; };
  const size_t list = padded((size_t)s.n * sizeof(int32_t)), starts = padded(((size_t)s.rows + 1) * sizeof(int32_t));
  const size_t counts = padded((size_t)s.tiles * s.buckets * sizeof(int32_t)), buckets = padded(((size_t)s.buckets + 1) * sizeof(int32_t));
  const size_t sums = padded((size_t)pieces * a.channels * sizeof(float)), joins = padded((size_t)pieces * sizeof(int2) + 256);
  ScratchLease lease;
  void* scratch = nullptr;
  Status st = lease.take(dev, stream, starts + 2 * list + (s.tiles > 0 ? 2 * list + counts + buckets : 0) + 2 * sums + joins, &scratch);
  if (!st.ok()) return st;
  unsigned char* p = static_cast<unsigned char*>(scratch);
  const auto part = [&](size_t bytes) {
    unsigned char* q = p;
    p += bytes;
    return q;
  };
  s.start = reinterpret_cast<int32_t*>(part(starts));
  s.order = reinterpret_cast<int32_t*>(part(list));
  s.row = reinterpret_cast<int32_t*>(part(list));
  a.head = reinterpret_cast<float*>(part(sums));
  a.tail = reinterpret_cast<float*>(part(sums));
  s.joins = reinterpret_cast<int32_t*>(part(256));
  a.join = reinterpret_cast<int2*>(part(joins - 256));
  auto* dtable = static_cast<typename Elem<D>::T*>(a.dtable);
  if (s.tiles > 0) {
    s.split = reinterpret_cast<int2*>(part(2 * list));
    s.counts = reinterpret_cast<int32_t*>(part(counts));
    s.bucket = reinterpret_cast<int32_t*>(part(buckets));
    embedding_count_kernel<<<s.tiles, kSplitThreads, 0, stream>>>(s);
    embedding_split_kernel<D><<<s.tiles, kSplitThreads, 0, stream>>>(s, dtable, a.channels);
    SUBM_HIP_TRY(hipGetLastError());
  }
  if (s.tiles == 0 || s.span_bits > 0) {
    const auto lds = [&](int waves) { return (size_t)(waves + 1) * sizeof(int32_t) << s.span_bits; };
    if (s.span_bits <= 9) embedding_sort_kernel<D, 16><<<s.buckets, 1024, lds(16), stream>>>(s, dtable, a.channels);
    else embedding_sort_kernel<D, 4><<<s.buckets, 256, lds(4), stream>>>(s, dtable, a.channels);
    SUBM_HIP_TRY(hipGetLastError());
  }
  if (s.n == 0) return Status{};
  a.order = s.order;
  a.row = s.row;
  a.start = s.start;
  a.joins = s.joins;
  if (a.channels % kChunk<D> == 0) launch_pieces<D, false>(a, pieces, stream);
  else launch_pieces<D, true>(a, pieces, stream);
  SUBM_HIP_TRY(hipGetLastError());
  if (pieces > 1) {
    const dim3 grid((unsigned)std::min<int64_t>(pieces, 512), (a.channels + 255) / 256);
    embedding_join_kernel<D><<<grid, kJoinGroups * 64, 0, stream>>>(a);
    SUBM_HIP_TRY(hipGetLastError());
  }
  return Status{};
}

template <DT D>
hipError_t forward(const void* table, int rows, int channels, const void* tokens, int wide, int64_t n, float scale, void* out,
                   hipStream_t stream) {
  using T = typename Elem<D>::T;
  const int lanes = short_lanes((channels + kChunk<D> - 1) / kChunk<D>), step = 256 / lanes;
  const unsigned blocks = (unsigned)std::min<int64_t>((n + step - 1) / step, 256 * 16);
  const T *t = static_cast<const T*>(table);
  if (channels % kChunk<D> == 0)
    embedding_forward_kernel<D, false><<<blocks, 256, 0, stream>>>(t, rows, channels, tokens, wide, n, scale, static_cast<T*>(out), lanes);
  else
    embedding_forward_kernel<D, true><<<blocks, 256, 0, stream>>>(t, rows, channels, tokens, wide, n, scale, static_cast<T*>(out), lanes);
  return hipGetLastError();
}

Status check_embedding(int rows, int channels, int dtype, int token_bytes, int64_t n, float scale) {
  if (dtype != SUBM_F32 && dtype != SUBM_F16 && dtype != SUBM_BF16)
    return make_status(SUBM_ERR_UNSUPPORTED, "dtype must be SUBM_F32, SUBM_F16 or SUBM_BF16");
  if (token_bytes != 4 && token_bytes != 8) return make_status(SUBM_ERR_INVALID_ARG, "token_bytes must be 4 or 8");
  if (n < 0 || n > INT32_MAX) return make_status(SUBM_ERR_INVALID_ARG, "n must be 0 .. 2^31 - 1");
  if (rows < 1) return make_status(SUBM_ERR_INVALID_ARG, "rows must be at least 1");
  if (rows > kMaxRows) return make_status(SUBM_ERR_UNSUPPORTED, "rows exceeds 2^21");
  if (channels < 1) return make_status(SUBM_ERR_INVALID_ARG, "channels must be at least 1");
  if (channels > 16384) return make_status(SUBM_ERR_UNSUPPORTED, "channels exceeds 16384");
  if (!std::isfinite(scale)) return make_status(SUBM_ERR_INVALID_ARG, "scale must be finite");
  return Status{};
}

bool misaligned(const void* p, int size) { return reinterpret_cast<uintptr_t>(p) % size != 0; }

}  // namespace
}  // namespace submconv

using namespace submconv;

extern "C" int sparse_embedding_forward(const void* table, int rows, int channels, int dtype, const void* tokens, int token_bytes,
                                        int64_t n, float scale, void* out, hipStream_t stream) {
  return no_throw([&]() -> int {
    clear_error();
    const Status st = check_embedding(rows, channels, dtype, token_bytes, n, scale);
    if (!st.ok()) return fail(st);
    if (n == 0) return SUBM_OK;
    if (table == nullptr || tokens == nullptr || out == nullptr) return fail(SUBM_ERR_INVALID_ARG, "table, tokens or out is NULL");
    const int elem = dtype == SUBM_F32 ? 4 : 2;
    if (misaligned(table, elem) || misaligned(out, elem) || misaligned(tokens, token_bytes))
      return fail(SUBM_ERR_INVALID_ARG, "a pointer is not aligned to its element");
    if (out == table) return fail(SUBM_ERR_INVALID_ARG, "out must not alias the table");
    const int wide = token_bytes == 8;
    hipError_t e;
    if (dtype == SUBM_F32) e = forward<DT::F32>(table, rows, channels, tokens, wide, n, scale, out, stream);
    else if (dtype == SUBM_F16) e = forward<DT::F16>(table, rows, channels, tokens, wide, n, scale, out, stream);
    else e = forward<DT::BF16>(table, rows, channels, tokens, wide, n, scale, out, stream);
    if (e != hipSuccess) return fail(hip_status(e, "sparse_embedding_forward launch"));
    return SUBM_OK;
  });
}

extern "C" int sparse_embedding_backward(const void* dout, int rows, int channels, int dtype, const void* tokens, int token_bytes,
                                         int64_t n, float scale, void* dtable, hipStream_t stream) {
  return no_throw([&]() -> int {
    clear_error();
    Status st = check_embedding(rows, channels, dtype, token_bytes, n, scale);
    if (!st.ok()) return fail(st);
    if (dtable == nullptr || (n > 0 && (dout == nullptr || tokens == nullptr)))
      return fail(SUBM_ERR_INVALID_ARG, "dout, tokens or dtable is NULL");
    const int elem = dtype == SUBM_F32 ? 4 : 2;
    if (misaligned(dout, elem) || misaligned(dtable, elem) || misaligned(tokens, token_bytes))
      return fail(SUBM_ERR_INVALID_ARG, "a pointer is not aligned to its element");
    if (dtable == dout) return fail(SUBM_ERR_INVALID_ARG, "dtable must not alias dout");
    Sort s{};
    s.tokens = tokens;
    s.wide = token_bytes == 8;
    s.rows = rows;
    s.n = n;
    Sums a{};
    a.dout = dout;
    a.dtable = dtable;
    a.rows = rows;
    a.channels = channels;
    a.scale = scale;
    if (dtype == SUBM_F32) st = backward<DT::F32>(s, a, stream);
    else if (dtype == SUBM_F16) st = backward<DT::F16>(s, a, stream);
    else st = backward<DT::BF16>(s, a, stream);
    if (!st.ok()) return fail(st);
    return SUBM_OK;
  });
}
