// The backward kernels of attention, for whole items (attention_backward.hip) and for windows of them
// (window_attention_backward.hip), and their launches.
#pragma once

#include <algorithm>
#include <cmath>

#include "attention_common.h"
#include "attention_window.h"

namespace submconv {
namespace {

struct BwdArgs {
  subm_heads_t dout, q, k, v, out, dq, dk, dv;
  const float* lse;
  float *norm, *delta;  // [kv_heads, nq * group]: log2 of each packed row's normaliser (less kF16Shift), and d
  // float16 only: [kv_heads, q_slots] the largest |dout| and bound of |dp - d| of each query block,
  // and [kv_heads, v_slots] a bound of |v|_2 over each block of kNormKeys keys; with WINDOW also those of
  // each packed row, [kv_heads, nq * group], and |v|_2 of each key, [kv_heads, nk]
  float2 *peak, *row_peak;
  float *v_norm, *key_norm;
  const int64_t *q_offsets, *k_offsets;
  int64_t nq, nk, q_slots, v_slots;
  int items, heads, kv_heads, head_dim;
  float scale;
  int q_rows;  // packed rows of a workgroup of the dq kernel
  // Tiles in parts: float32 sums of dq by the first cut, of dk and dv by the second, [place][rows of
  // a tile][DP], summed by a third kernel.
  Cut q_cut, k_cut;
  float *dq_part, *dk_part, *dv_part;
  // Of the kernels with WINDOW.  The first `sinks` keys of an item are seen by all rows behind them: their
  // dk and dv come from chunks of `sink_rows` packed rows, [kv_heads][chunk][sinks][2][DP] float32 sums, added up
  // by a kernel of their own.
  Window window;
  int sink_rows;
  int64_t sink_slots;
  float* sink_part;
};

constexpr int kStep = 32;  // rows of the walked tile

constexpr int kNormKeys = 256;  // keys of a workgroup of the kernel that leaves v's norms

constexpr float kF16Shift = 15.f;  // p is scaled by 2^15 in float16 products

// 2^-floor(log2 x): the power of two that takes x to [1, 2); 1 for 0, subnormal and non-finite x.
__device__ __forceinline__ float unit_scale(float x) {
  const int e = (int)(__float_as_uint(x) >> 23) & 255;
  return e == 0 || e >= 254 ? 1.f : __uint_as_float((uint32_t)(254 - e) << 23);
}

// The power of two for e (see the top): from the largest |dout| and a bound of |dp - d|.
__device__ __forceinline__ float e_scale(float peak, float bound) {
  return fminf(unit_scale(peak), unit_scale(bound) * 16384.f);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int mk = 32; mk >= 1; mk >>= 1) v = fmaxf(v, __shfl_xor(v, mk, 64));
  return v;
}

// A bound of |v|_2 over the item's keys, from their blocks: the same in every thread of the
// workgroup, all of which call it (`slots`: a float a wave).
template <int W> __device__ __forceinline__ float item_norm(const BwdArgs& a, int head, int item, int64_t k0, int nk, float* slots) {
  const float* norms = a.v_norm + head * a.v_slots + k0 / kNormKeys + item;
  const int blocks = (int)(((int64_t)nk + kNormKeys - 1) / kNormKeys);
  float v = 0.f;
  for (int t = threadIdx.x; t < blocks; t += W * 64) v = fmaxf(v, norms[t]);
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) v = fmaxf(v, slots[w]);
  return v;
}

__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float2 larger(float2 a, float2 b) { return make_float2(fmaxf(a.x, b.x), fmaxf(a.y, b.y)); }

// Of values >= 0: the largest of the own lane and of those after it up to 31 (lanes 0 .. 31), or of those before it
// from 32 on (lanes 32 .. 63), in VALU instructions.
__device__ __forceinline__ float max_outwards(float v, int lane) {
  float after = v, before = v;  // in rows of 16: lanes shifted down, and up
  after = dpp_max<0x101>(after);
  after = dpp_max<0x102>(after);
  after = dpp_max<0x104>(after);
  after = dpp_max<0x108>(after);
  before = dpp_max<0x111>(before);
  before = dpp_max<0x112>(before);
  before = dpp_max<0x114>(before);
  before = dpp_max<0x118>(before);
  if (lane < 16) after = fmaxf(after, lane_value(after, 16));
  if (lane >= 48) before = fmaxf(before, lane_value(before, 47));
  return lane < 32 ? after : before;
}
__device__ __forceinline__ float2 max_outwards(float2 v, int lane) {
  return make_float2(max_outwards(v.x, lane), max_outwards(v.y, lane));
}
__device__ __forceinline__ float max_of_wave(float v) { return lanes_max(v, 64); }
__device__ __forceinline__ float2 max_of_wave(float2 v) { return make_float2(lanes_max(v.x, 64), lanes_max(v.y, 64)); }
__device__ __forceinline__ float max_of_halves(float v) { return half_max(v); }
__device__ __forceinline__ float2 max_of_halves(float2 v) { return make_float2(half_max(v.x), half_max(v.y)); }

// The largest of `one` over the lane's own range [lo, hi), which rises from lane to lane of 0 .. 31 by at most
// `step` at either end (lanes l and l + 32: the same); `whole`: the largest of each `block` of them.  What all
// lanes' ranges share is read by the wave together; to it come each lane's first `step` values and those of the
// lanes after it, and each lane's last and those of the lanes before it.  (A value may be read twice; loads of a
// batch are in flight at once.)
template <typename V>
__device__ __forceinline__ V range_max(int lo, int hi, int step, int block, const V* one, const V* whole, int lane) {
  constexpr int kBatch = 4;
  const int first = __builtin_amdgcn_readlane(lo, 31), end = __builtin_amdgcn_readlane(hi, 0);
  const bool upper = lane >= 32;
  V m{}, all{};
  if (first < end) {
    const V* edge = one + (upper ? hi - step : lo);
    const int b0 = (first + block - 1) / block, b1 = max(end / block, b0);  // whole blocks b0 .. b1 - 1, values before and after
    const bool any = b0 < b1;
    const int before = any ? b0 * block - first : end - first, after = any ? end - b1 * block : 0;
    const int count = before + after + b1 - b0;
    const auto value = [&](int i) {
      return *(i < before ? one + first + i : i < before + after ? one + b1 * block + (i - before) : whole + b0 + (i - before - after));
    };
    m = edge[0];
    for (int i0 = lane; i0 < count; i0 += 64 * kBatch) {
      V v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) v[i] = value(min(i0 + i * 64, count - 1));
#pragma unroll
      for (int i = 0; i < kBatch; ++i) all = larger(all, v[i]);
    }
    for (int i0 = 1; i0 < step; i0 += 2 * kBatch) {
      V v[2 * kBatch];
#pragma unroll
      for (int i = 0; i < 2 * kBatch; ++i) v[i] = edge[min(i0 + i, step - 1)];
#pragma unroll
      for (int i = 0; i < 2 * kBatch; ++i) m = larger(m, v[i]);
    }
    m = larger(max_outwards(m, lane), max_of_wave(all));
  } else {  // a window of few rows: all of the lane's own
    for (int i0 = lo + (upper ? 1 : 0); i0 < hi; i0 += 2 * kBatch) {
      V v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) v[i] = one[min(i0 + 2 * i, hi - 1)];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) m = larger(m, v[i]);
    }
  }
  return max_of_halves(m);
}

// The largest |v|_2 of the keys that the lane's row, of token `token`, sees (rows rise by at most a token from
// lane to lane).
__device__ __forceinline__ float window_norm(const BwdArgs& a, int head, int item, int64_t k0, int nk, int64_t p, int lane) {
  const float* keys = a.key_norm + head * a.nk + k0;
  const float* blocks = a.v_norm + head * a.v_slots + k0 / kNormKeys + item;
  const int64_t first = p - a.window.left, past = p + a.window.right + 1;
  const int lo = (int)(first < 0 ? 0 : first < nk ? first : nk), hi = (int)(past < 0 ? 0 : past < nk ? past : nk);
  float m = range_max(lo, hi, 1, kNormKeys, keys, blocks, lane);
  if (a.window.sinks > 0) {  // those before p + right, from running maxima of the first 64 and the next
    const int most = min(a.window.sinks, nk), mine = min(a.window.sinks, hi);
    float low = lane < most ? keys[lane] : 0.f, high = lane + 64 < most ? keys[lane + 64] : 0.f;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const float a_low = __shfl_up(low, o, 64), a_high = __shfl_up(high, o, 64);
      if (lane >= o) low = fmaxf(low, a_low), high = fmaxf(high, a_high);
    }
    const float in_low = __shfl(low, max(min(mine, 64) - 1, 0), 64), in_high = __shfl(high, max(mine - 65, 0), 64);
    if (mine > 0) m = fmaxf(m, in_low);
    if (mine > 64) m = fmaxf(m, in_high);
  }
  return m;
}

template <DT D> __device__ __forceinline__ float absmax_frag(const Frag<D>& f) {
  float m = 0.f;
  const uint32_t w[4] = {f.v[0].x, f.v[0].y, f.v[0].z, f.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = fmaxf(m, fmaxf(fabsf(to_float<D>((uint16_t)w[i])), fabsf(to_float<D>((uint16_t)(w[i] >> 16)))));
  return m;
}

template <DT D> __device__ __forceinline__ float dot_frag(const Frag<D>& a, const Frag<D>& b, float s) {
#pragma unroll
  for (int k = 0; k < Elem<D>::kSize / 2; ++k) {
    const uint32_t x[4] = {a.v[k].x, a.v[k].y, a.v[k].z, a.v[k].w}, y[4] = {b.v[k].x, b.v[k].y, b.v[k].z, b.v[k].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (D == DT::F32) {
        s = fmaf(__uint_as_float(x[i]), __uint_as_float(y[i]), s);
      } else {
        s = fmaf(to_float<D>((uint16_t)x[i]), to_float<D>((uint16_t)y[i]), s);
        s = fmaf(to_float<D>((uint16_t)(x[i] >> 16)), to_float<D>((uint16_t)(y[i] >> 16)), s);
      }
    }
  }
  return s;
}

// A row's accumulator times `f` to a float32 copy.
template <int DC> __device__ __forceinline__ void store_part(float* row, const f32x16_t (&acc)[DC / 32], float f, int lane) {
#pragma unroll
  for (int db = 0; db < DC / 32; ++db)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(row + db * 32 + 8 * i + 4 * (lane >> 5)) =
          make_float4(acc[db][4 * i] * f, acc[db][4 * i + 1] * f, acc[db][4 * i + 2] * f, acc[db][4 * i + 3] * f);
}

// A bound of |v|_2 over each block of keys (blockIdx.x of those, blockIdx.y the key head): 16 lanes a
// row, each with the largest square sum of its 8 channels, added up (one sum a block and not one a
// row; the longest row's norm is between a quarter of the bound and all of it).  With WINDOW each key's own,
// too, and the largest of them.
template <DT D, bool WINDOW> __global__ __launch_bounds__(256) void attention_norm_kernel(BwdArgs a) {
  __shared__ float s_top[64];
  const int head = blockIdx.y, c = threadIdx.x % 16 * 8;
  int tile;
  const int item = find_item(a.k_offsets, a.nk, a.items, 1, kNormKeys, blockIdx.x, &tile);
  int64_t k0;
  int nk;
  item_rows(a.k_offsets, a.nk, item, &k0, &nk);
  const int64_t first = (int64_t)tile * kNormKeys;
  if (first >= nk) return;
  const int rows = (int)(nk - first < kNormKeys ? nk - first : kNormKeys);
  const Heads<D> v = heads_of<D>(a.v);
  const typename Elem<D>::T* p = v.data + (k0 + first) * v.row + (int64_t)head * v.head + c;
  Frag<D> f[kNormKeys / 16];
#pragma unroll
  for (int i = 0; i < kNormKeys / 16; ++i) {
    const int r = i * 16 + threadIdx.x / 16;
    f[i].v[0] = r < rows && c < a.head_dim ? *reinterpret_cast<const uint4*>(p + (int64_t)r * v.row) : make_uint4(0, 0, 0, 0);
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kNormKeys / 16; ++i) {
    float sq = dot_frag<D>(f[i], f[i], 0.f);
    if constexpr (WINDOW) {
      sq = lanes_sum<16>(sq);
      const int r = i * 16 + threadIdx.x / 16;
      if (c == 0 && r < rows) a.key_norm[head * a.nk + k0 + first + r] = sqrtf(sq);
    }
    top = fmaxf(top, sq);
  }
  top = fmaxf(top, __shfl_xor(top, 16, 64));
  top = fmaxf(top, __shfl_xor(top, 32, 64));
  if ((threadIdx.x & 63) < 16) s_top[threadIdx.x / 64 * 16 + threadIdx.x % 64] = top;
  __syncthreads();
  if (threadIdx.x != 0) return;
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < (WINDOW ? 1 : 16); ++i) sq += fmaxf(fmaxf(s_top[i], s_top[16 + i]), fmaxf(s_top[32 + i], s_top[48 + i]));
  a.v_norm[head * a.v_slots + blockIdx.x] = sqrtf(sq);
}

// The rows `odd` of a wave's dq, or the keys `odd` of its dk and dv, one by one (see attention_window.h), from the
// kernel's arguments and what was stored on, so that the accumulators need not outlive their store.
template <DT D> __device__ __forceinline__ void put_pair(typename Elem<D>::T* row, float2 o, int head_dim, int lane) {
  if (2 * lane >= head_dim) return;
  row[2 * lane] = from_float<D>(o.x);
  row[2 * lane + 1] = from_float<D>(o.y);
}

template <DT D, int DC, int W, int CUT>
__device__ __forceinline__ void dq_again(uint64_t odd, float base, float d, float unit, int wave, int lane) {
  constexpr DT S = CUT == kNoCut ? D : DT::F32;  // of what was stored
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
  const BwdArgs a = fresh_args<BwdArgs>();
  const int group = a.heads / a.kv_heads;
  const Share share = window_share<CUT>(a.q_cut, a.window, true);
  int tile;
  const int item = find_item(a.q_offsets, a.nq, a.items, group, 32 * W, share.slot, &tile);
  int64_t q0, k0;
  int nq, nk;
  item_rows(a.q_offsets, a.nq, item, &q0, &nq);
  item_rows(a.k_offsets, a.nk, item, &k0, &nk);
  const int first = tile * 32 * W, last = min(nq * group, first + 32 * W) - 1;
  const RowMap qmap{q0, share.head * group, group};
  const Heads<D> k = heads_of<D>(a.k), v = heads_of<D>(a.v);
  const typename Elem<D>::T* kp = k.data + k0 * k.row + (int64_t)share.head * k.head;
  const typename Elem<D>::T* vp = v.data + k0 * v.row + (int64_t)share.head * v.head;
  KeyTiles<kStep> walk;
  walk.place(a.window, nk, nk - nq, first / group, last / group);
  if constexpr (CUT != kNoCut) {
    int tiles = walk.tiles;
    const int from = part_steps(a.q_cut, share.part, &tiles);
    walk.cut(from, tiles);
  }
  for (; odd != 0; odd &= odd - 1) {
    const int l = __builtin_ctzll(odd), row = first + wave * 32 + l, p = row / group + nk - nq;
    if (!hidden_odd<D>(a.window, walk, p, nk, kp, k.row, a.head_dim, lane)) continue;
    const float2 qr = row_pair<D>(qmap.at<D>(heads_of<D>(a.q), row), a.head_dim, lane);
    const float2 gr = row_pair<D>(qmap.at<D>(heads_of<D>(a.dout), row), a.head_dim, lane);
    const float b = lane_value(base, l), dr = lane_value(d, l), u = lane_value(unit, l);
    typename Elem<S>::T* stored;
    if constexpr (CUT == kNoCut) stored = qmap.at<D>(heads_of<D>(a.dq), row);
    else stored = a.dq_part + ((int64_t)share.place * 32 * W + wave * 32 + l) * tile_width(DC);
    const float2 was = row_pair<S>(stored, a.head_dim, lane);
    float2 o = make_float2(0.f, 0.f);
    for (int t = 0; t < walk.tiles && still_finite(was, o); ++t)
      for (int j = walk.key(t); j < min(walk.key(t) + kStep, walk.end(t)); ++j) {
        if (!a.window.sees(p, j)) continue;
        const float2 kr = row_pair<D>(kp + (int64_t)j * k.row, a.head_dim, lane);
        const float2 vr = row_pair<D>(vp + (int64_t)j * v.row, a.head_dim, lane);
        const float e = exp2_fast(fmaf(pair_dot(qr, kr), a.scale * kLog2e, -b)) * (pair_dot(gr, vr) - dr) * u;
        add_scaled(o, to_float<D>(from_float<D>(e)), kr);
      }
    const float f = a.scale / u;
    put_pair<S>(stored, mended(was, make_float2(o.x * f, o.y * f)), a.head_dim, lane);
  }
}

// Of key l of a wave of the dk and dv kernel: the query rows that this workgroup walks for it, and those that see it.
struct KeyRows {
  int share_head, share_place, group, key;
  int64_t q0, k0;
  int begin, end, from, to;
};
template <DT D, int W, int CUT, bool SINKS> __device__ __forceinline__ KeyRows key_rows(const BwdArgs& a, int wave, int l) {
  KeyRows r;
  r.group = a.heads / a.kv_heads;
  const Share share = !SINKS ? window_share<CUT>(a.k_cut, a.window, false) : share_of<CUT>(a.k_cut, blockIdx.x);
  r.share_head = share.head;
  r.share_place = SINKS ? share.slot : share.place;
  int tile, chunk = 0;
  const int item = SINKS ? find_item(a.q_offsets, a.nq, a.items, r.group, a.sink_rows, share.slot, &chunk)
                         : find_item(a.k_offsets, a.nk, a.items, 1, 32 * W, share.slot, &tile);
  if constexpr (SINKS) tile = blockIdx.z;
  int nq, nk;
  item_rows(a.q_offsets, a.nq, item, &r.q0, &nq);
  item_rows(a.k_offsets, a.nk, item, &r.k0, &nk);
  const int shift = nk - nq, first = tile * 32 * W, last = min(SINKS ? min(nk, a.window.sinks) : nk, first + 32 * W) - 1;
  int unused;
  a.window.rows(SINKS ? first : max(first, min(a.window.sinks, last)), SINKS, nq, shift, r.group, &r.begin, &unused);
  a.window.rows(last, SINKS, nq, shift, r.group, &unused, &r.end);
  if constexpr (SINKS) {
    r.begin = max(r.begin, chunk * a.sink_rows);
    r.end = (int)min((int64_t)r.end, (int64_t)(chunk + 1) * a.sink_rows);
  } else if constexpr (CUT != kNoCut) {
    int steps = (max(r.end - r.begin, 0) + kStep - 1) / kStep;
    r.begin += part_steps(a.k_cut, share.part, &steps) * kStep;
    r.end = min(r.end, r.begin + steps * kStep);
  }
  r.key = first + wave * 32 + l;
  a.window.rows(r.key, SINKS, nq, shift, r.group, &r.from, &r.to);
  return r;
}

// (hidden_odd of attention_window.h, of the rows that do not see key l.  From the arguments on once more, as what it
// and dkv_again need at once would not fit the scalar registers.)
template <DT D, int W, int CUT, bool SINKS> __device__ __forceinline__ bool dkv_hidden_odd(int l, int wave, int lane) {
  const BwdArgs a = fresh_args<BwdArgs>();
  const KeyRows r = key_rows<D, W, CUT, SINKS>(a, wave, l);
  if (!SINKS && r.key < a.window.sinks) return false;  // (not this kernel's)
  const RowMap qmap{r.q0, r.share_head * r.group, r.group};
  float z = 0.f;
#pragma unroll 1
  for (int i = r.begin; i < r.end; ++i) {
    if (i >= r.from && i < r.to) {
      i = r.to - 1;
      continue;
    }
    add_odd<D>(z, qmap.at<D>(heads_of<D>(a.q), i), a.head_dim, lane);
    add_odd<D>(z, qmap.at<D>(heads_of<D>(a.dout), i), a.head_dim, lane);
  }
  return __builtin_amdgcn_ballot_w64(!(z == 0.f)) != 0;
}

template <DT D, int DC, int W, int CUT, bool SINKS> __device__ __forceinline__ void dkv_again(uint64_t odd, float unit, int wave, int lane) {
  constexpr bool kPart = SINKS || CUT != kNoCut;
  constexpr DT S = kPart ? DT::F32 : D;
  constexpr int DP = tile_width(DC);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
  for (; odd != 0; odd &= odd - 1) {
    const int l = __builtin_ctzll(odd);
    if (!dkv_hidden_odd<D, W, CUT, SINKS>(l, wave, lane)) continue;
    const BwdArgs a = fresh_args<BwdArgs>();
    const KeyRows r = key_rows<D, W, CUT, SINKS>(a, wave, l);
    const RowMap qmap{r.q0, r.share_head * r.group, r.group}, kmap{r.k0, r.share_head, 1};
    const int64_t stats = r.share_head * (a.nq * r.group) + r.q0 * r.group;
    const float u = D == DT::F16 ? lane_value(unit, l) : 1.f, f = D == DT::F16 ? u / 32768.f : 1.f;
    const float2 kr = row_pair<D>(kmap.at<D>(heads_of<D>(a.k), r.key), a.head_dim, lane);
    const float2 vr = row_pair<D>(kmap.at<D>(heads_of<D>(a.v), r.key), a.head_dim, lane);
    typename Elem<S>::T *dk, *dv;
    if constexpr (SINKS) {
      dk = a.sink_part + (((int64_t)r.share_head * a.sink_slots + r.share_place) * a.window.sinks + r.key) * 2 * DP;
      dv = dk + DP;
    } else if constexpr (kPart) {
      const int64_t at = ((int64_t)r.share_place * 32 * W + wave * 32 + l) * DP;
      dk = a.dk_part + at;
      dv = a.dv_part + at;
    } else {
      dk = kmap.at<D>(heads_of<D>(a.dk), r.key);
      dv = kmap.at<D>(heads_of<D>(a.dv), r.key);
    }
    const float2 was_k = row_pair<S>(dk, a.head_dim, lane), was_v = row_pair<S>(dv, a.head_dim, lane);
    float2 ok = make_float2(0.f, 0.f), ov = ok;
    for (int i = max(r.from, r.begin); i < min(r.to, r.end) && (still_finite(was_k, ok) || still_finite(was_v, ov)); ++i) {
      const float2 qr = row_pair<D>(qmap.at<D>(heads_of<D>(a.q), i), a.head_dim, lane);
      const float2 gr = row_pair<D>(qmap.at<D>(heads_of<D>(a.dout), i), a.head_dim, lane);
      const float p = exp2_fast(fmaf(pair_dot(qr, kr), a.scale * kLog2e, -a.norm[stats + i]));
      const float e = p * (pair_dot(gr, vr) - a.delta[stats + i]) * f;
      add_scaled(ov, to_float<D>(from_float<D>(p)), gr);
      add_scaled(ok, to_float<D>(from_float<D>(e)), qr);
    }
    const float fk = a.scale / u, fv = D == DT::F16 ? 1.f / 32768.f : 1.f;
    put_pair<S>(dk, mended(was_k, make_float2(ok.x * fk, ok.y * fk)), a.head_dim, lane);
    put_pair<S>(dv, mended(was_v, make_float2(ov.x * fv, ov.y * fv)), a.head_dim, lane);
  }
}

// d of the own query rows, then dq over the keys, which stream through LDS in tiles of 32.  As in
// the forward pass a step holds independent pieces of work:
//   scores and dp of tile t + 1 (k, v),  e of tile t,  product of tile t - 1 (k).
template <DT D, int DC, int W, int OCC, int CUT, bool WINDOW>
__global__ __launch_bounds__(W * 64, OCC) void attention_dq_kernel(BwdArgs a) {
  constexpr int DP = tile_width(DC), kRows = 32 * W;
  constexpr int kTile = kStep * kRowBytes<D, DP>;
  using Loader = TileLoader<D, DP, kStep, W>;
  __shared__ __attribute__((aligned(1024))) unsigned char s_kv[6 * kTile];  // four tiles of k, two of v
  __shared__ float2 s_peak[W];
  __shared__ float s_norm[W];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.heads / a.kv_heads;
  const Share share = WINDOW ? window_share<CUT>(a.q_cut, a.window, true) : share_of<CUT>(a.q_cut, blockIdx.x);
  const int head = share.head;
  int tile;
  const int item = find_item(a.q_offsets, a.nq, a.items, group, kRows, share.slot, &tile);
  int64_t q0, k0;
  int nq, nk;
  item_rows(a.q_offsets, a.nq, item, &q0, &nq);
  item_rows(a.k_offsets, a.nk, item, &k0, &nk);
  const int rows = nq * group;
  if ((int64_t)tile * kRows >= rows) return;
  const RowMap qmap{q0, head * group, group};
  const Heads<D> k = heads_of<D>(a.k), v = heads_of<D>(a.v);
  const typename Elem<D>::T* kp = k.data + k0 * k.row + (int64_t)head * k.head;
  const typename Elem<D>::T* vp = v.data + k0 * v.row + (int64_t)head * v.head;

  const int row = tile * kRows + wave * 32 + (lane & 31);
  const bool there = row < rows;
  const int safe = there ? row : 0;
  Frag<D> qf[DC / 16], gf[DC / 16];  // own rows of q and dout
  const typename Elem<D>::T* qrow = qmap.at<D>(heads_of<D>(a.q), safe);
  const typename Elem<D>::T* grow = qmap.at<D>(heads_of<D>(a.dout), safe);
  const typename Elem<D>::T* orow = qmap.at<D>(heads_of<D>(a.out), safe);
  float d = 0.f, peak = 0.f, sq = 0.f;
#pragma unroll
  for (int kk = 0; kk < DC / 16; ++kk) {
    qf[kk] = own_frag<D>(qrow, there, kk, a.head_dim, lane);
    gf[kk] = own_frag<D>(grow, there, kk, a.head_dim, lane);
    d = dot_frag<D>(gf[kk], own_frag<D>(orow, there, kk, a.head_dim, lane), d);
    if constexpr (D == DT::F16) {
      peak = fmaxf(peak, absmax_frag<D>(gf[kk]));
      sq = dot_frag<D>(gf[kk], gf[kk], sq);
    }
  }
  d = half_sum(d);
  const bool first = CUT == kNoCut || share.part <= 0;  // (every part needs d, one leaves it for dk and dv)
  const float base = there ? a.lse[qmap.stat(row, a.heads)] * kLog2e : 0.f;  // log2 of the row's normaliser
  if (first && there && lane < 32) {
    const int64_t at = head * (a.nq * group) + q0 * group + row;
    a.norm[at] = D == DT::F16 ? base - kF16Shift : base;
    a.delta[at] = d;
  }
  float unit = 1.f;
  const auto scale_rows = [&]() __attribute__((always_inline)) {  // float16
    peak = half_max(peak);
    float v_norm;
    // (of the keys that the row sees and no others: a hidden value must not take this row's precision)
    if constexpr (WINDOW) v_norm = window_norm(a, head, item, k0, nk, (int64_t)(min(row, rows - 1) / group) + nk - nq, lane);
    else v_norm = item_norm<W>(a, head, item, k0, nk, s_norm);
    const float bound = 2.f * sqrtf(half_sum(sq)) * v_norm;
    unit = e_scale(peak, bound);
    if constexpr (WINDOW) {
      if (first && there && lane < 32) a.row_peak[head * (a.nq * group) + q0 * group + row] = make_float2(peak, bound);
    }
    const float2 top = make_float2(wave_max(peak), wave_max(bound));
    if (lane == 0) s_peak[wave] = top;
    __syncthreads();
    if (first && threadIdx.x == 0) {
      float2 all = top;
#pragma unroll
      for (int w = 0; w < W; ++w) all = make_float2(fmaxf(all.x, s_peak[w].x), fmaxf(all.y, s_peak[w].y));
      a.peak[head * a.q_slots + share.slot] = all;
    }
  };
  // (a window's scale takes some dependent loads, which go behind those of the first tiles)
  constexpr bool kScaleLate = D == DT::F16 && WINDOW;
  if constexpr (D == DT::F16 && !WINDOW) scale_rows();
  const float c = a.scale * kLog2e;

  Loader lk, lv;
  lk.wave = lv.wave = wave;
  lk.lane = lv.lane = lane;
  lk.place(k, a.head_dim, 1, 0, 0);
  lv.place(v, a.head_dim, 1, 0, 0);
  const uint32_t lds = lds_offset(s_kv);
  const TileReader<D, DP> rd(lane, lds, lds);
  int tiles = (nk + kStep - 1) / kStep, left = nk;
  KeyTiles<kStep> walk;
  RowView view;
  if constexpr (WINDOW) {
    const int r0 = tile * kRows, last = min(rows, r0 + kRows) - 1;
    walk.place(a.window, nk, nk - nq, r0 / group, last / group);
    view.place(a.window, nk, nk - nq, min(row, last) / group, min(r0 + wave * 32, last) / group,
               min(r0 + wave * 32 + 31, last) / group);
    tiles = walk.tiles;
  }
  if constexpr (CUT != kNoCut) {
    const int t0 = part_steps(a.q_cut, share.part, &tiles);
    if constexpr (WINDOW) {
      walk.cut(t0, tiles);
    } else {
      left = min(nk - t0 * kStep, tiles * kStep);
      kp += (int64_t)t0 * kStep * k.row;
      vp += (int64_t)t0 * kStep * v.row;
    }
  }
  const auto load_k = [&](int t, int slot) {
    if constexpr (WINDOW) {
      const int key = t < 0 ? 0 : walk.key(t);
      lk.load(kp + (int64_t)key * k.row, t < 0 ? 0 : walk.end(t) - key, lds + slot * kTile);
    } else {
      lk.load(kp + (int64_t)t * kStep * k.row, t < 0 ? 0 : left - t * kStep, lds + slot * kTile);
    }
  };
  const auto load_v = [&](int t, int slot) {
    if constexpr (WINDOW) {
      const int key = walk.key(t);
      lv.load(vp + (int64_t)key * v.row, walk.end(t) - key, lds + (4 + slot) * kTile);
    } else {
      lv.load(vp + (int64_t)t * kStep * v.row, left - t * kStep, lds + (4 + slot) * kTile);
    }
  };
  const auto scores = [&](int slot, f32x16_t& s, f32x16_t& dp) {
    s = zero16();
    dp = zero16();
#pragma unroll
    for (int kk = 0; kk < DC / 16; ++kk) {
      s = mma<D>(rd.row_frag(slot * kTile, 0, kk), qf[kk], s);
      dp = mma<D>(rd.row_frag((4 + slot % 2) * kTile, 0, kk), gf[kk], dp);
    }
  };
  f32x16_t acc[DC / 32];
#pragma unroll
  for (int db = 0; db < DC / 32; ++db) acc[db] = zero16();
  const auto product = [&](int slot, const Frag<D> (&e)[2]) {
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int db = 0; db < DC / 32; ++db) acc[db] = mma<D>(rd.column_frag(slot * kTile, st * 16, db), e[st], acc[db]);
  };
  // Step t reads k and v of tile t + 1 and k of tile t - 1 and starts the loads of tile t + 2.
  const auto start = [&]() __attribute__((always_inline)) {
    load_k(0, 0);
    load_v(0, 0);
    load_k(-1, 3);  // (zeros)
    load_k(1, 1);
    load_v(1, 1);
  };
  if constexpr (kScaleLate) {
    if (tiles > 0) start();
    scale_rows();
  }
  if (tiles > 0) {
    if constexpr (!kScaleLate) start();
    wait_vmcnt<3 * Loader::N>();
    barrier_no_fence();
    f32x16_t s0, dp0, s1, dp1;
    Frag<D> e[2];
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int i = 0; i < Elem<D>::kSize / 2; ++i) e[st].v[i] = make_uint4(0, 0, 0, 0);
    scores(0, s0, dp0);
    const auto step = [&](int t, int slot, f32x16_t& s, f32x16_t& dp, f32x16_t& s_next, f32x16_t& dp_next) {
      wait_lgkmcnt0();  // this wave's reads of the slots that are about to be loaded have returned
      wait_vmcnt<0>();
      barrier_no_fence();
      load_k(t + 2, (slot + 2) % 4);
      load_v(t + 2, slot % 2);
      scores((slot + 1) % 4, s_next, dp_next);
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = exp2_fast(fmaf(s[i], c, -base)) * (dp[i] - d) * unit;
      if constexpr (WINDOW) {
        const int key = walk.key(t), end = walk.end(t);
        if (!view.sees_all(key, kStep, end)) view.template mask<1>(key, end, lane, [&](int, int i) { s[i] = 0.f; });
      } else if ((t + 1) * kStep > left) {  // (a key past the end scores 0, which p need not take to 0)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (t * kStep + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3) >= left) s[i] = 0.f;
      }
      product((slot + 3) % 4, e);
#pragma unroll
      for (int st = 0; st < 2; ++st) e[st] = to_frag<D>(s, st);
    };
    for (int t = 0;;) {
      step(t, 0, s0, dp0, s1, dp1);
      if (++t == tiles) break;
      step(t, 1, s1, dp1, s0, dp0);
      if (++t == tiles) break;
      step(t, 2, s0, dp0, s1, dp1);
      if (++t == tiles) break;
      step(t, 3, s1, dp1, s0, dp0);
      if (++t == tiles) break;
    }
    wait_lgkmcnt0();
    wait_vmcnt<0>();
    product((tiles - 1) % 4, e);
  }
  if constexpr (WINDOW) {
    // (a row without any key, whose log sum is -infinity, meets hidden ones alone: 0 is its gradient)
    const uint64_t odd = odd_rows<DC>(acc, there && (base == -INFINITY || (__builtin_isfinite(base) && __builtin_isfinite(d))));
    if (there) {
      if constexpr (CUT != kNoCut)
        store_part<DC>(a.dq_part + ((int64_t)share.place * kRows + wave * 32 + (lane & 31)) * DP, acc, a.scale / unit, lane);
      else
        store_row<D, DC>(qmap.at<D>(heads_of<D>(a.dq), row), acc, a.scale / unit, a.head_dim, lane);
    }
    if (odd != 0) dq_again<D, DC, W, CUT>(odd, base, d, unit, wave, lane);
    return;
  }
  if (!there) return;
  if (CUT == kCutAll || (CUT == kCutLast && share.part >= 0))
    store_part<DC>(a.dq_part + ((int64_t)share.place * kRows + wave * 32 + (lane & 31)) * DP, acc, a.scale / unit, lane);
  else
    store_row<D, DC>(qmap.at<D>(heads_of<D>(a.dq), row), acc, a.scale / unit, a.head_dim, lane);
}

// The next 32 of `left` floats (zeros past them) straight to LDS, which takes 64 of them.
__device__ __forceinline__ void load_stats(const float* p, int left, uint32_t lds, int lane) {
  const i32x4_t rsrc = make_rsrc(p, kOutOfRange);
  lds = __builtin_amdgcn_readfirstlane(lds);
  const uint32_t at = lane < 32 && lane < left ? lane * 4u : kOutOfRange;
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "buffer_load_dword %0, %1, 0 offen lds"
      :
      : "v"(at), "s"(rsrc), "s"(lds));
}

// dk and dv of the own keys, over the query rows of all heads that share the key head, which
// stream through LDS in tiles of 32.  Two waves a SIMD overlap each other's exponentials and
// products.  At 128 channels in 16 bits the own rows of v stay in LDS: with the two accumulators
// and k there is no room for them in 256 registers.  Windows at 64 channels park them too, where three workgroups
// a compute unit have 168 (9,000 tokens, 6 heads, 2,048 keys: 205 us without, of k and v some in scratch memory, and 190).
//
// WINDOW: the rows from the first that sees the tile's first key to the last that sees its last, but not of
// the sinks, which are left to the kernel with SINKS: 32 of those and a chunk of rows a workgroup (of one
// wave).
template <DT D, int DC, int W, int OCC, int CUT, bool WINDOW, bool SINKS>
__global__ __launch_bounds__(W * 64, OCC) void attention_dkv_kernel(BwdArgs a) {
  constexpr int DP = tile_width(DC), kKeys = 32 * W;
  constexpr int kTile = kStep * kRowBytes<D, DP>;
  constexpr bool kParked = D != DT::F32 && (DP == 128 || (WINDOW && !SINKS && DC == 64));
  using Loader = TileLoader<D, DP, kStep, W>;
  using Parker = TileLoader<D, DP, kKeys, W>;
  // q, q, dout, dout, own v
  __shared__ __attribute__((aligned(1024))) unsigned char s_qg[4 * kTile + (kParked ? W * kTile : 0)];
  __shared__ __attribute__((aligned(16))) float s_stat[2 * 2 * 64];  // norm and d of two tiles
  __shared__ float2 s_peak[W];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.heads / a.kv_heads;
  const Share share = WINDOW && !SINKS ? window_share<CUT>(a.k_cut, a.window, false) : share_of<CUT>(a.k_cut, blockIdx.x);
  const int head = share.head;
  int tile, chunk = 0;
  const int item = SINKS ? find_item(a.q_offsets, a.nq, a.items, group, a.sink_rows, share.slot, &chunk)
                         : find_item(a.k_offsets, a.nk, a.items, 1, kKeys, share.slot, &tile);
  if constexpr (SINKS) tile = blockIdx.z;
  int64_t q0, k0;
  int nq, nk;
  item_rows(a.q_offsets, a.nq, item, &q0, &nq);
  item_rows(a.k_offsets, a.nk, item, &k0, &nk);
  const int rows = nq * group, shift = nk - nq;
  if constexpr (SINKS) {
    nk = min(nk, a.window.sinks);
    if ((int64_t)chunk * a.sink_rows >= rows) return;
  }
  if ((int64_t)tile * kKeys >= nk) return;
  // The packed rows that some key of the tile is seen by: all, or those of the window.
  int row0 = 0, row_end = rows;
  KeyView view;
  if constexpr (WINDOW) {
    const int first = tile * kKeys, last = min(nk, first + kKeys) - 1, least = SINKS ? 0 : min(a.window.sinks, last);
    const auto key_at = [&](int j) { return max(least, min(j, last)); };
    view.place(a.window, SINKS, nq, shift, group, key_at(first + wave * 32 + (lane & 31)), key_at(first + wave * 32),
               key_at(first + wave * 32 + 31));
    int unused;
    a.window.rows(key_at(first), SINKS, nq, shift, group, &row0, &unused);
    a.window.rows(last, SINKS, nq, shift, group, &unused, &row_end);
    if constexpr (SINKS) {
      row0 = max(row0, chunk * a.sink_rows);
      row_end = (int)min((int64_t)row_end, (int64_t)(chunk + 1) * a.sink_rows);
    }
    row0 = first_lane(row0);
    row_end = first_lane(row_end);
  }
  const RowMap kmap{k0, head, 1};
  const Heads<D> q = heads_of<D>(a.q), g = heads_of<D>(a.dout), v = heads_of<D>(a.v);
  const typename Elem<D>::T* qp = q.data + q0 * q.row + (int64_t)head * group * q.head;
  const typename Elem<D>::T* gp = g.data + q0 * g.row + (int64_t)head * group * g.head;
  const float* norm = a.norm + head * (a.nq * group) + q0 * group;
  const float* delta = a.delta + head * (a.nq * group) + q0 * group;

  float unit = 1.f;
  if constexpr (D == DT::F16 && !WINDOW) {  // the largest |dout| and bound of the item and head, from its query blocks
    const int64_t first = q0 * group / a.q_rows + item;
    float2 top = make_float2(0.f, 0.f);
    for (int t = threadIdx.x; t < (rows + a.q_rows - 1) / a.q_rows; t += W * 64) {
      const float2 b = a.peak[head * a.q_slots + first + t];
      top = make_float2(fmaxf(top.x, b.x), fmaxf(top.y, b.y));
    }
    top = make_float2(wave_max(top.x), wave_max(top.y));
    if (lane == 0) s_peak[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) top = make_float2(fmaxf(top.x, s_peak[w].x), fmaxf(top.y, s_peak[w].y));
    unit = e_scale(top.x, top.y);
  }
  const float p_unit = D == DT::F16 ? 1.f / 32768.f : 1.f;

  const uint32_t lds = lds_offset(s_qg);
  const int key = tile * kKeys + wave * 32 + (lane & 31);
  const bool there = key < nk;
  Frag<D> kf[DC / 16], vf[kParked ? 1 : DC / 16];
  const typename Elem<D>::T* krow = kmap.at<D>(heads_of<D>(a.k), there ? key : 0);
  const typename Elem<D>::T* vrow = kmap.at<D>(v, there ? key : 0);
#pragma unroll
  for (int kk = 0; kk < DC / 16; ++kk) {
    kf[kk] = own_frag<D>(krow, there, kk, a.head_dim, lane);
    if constexpr (!kParked) vf[kk] = own_frag<D>(vrow, there, kk, a.head_dim, lane);
  }
  if constexpr (kParked) {
    Parker park;
    park.wave = wave;
    park.lane = lane;
    park.place(v, a.head_dim, 1, 0, 0);
    park.load(kmap.at<D>(v, tile * kKeys), nk - tile * kKeys, lds + 4 * kTile);
  }
  Loader lq, lg;
  lq.wave = lg.wave = wave;
  lq.lane = lg.lane = lane;
  const int magic = 65536 / group + 1;
  const TileReader<D, DP> rd(lane, lds, lds);
  const uint32_t own = wave * kTile;  // (this wave's rows of the parked tile)
  const uint32_t stat = __builtin_amdgcn_readfirstlane(lds_offset(s_stat));
  // this workgroup's query rows: all, or its share of whole tiles (a share may be empty)
  int steps = (rows + kStep - 1) / kStep, r0 = 0, end = rows;
  if constexpr (WINDOW) {
    r0 = row0;
    end = max(row0, row_end);
    steps = (end - row0 + kStep - 1) / kStep;
  }
  if constexpr (CUT != kNoCut) {
    r0 = (WINDOW ? row0 : 0) + part_steps(a.k_cut, share.part, &steps) * kStep;
    end = min(end, r0 + steps * kStep);
  }
  int tok = r0 / group, rem = r0 - tok * group;  // of the next tile to load
  const int tok_step = kStep / group, rem_step = kStep % group;
  lq.place(q, a.head_dim, group, rem, magic);
  lg.place(g, a.head_dim, group, rem, magic);
  const auto load = [&](int slot) __attribute__((always_inline)) {  // the next tile
    lq.load(qp + (int64_t)tok * q.row, end - r0, lds + slot * kTile);
    lg.load(gp + (int64_t)tok * g.row, end - r0, lds + (2 + slot) * kTile);
    if (wave == 0) load_stats(norm + r0, end - r0, stat + slot * 512, lane);
    if (wave == (W > 1 ? 1 : 0)) load_stats(delta + r0, end - r0, stat + slot * 512 + 256, lane);
    r0 += kStep;
    tok += tok_step;
    if (rem_step != 0) {  // (uniform) tiles start inside a token
      rem += rem_step;
      if (rem >= group) {
        rem -= group;
        ++tok;
      }
      lq.place(q, a.head_dim, group, rem, magic);
      lg.place(g, a.head_dim, group, rem, magic);
    }
  };
  const float c = a.scale * kLog2e;
  f32x16_t dk[DC / 32], dv[DC / 32];
#pragma unroll
  for (int db = 0; db < DC / 32; ++db) dk[db] = dv[db] = zero16();
  const auto step = [&](int slot) __attribute__((always_inline)) {
    wait_lgkmcnt0();
    wait_vmcnt<0>();
    barrier_no_fence();
    const int r = r0 - kStep;  // (the rows of this step; r0 is the next to load)
    load(slot ^ 1);
    if constexpr (WINDOW) {
      if (!view.sees_any(r, kStep)) return;
    }
    f32x16_t s = zero16(), dp = zero16();
#pragma unroll
    for (int kk = 0; kk < DC / 16; ++kk) {
      s = mma<D>(rd.row_frag(slot * kTile, 0, kk), kf[kk], s);
      if constexpr (kParked) dp = mma<D>(rd.row_frag((2 + slot) * kTile, 0, kk), rd.row_frag(4 * kTile + own, 0, kk), dp);
      else dp = mma<D>(rd.row_frag((2 + slot) * kTile, 0, kk), vf[kk], dp);
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const float4 ls = *reinterpret_cast<const float4*>(s_stat + slot * 128 + 8 * b + 4 * (lane >> 5));
      const float4 dl = *reinterpret_cast<const float4*>(s_stat + slot * 128 + 64 + 8 * b + 4 * (lane >> 5));
      const float lse4[4] = {ls.x, ls.y, ls.z, ls.w}, del4[4] = {dl.x, dl.y, dl.z, dl.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = exp2_fast(fmaf(s[4 * b + i], c, -lse4[i]));
        s[4 * b + i] = p;
        dp[4 * b + i] = p * (dp[4 * b + i] - del4[i]);
        if constexpr (D == DT::F16) dp[4 * b + i] *= unit * p_unit;
      }
    }
    if constexpr (WINDOW) {
      if (!view.sees_all(r, kStep)) view.mask(r, lane, [&](int i) { s[i] = dp[i] = 0.f; });
    }
    // (rows past the end: q, dout, norm and d read 0, so p is 1 and meets a dout of 0, and e is 0; both in the storage
    // type, as the matrix cores take them, each off by half a step of either sign)
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const Frag<D> p = to_frag<D>(s, st), e = to_frag<D>(dp, st);
#pragma unroll
      for (int db = 0; db < DC / 32; ++db) {
        dv[db] = mma<D>(rd.column_frag((2 + slot) * kTile, st * 16, db), p, dv[db]);
        dk[db] = mma<D>(rd.column_frag(slot * kTile, st * 16, db), e, dk[db]);
      }
    }
  };
  if (steps > 0) {
    load(0);
    if constexpr (D == DT::F16 && WINDOW) {  // the largest |dout| and bound of the rows that see the own key
      const float2* one = a.row_peak + head * (a.nq * group) + q0 * group;
      const float2* blocks = a.peak + head * a.q_slots + q0 * group / a.q_rows + item;
      int from = view.from, to = view.from + (int)view.span;
      if constexpr (SINKS) from = min(max(from, row0), row_end), to = max(from, min(to, row_end));  // (of the chunk)
      const float2 top = range_max(from, to, group, a.q_rows, one, blocks, lane);
      unit = e_scale(top.x, top.y);
    }
    for (int t = 0; t < steps; t += 2) {  // (an odd end takes a step of zeros: a second exit costs registers)
      step(0);
      step(1);
    }
  }
  wait_vmcnt<0>();  // (the loads past the end)
  if constexpr (WINDOW) {
    // (64 channels and float16: what the lane's number gives is not kept over the loop)
    const int own_lane = DP == 64 || (D == DT::F16 && !SINKS) ? fresh_lane() : lane, key = tile * kKeys + wave * 32 + (own_lane & 31);
    const bool there = key < nk;
    const uint64_t odd = odd_rows<DC>(dk, there) | odd_rows<DC>(dv, there);
    if constexpr (SINKS) {
      const int64_t at = (((int64_t)head * a.sink_slots + share.slot) * a.window.sinks + key) * 2 * DP;
      if (there) {
        store_part<DC>(a.sink_part + at, dk, a.scale / unit, own_lane);
        store_part<DC>(a.sink_part + at + DP, dv, p_unit, own_lane);
      }
    } else if constexpr (CUT != kNoCut) {
      const int64_t at = ((int64_t)share.place * kKeys + wave * 32 + (own_lane & 31)) * DP;
      if (there) {
        store_part<DC>(a.dk_part + at, dk, a.scale / unit, own_lane);
        store_part<DC>(a.dv_part + at, dv, p_unit, own_lane);
      }
    } else if (there && key >= a.window.sinks) {
      store_row<D, DC>(kmap.at<D>(heads_of<D>(a.dk), key), dk, a.scale / unit, a.head_dim, own_lane);
      store_row<D, DC>(kmap.at<D>(heads_of<D>(a.dv), key), dv, p_unit, a.head_dim, own_lane);
    }
    if (odd != 0) dkv_again<D, DC, W, CUT, SINKS>(odd, unit, wave, own_lane);
    return;
  }
  if (!there) return;
  if (CUT == kCutAll || (CUT == kCutLast && share.part >= 0)) {
    const int64_t at = ((int64_t)share.place * kKeys + wave * 32 + (lane & 31)) * DP;
    store_part<DC>(a.dk_part + at, dk, a.scale / unit, lane);
    store_part<DC>(a.dv_part + at, dv, p_unit, lane);
  } else {
    store_row<D, DC>(kmap.at<D>(heads_of<D>(a.dk), key), dk, a.scale / unit, a.head_dim, lane);
    store_row<D, DC>(kmap.at<D>(heads_of<D>(a.dv), key), dv, p_unit, a.head_dim, lane);
  }
}

// dk and dv of the sinks: the sums of an item's chunks (blockIdx.x the item, y the key head, z the sink),
// DP / 2 threads a sum of both, the other groups of threads every second, fourth .. chunk.
template <DT D, int DP> __global__ __launch_bounds__(256) void attention_sink_sum_kernel(BwdArgs a) {
  constexpr int kThreads = DP / 2, kGroups = 256 / kThreads;
  __shared__ float4 s_sum[256];
  const int item = blockIdx.x, head = blockIdx.y, key = blockIdx.z, group = a.heads / a.kv_heads;
  int64_t q0, k0;
  int nq, nk;
  item_rows(a.q_offsets, a.nq, item, &q0, &nq);
  item_rows(a.k_offsets, a.nk, item, &k0, &nk);
  if (key >= nk) return;
  const int chunks = (int)(((int64_t)nq * group + a.sink_rows - 1) / a.sink_rows);
  const int64_t first = (int64_t)head * a.sink_slots + q0 * group / a.sink_rows + item;
  const int at = threadIdx.x % kThreads * 4, mine = threadIdx.x / kThreads;
  const float* part = a.sink_part + (first * a.window.sinks + key) * 2 * DP + at;
  const int64_t step = (int64_t)a.window.sinks * 2 * DP;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = mine; s < chunks; s += kGroups) {
    const float4 p = *reinterpret_cast<const float4*>(part + s * step);
    o.x += p.x;
    o.y += p.y;
    o.z += p.z;
    o.w += p.w;
  }
  s_sum[threadIdx.x] = o;
  __syncthreads();
  if (mine != 0) return;
#pragma unroll
  for (int s = 1; s < kGroups; ++s) {
    const float4 p = s_sum[s * kThreads + threadIdx.x];
    o.x += p.x;
    o.y += p.y;
    o.z += p.z;
    o.w += p.w;
  }
  const int c = at % DP;
  if (c >= a.head_dim) return;
  const Heads<D> out = heads_of<D>(at < DP ? a.dk : a.dv);
  store4<D>(out.data + (k0 + key) * out.row + (int64_t)head * out.head + c, o.x, o.y, o.z, o.w);
}

// The sums of tiles in parts (blockIdx.x of those), DP / 4 threads a row, blockIdx.y the rows of
// the tile; blockIdx.z 0 is dq, 1 dk and 2 dv.
template <DT D, int DP>
__global__ __launch_bounds__(256) void attention_sum_kernel(BwdArgs a, int q_rows, int k_rows) {
  constexpr int kThreads = DP / 4;
  const int job = a.dq_part != nullptr ? blockIdx.z : blockIdx.z + 1;
  const Cut cut = job == 0 ? a.q_cut : a.k_cut;
  const int tile_rows = job == 0 ? q_rows : k_rows, group = job == 0 ? a.heads / a.kv_heads : 1, parts = cut.parts;
  const int64_t step = (int64_t)tile_rows * DP;
  if ((int)blockIdx.x >= cut.cut) return;
  const Share share = tile_share(cut, blockIdx.x);
  const int64_t* offsets = job == 0 ? a.q_offsets : a.k_offsets;
  const int64_t total = job == 0 ? a.nq : a.nk;
  int tile, count;
  const int item = find_item(offsets, total, a.items, group, tile_rows, share.slot, &tile);
  int64_t first;
  item_rows(offsets, total, item, &first, &count);
  const RowMap map{first, share.head * group, group};
  const Heads<D> out = heads_of<D>(job == 0 ? a.dq : job == 1 ? a.dk : a.dv);
  const float* all = job == 0 ? a.dq_part : job == 1 ? a.dk_part : a.dv_part;
  const int c = threadIdx.x % kThreads * 4;
  if (c >= a.head_dim) return;
  const int r = blockIdx.y * (256 / kThreads) + threadIdx.x / kThreads;
  const int64_t row = (int64_t)tile * tile_rows + r;
  if (r >= tile_rows || row >= (int64_t)count * group) return;
  const float* part = all + ((int64_t)share.place * tile_rows + r) * DP + c;
  float4 o = *reinterpret_cast<const float4*>(part);
#pragma unroll 8
  for (int s = 1; s < parts; ++s) {
    const float4 p = *reinterpret_cast<const float4*>(part + s * step);
    o.x += p.x;
    o.y += p.y;
    o.z += p.z;
    o.w += p.w;
  }
  store4<D>(map.at<D>(out, (int)row) + c, o.x, o.y, o.z, o.w);
}

template <DT D, int DC, int W, int CUT, bool WINDOW> hipError_t launch_dq(const BwdArgs& a, hipStream_t stream) {
  constexpr int OCC = D == DT::F32 ? 1 : DC <= 64 ? 3 : 2;
  const dim3 grid =
      CUT == kNoCut ? dim3((unsigned)a.q_cut.slots, (unsigned)a.kv_heads) : dim3((unsigned)cut_blocks(a.q_cut));
  attention_dq_kernel<D, DC, W, OCC, CUT, WINDOW><<<grid, W * 64, 0, stream>>>(a);
  return hipGetLastError();
}
template <DT D, int DC, int W, int CUT, bool WINDOW> hipError_t launch_dkv(const BwdArgs& a, hipStream_t stream) {
  constexpr int OCC = D == DT::F32 ? 1 : DC <= 64 ? 3 : 2;
  const dim3 grid =
      CUT == kNoCut ? dim3((unsigned)a.k_cut.slots, (unsigned)a.kv_heads) : dim3((unsigned)cut_blocks(a.k_cut));
  attention_dkv_kernel<D, DC, W, OCC, CUT, WINDOW, false><<<grid, W * 64, 0, stream>>>(a);
  return hipGetLastError();
}

// The cuts that plan_cut can give: of 8 waves' tiles, which fill the machine, the last; of 4 waves'
// at 128 channels in 16 bits all (if they filled it, their items would be too short).
template <DT D, int DC, int W, bool WINDOW> hipError_t launch_dq(const BwdArgs& a, hipStream_t stream) {
  constexpr bool kFull = D != DT::F32 && tile_width(DC) == 128;
  if constexpr (!WINDOW && (W == 8 || !kFull)) {
    if (a.q_cut.parts > 1 && a.q_cut.whole > 0) return launch_dq<D, DC, W, kCutLast, WINDOW>(a, stream);
  }
  if constexpr (W == 4) {
    if (a.q_cut.parts > 1) return launch_dq<D, DC, W, kCutAll, WINDOW>(a, stream);
  }
  return launch_dq<D, DC, W, kNoCut, WINDOW>(a, stream);
}
template <DT D, int DC, int W, bool WINDOW> hipError_t launch_dkv(const BwdArgs& a, hipStream_t stream) {
  constexpr bool kFull = D != DT::F32 && tile_width(DC) == 128;
  if constexpr (!WINDOW && (W == 8 || !kFull)) {
    if (a.k_cut.parts > 1 && a.k_cut.whole > 0) return launch_dkv<D, DC, W, kCutLast, WINDOW>(a, stream);
  }
  if constexpr (W == 4) {
    if (a.k_cut.parts > 1) return launch_dkv<D, DC, W, kCutAll, WINDOW>(a, stream);
  }
  return launch_dkv<D, DC, W, kNoCut, WINDOW>(a, stream);
}

template <DT D, int DC, bool WINDOW>
Status launch(BwdArgs a, hipStream_t stream) {
  constexpr int DP = tile_width(DC), kUnits = 256;
  const int group = a.heads / a.kv_heads;
  const int64_t rows = a.nq * group, spare = (int64_t)a.items * a.kv_heads;
  // 128 channels in 16 bits: 8 waves share a tile stream where they fill the compute units.
  constexpr bool kWide = D != DT::F32 && DP == 128 && !WINDOW;
  const bool wide_q = kWide && (rows / 256 + a.items) * a.kv_heads >= kUnits && rows / a.items >= 256;
  const bool wide_k = kWide && (a.nk / 256 + a.items) * a.kv_heads >= kUnits && a.nk / a.items >= 256;
  const int q_rows = wide_q ? 256 : 128, k_rows = wide_k ? 256 : 128;
  // Parts, measured (forward and backward): 7,813 tokens, 12 / 4 heads of 64, f16: 451 us whole, 368
  // with 4 workgroups a unit, 376 with 3 or 6; 3,000 tokens, 12 heads of 128, bf16: 337 us with 2,
  // 345 with 4, 385 with 3; 800 tokens, 8 heads of 64: 41.8 us with parts of 128 rows, 46.8 with 256.
  // float32 waves are slow and one a SIMD: one workgroup a unit, whatever is left to each (265
  // queries, 304 keys in two items, 16 heads of 80: 90 us, 135 with at least 96 rows).
  constexpr int kFew = kUnits * (D == DT::F32 ? 1 : DP == 64 ? 4 : 2), kLeast = D == DT::F32 ? 32 : 128;
  constexpr int kResident = kWide ? INT32_MAX : kUnits * (D == DT::F32 ? 1 : 3);  // of 4 waves
  a.q_rows = q_rows;
  a.q_slots = rows / q_rows + a.items;
  constexpr double kLess = kWide ? kGainAt128 : kGain;
  const int64_t k_slots = a.nk / k_rows + a.items;
  const int64_t q_full = wide_q ? kUnits : kResident, k_full = wide_k ? kUnits : kResident;
  if constexpr (WINDOW) {
    const int64_t q_walks = a.window.walked(a.nk / a.items, q_rows / group);
    const int64_t k_walks = a.window.walked(a.nq / a.items, k_rows) * group;
    a.window.runs = a.window.in_runs(a.nk / a.items, group);
    constexpr int64_t kSlots = kUnits * (D == DT::F32 ? 1 : DP == 64 ? 3 : 2);
    a.q_cut = plan_window_cut(a.window, a.q_slots, a.kv_heads, a.nk / a.items, q_walks, kLeast, kSlots, kFew);
    a.k_cut = plan_window_cut(a.window, k_slots, a.kv_heads, a.nq / a.items, k_walks, kLeast, kSlots, kFew);
  } else {
    a.q_cut = plan_cut(a.q_slots, a.kv_heads, spare, a.nk / a.items, kLeast, q_full, kFew, kLess);
    a.k_cut = plan_cut(k_slots, a.kv_heads, spare, rows / a.items, kLeast, k_full, kFew, kLess);
  }
  const bool sinks = WINDOW && a.window.sinks > 0 && a.nk > 0;
  if (sinks) {  // chunks for four waves a unit
    const int blocks = (a.window.sinks + 31) / 32;
    const int64_t chunk = rows * a.kv_heads * blocks / (kUnits * 4);
    a.sink_rows = (int)std::min<int64_t>(std::max<int64_t>(chunk, 128), 8192) / group * group;
    a.sink_slots = rows / a.sink_rows + a.items;
  }

  int dev = 0;
  SUBM_HIP_TRY(hipGetDevice(&dev));
  ScratchLease lease;
  const auto padded = [](size_t bytes) { return (bytes + 255) / 256 * 256; };
  // norm and d of every query row, peaks of query and key blocks, and the parts
  const size_t stat = padded((size_t)rows * a.kv_heads * sizeof(float));
  a.v_slots = a.nk / kNormKeys + a.items;
  const size_t peak = D == DT::F16 ? padded((size_t)a.q_slots * a.kv_heads * sizeof(float2)) : 0;
  const size_t norm = D == DT::F16 ? padded((size_t)a.v_slots * a.kv_heads * sizeof(float)) : 0;
  constexpr bool kEach = D == DT::F16 && WINDOW;
  const size_t row_peak = kEach ? padded((size_t)rows * a.kv_heads * sizeof(float2)) : 0;
  const size_t key_norm = kEach ? padded((size_t)a.nk * a.kv_heads * sizeof(float)) : 0;
  const size_t part_q = (size_t)cut_places(a.q_cut) * q_rows * DP * sizeof(float);
  const size_t part_k = (size_t)cut_places(a.k_cut) * k_rows * DP * sizeof(float);
  void* scratch = nullptr;
  const size_t part_s = sinks ? (size_t)a.sink_slots * a.kv_heads * a.window.sinks * 2 * DP * sizeof(float) : 0;
  Status st = lease.take(dev, stream, 2 * stat + peak + norm + row_peak + key_norm + part_q + 2 * part_k + part_s, &scratch);
  if (!st.ok()) return st;
  unsigned char* p = static_cast<unsigned char*>(scratch);
  a.norm = reinterpret_cast<float*>(p);
  a.delta = reinterpret_cast<float*>(p + stat);
  a.peak = reinterpret_cast<float2*>(p + 2 * stat);
  a.v_norm = reinterpret_cast<float*>(p + 2 * stat + peak);
  p += 2 * stat + peak + norm;
  a.row_peak = reinterpret_cast<float2*>(p);
  a.key_norm = reinterpret_cast<float*>(p + row_peak);
  p += row_peak + key_norm;
  if (part_q > 0) a.dq_part = reinterpret_cast<float*>(p);
  if (part_k > 0) {
    a.dk_part = reinterpret_cast<float*>(p + part_q);
    a.dv_part = reinterpret_cast<float*>(p + part_q + part_k);
  }
  a.sink_part = reinterpret_cast<float*>(p + part_q + 2 * part_k);
  if constexpr (D == DT::F16) {
    if (a.nk > 0) {
      attention_norm_kernel<D, WINDOW><<<dim3((unsigned)a.v_slots, (unsigned)a.kv_heads), 256, 0, stream>>>(a);
      SUBM_HIP_TRY(hipGetLastError());
    }
  }
  if (a.nq > 0) {
    if constexpr (kWide) {
      if (wide_q) SUBM_HIP_TRY((launch_dq<D, DC, 8, WINDOW>(a, stream)));
    }
    if (!wide_q) SUBM_HIP_TRY((launch_dq<D, DC, 4, WINDOW>(a, stream)));
  }
  if (a.nk > 0) {
    if constexpr (kWide) {
      if (wide_k) SUBM_HIP_TRY((launch_dkv<D, DC, 8, WINDOW>(a, stream)));
    }
    if (!wide_k) SUBM_HIP_TRY((launch_dkv<D, DC, 4, WINDOW>(a, stream)));
  }
  const unsigned jobs = (part_q > 0 ? 1 : 0) + (part_k > 0 ? 2 : 0);
  if (jobs > 0) {
    const dim3 grid((unsigned)std::max(a.q_cut.cut, a.k_cut.cut), std::max(q_rows, k_rows) * (DP / 4) / 256, jobs);
    attention_sum_kernel<D, DP><<<grid, 256, 0, stream>>>(a, q_rows, k_rows);
    SUBM_HIP_TRY(hipGetLastError());
  }
  if constexpr (WINDOW) {
    if (sinks) {
      a.k_cut = Cut{(int)a.sink_slots, 0, 0, 1, false};
      if (a.nq > 0) {
        const dim3 grid((unsigned)a.sink_slots, (unsigned)a.kv_heads, (unsigned)((a.window.sinks + 31) / 32));
        attention_dkv_kernel<D, DC, 1, 1, kNoCut, true, true><<<grid, 64, 0, stream>>>(a);
        SUBM_HIP_TRY(hipGetLastError());
      }
      attention_sink_sum_kernel<D, DP><<<dim3((unsigned)a.items, (unsigned)a.kv_heads, (unsigned)a.window.sinks), 256, 0, stream>>>(a);
      SUBM_HIP_TRY(hipGetLastError());
    }
  }
  return Status{};
}

template <DT D, bool WINDOW> Status launch_dim(const BwdArgs& a, hipStream_t stream) {
  if (a.head_dim <= 32) return launch<D, 32, WINDOW>(a, stream);
  if (a.head_dim <= 64) return launch<D, 64, WINDOW>(a, stream);
  if (a.head_dim <= 96) return launch<D, 96, WINDOW>(a, stream);
  return launch<D, 128, WINDOW>(a, stream);
}

BwdArgs backward_args(const subm_heads_t* dout, const subm_heads_t* q, const subm_heads_t* k, const subm_heads_t* v,
                      const subm_heads_t* out, const float* lse, const subm_heads_t* dq, const subm_heads_t* dk,
                      const subm_heads_t* dv, const AttentionShape& s) {
  BwdArgs a{};
  a.dout = *dout;
  a.q = *q;
  a.k = *k;
  a.v = *v;
  a.out = *out;
  a.dq = *dq;
  a.dk = *dk;
  a.dv = *dv;
  a.lse = lse;
  a.q_offsets = s.q_offsets;
  a.k_offsets = s.k_offsets;
  a.nq = s.nq;
  a.nk = s.nk;
  a.items = s.items;
  a.heads = s.heads;
  a.kv_heads = s.kv_heads;
  a.head_dim = s.head_dim;
  a.scale = s.scale;
  return a;
}

}  // namespace
}  // namespace submconv
