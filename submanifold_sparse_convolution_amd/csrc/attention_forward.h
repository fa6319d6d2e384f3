// The forward kernels of attention, for whole items (attention.hip) and for windows of them
// (window_attention.hip), and their launches.
#pragma once

#include <algorithm>
#include <cmath>

#include "attention_common.h"
#include "attention_window.h"

namespace submconv {
namespace {

struct FwdArgs {
  subm_heads_t q, k, v, out;
  float* lse;
  const int64_t *q_offsets, *k_offsets;
  int64_t nq, nk;
  int items, heads, kv_heads, head_dim;
  float scale;
  // Tiles in parts: what a part leaves, [place][rows of a tile][DP] unnormalised sums and their
  // (base, sum).
  Cut cut;
  float* part;
  float2* state;
  Window window;  // of the kernels with WINDOW
};

// (fmaxf would first quiet every operand)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// Keeps the values computed here: the compiler would sink them past the next branch, away from the
// matrix products that they overlap with.
template <DT D> __device__ __forceinline__ void pin(Frag<D>& f) {
#pragma unroll
  for (int i = 0; i < Elem<D>::kSize / 2; ++i)
    asm volatile("" : "+v"(f.v[i].x), "+v"(f.v[i].y), "+v"(f.v[i].z), "+v"(f.v[i].w));
}

constexpr float kNone = -1.7e38f;  // a running maximum before any score (finite: differences stay numbers)

// The running softmax of one own row (held by the lanes l and l + 32, half its scores each):
// scores are kept as c * s - base in powers of two; base is a maximum, less kLift, that may lag behind
// the true one by kSlack, so that most tiles do not rescale the accumulator.  p stays below
// 2^(kLift + kSlack), which the storage type holds.  float16 rounds what is below 2^-25 to zero, and
// thousands of such keys beside one large score are not nothing (60,000 at 2^-25.5 of it are a
// thousandth): there p starts from 2^11, and what vanishes is below 2^-36 of the largest.
template <DT D> constexpr float kLift = D == DT::F16 ? 11.f : 0.f;
template <DT D> constexpr float kSlack = D == DT::F16 ? 4.f : 8.f;
struct RowState {
  float base = kNone;
  float sum = 0.f;  // of this lane's half
};

// Scores (raw) -> probabilities in place; returns the factor that earlier sums shrink by, and
// whether any row of the wave does shrink.  All rows of the wave take their maximum then; with WINDOW each by
// itself, so that what it does not see has no part in its roundings either.
template <DT D, int KB, bool WINDOW>
__device__ __forceinline__ bool softmax_tile(f32x16_t (&s)[KB], float c, RowState& st, float* shrink) {
  float top = s[0][0];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 16; i += 2) top = max3(top, s[kb][i], s[kb][i + 1]);
  top = half_max(top);
  top = kLift<D> == 0.f ? top * c : fmaf(top, c, -kLift<D>);
  const bool rises = top > st.base + kSlack<D>, moves = __builtin_amdgcn_ballot_w64(rises) != 0;
  // (a gate instead of a branch, which would part the matrix products from the exponentials)
  const float base = WINDOW ? (rises ? top : st.base) : fmaxf(st.base, top + (moves ? 0.f : -INFINITY));
  *shrink = exp2_fast(st.base - base);
  st.base = base;
  float sum = 0.f;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[kb][i] = exp2_fast(fmaf(s[kb][i], c, -base));
      sum += s[kb][i];
    }
  st.sum = fmaf(st.sum, *shrink, sum);
  return moves;
}

// The rows `odd` of a wave's accumulators key by key: see attention_window.h.  (From the kernel's arguments
// on, so that nothing of it is kept in registers over the loop.)
template <DT D, int DC, int W, int KEYS, int CUT>
__device__ __forceinline__ void forward_again(f32x16_t (&acc)[DC / 32], uint64_t odd, float base, float c, int wave, int lane) {
  const FwdArgs a = fresh_args<FwdArgs>();
  const int group = a.heads / a.kv_heads;
  const Share share = window_share<CUT>(a.cut, a.window, true);
  int tile;
  const int item = find_item(a.q_offsets, a.nq, a.items, group, 32 * W, share.slot, &tile);
  int64_t q0, k0;
  int nq, nk;
  item_rows(a.q_offsets, a.nq, item, &q0, &nq);
  item_rows(a.k_offsets, a.nk, item, &k0, &nk);
  nk = a.window.keys(item, nk);
  const int first = tile * 32 * W, last = min(nq * group, first + 32 * W) - 1;
  const RowMap qmap{q0, share.head * group, group};
  const Heads<D> q = heads_of<D>(a.q), k = heads_of<D>(a.k), v = heads_of<D>(a.v);
  const typename Elem<D>::T* kp = k.data + k0 * k.row + (int64_t)share.head * k.head;
  const typename Elem<D>::T* vp = v.data + k0 * v.row + (int64_t)share.head * v.head;
  KeyTiles<KEYS> walk;
  walk.place(a.window, nk, nk - nq, first / group, last / group);
  if constexpr (CUT != kNoCut) {
    int tiles = walk.tiles;
    const int from = part_steps(a.cut, share.part, &tiles);
    walk.cut(from, tiles);
  }
  for (; odd != 0; odd &= odd - 1) {
    const int l = __builtin_ctzll(odd), row = first + wave * 32 + l, p = row / group + nk - nq;
    if (!hidden_odd<D>(a.window, walk, p, nk, vp, v.row, a.head_dim, lane)) continue;
    const float2 qr = row_pair<D>(qmap.at<D>(q, row), a.head_dim, lane);
    const float b = lane_value(base, l);
    const float2 was = take_row<DC>(acc, l, a.head_dim, lane);
    float2 o = make_float2(0.f, 0.f);
    for (int t = 0; t < walk.tiles && still_finite(was, o); ++t)
      for (int j = walk.key(t); j < min(walk.key(t) + KEYS, walk.end(t)); ++j) {
        if (!a.window.sees(p, j)) continue;
        const float s = pair_dot(qr, row_pair<D>(kp + (int64_t)j * k.row, a.head_dim, lane));
        const float e = exp2_fast(fmaf(s, a.scale < 0.f ? -c : c, -b));
        add_scaled(o, to_float<D>(from_float<D>(e)), row_pair<D>(vp + (int64_t)j * v.row, a.head_dim, lane));
      }
    put_row<DC>(acc, mended(was, o), l, lane);
  }
}

// Streams the keys through LDS in tiles of KEYS, two of k and two of v; one step of the loop holds
// three independent pieces of work, so that the matrix cores run while the exponentials do:
//   scores of tile t + 1 (k),  softmax of tile t,  product of tile t - 1 (v).
// (Four tiles of each in flight: the same time.)
//
// KG > 1: that many groups of W waves hold the same rows and take every KG-th tile of keys, joined through
// LDS at the end: where a compute unit gets one workgroup, a lone wave a SIMD would wait for each
// instruction's result in turn; and few rows are one wave's.
//
// WINDOW: each row sees a range of keys and the first `sinks`.  The tiles are those of the sinks and those
// from the first key to the last that one of the tile's rows sees; scores are masked in the tiles that some
// row of the wave does not see whole.
template <DT D, int DC, int W, int KG, int KEYS, int OCC, int CUT, bool WINDOW>
__global__ __launch_bounds__(KG * W * 64, OCC) void attention_forward_kernel(FwdArgs a) {
  constexpr int DP = tile_width(DC), KB = KEYS / 32;
  constexpr int kTile = KEYS * kRowBytes<D, DP>;
  constexpr int kRows = 32 * W;
  using Loader = TileLoader<D, DP, KEYS, W>;
  __shared__ __attribute__((aligned(1024))) unsigned char s_kv[KG * 4 * kTile];
  __shared__ float2 s_join[KG == 1 ? 1 : (KG - 1) * W * 64];
  const int lane = threadIdx.x & 63, every = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = KG == 1 ? 0 : every / W, wave = KG == 1 ? every : every % W;
  const int group = a.heads / a.kv_heads;
  const Share share = WINDOW ? window_share<CUT>(a.cut, a.window, true) : share_of<CUT>(a.cut, blockIdx.x);
  const int head = share.head;
  int item, tile, nq, nk;
  int64_t q0, k0;
  if constexpr (WINDOW) {
    const Item it = find_rows(a, a.window, group, kRows, share.slot);
    item = it.index, tile = it.tile, q0 = it.q0, nq = it.nq, k0 = it.k0, nk = it.nk;
  } else {
    item = find_item(a.q_offsets, a.nq, a.items, group, kRows, share.slot, &tile);
    item_rows(a.q_offsets, a.nq, item, &q0, &nq);
    item_rows(a.k_offsets, a.nk, item, &k0, &nk);
  }
  const int rows = nq * group;
  if ((int64_t)tile * kRows >= rows) return;
  const RowMap qmap{q0, head * group, group};
  const Heads<D> q = heads_of<D>(a.q), k = heads_of<D>(a.k), v = heads_of<D>(a.v), out = heads_of<D>(a.out);
  const typename Elem<D>::T* kp = k.data + k0 * k.row + (int64_t)head * k.head;
  const typename Elem<D>::T* vp = v.data + k0 * v.row + (int64_t)head * v.head;

  const int row = tile * kRows + wave * 32 + (lane & 31);
  const bool there = row < rows;
  Frag<D> qf[DC / 16];
  const typename Elem<D>::T* qrow = qmap.at<D>(q, there ? row : 0);
  // a negative scale goes into q, so that the largest score is the largest product
  const uint32_t flip = a.scale < 0.f ? (D == DT::F32 ? 0x80000000u : 0x80008000u) : 0u;
  const auto flip_frag = [&](Frag<D>& f) {
#pragma unroll
    for (int i = 0; i < Elem<D>::kSize / 2; ++i) {
      f.v[i].x ^= flip;
      f.v[i].y ^= flip;
      f.v[i].z ^= flip;
      f.v[i].w ^= flip;
    }
  };
#pragma unroll
  for (int kk = 0; kk < DC / 16; ++kk) {
    qf[kk] = own_frag<D>(qrow, there, kk, a.head_dim, lane);
    if constexpr (!WINDOW) flip_frag(qf[kk]);
  }
  // (a scale of 0 becomes tiny: a key past the end must still score -infinity)
  const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);

  Loader lk, lv;
  lk.wave = lv.wave = wave;
  lk.lane = lv.lane = lane;
  lk.place(k, a.head_dim, 1, 0, 0);
  lv.place(v, a.head_dim, 1, 0, 0);
  const uint32_t lds = lds_offset(s_kv) + part * 4 * kTile;
  const TileReader<D, DP> rd(lane, lds, lds + 2 * kTile);
  // this workgroup's keys: all, or its share of whole tiles (a share may be empty)
  int tiles = (nk + KEYS - 1) / KEYS, left = nk;
  KeyTiles<KEYS> walk;
  RowView view;
  if constexpr (WINDOW) {
    const int first = tile * kRows, last = min(rows, first + kRows) - 1;
    walk.place(a.window, nk, nk - nq, first / group, last / group);
    view.place(a.window, nk, nk - nq, min(row, last) / group, min(first + wave * 32, last) / group,
               min(first + wave * 32 + 31, last) / group);
    tiles = walk.tiles;
  }
  if constexpr (CUT != kNoCut) {
    const int first = part_steps(a.cut, share.part, &tiles);
    if constexpr (WINDOW) {
      walk.cut(first, tiles);
    } else {
      left = min(nk - first * KEYS, tiles * KEYS);
      kp += (int64_t)first * KEYS * k.row;
      vp += (int64_t)first * KEYS * v.row;
    }
  }
  // (t counts this part's tiles; t and slot apart: inside the loop the slot is a constant)
  const auto load_k = [&](int t, int slot) {
    if constexpr (WINDOW) {
      const int key = walk.key(t * KG + part);
      lk.load(kp + (int64_t)key * k.row, walk.end(t * KG + part) - key, lds + slot * kTile);
    } else {
      const int key = (t * KG + part) * KEYS;
      lk.load(kp + (int64_t)key * k.row, left - key, lds + slot * kTile);
    }
  };
  const auto load_v = [&](int t, int slot) {
    if constexpr (WINDOW) {
      const int key = t < 0 ? 0 : walk.key(t * KG + part);
      lv.load(vp + (int64_t)key * v.row, t < 0 ? 0 : walk.end(t * KG + part) - key, lds + (2 + slot) * kTile);
    } else {
      const int key = (t * KG + part) * KEYS;
      lv.load(vp + (int64_t)key * v.row, t < 0 ? 0 : left - key, lds + (2 + slot) * kTile);
    }
  };
  const auto scores = [&](int slot, f32x16_t (&s)[KB]) {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      s[kb] = zero16();
#pragma unroll
      for (int kk = 0; kk < DC / 16; ++kk) s[kb] = mma<D>(rd.row_frag(slot * kTile, kb * 32, kk), qf[kk], s[kb]);
    }
  };
  f32x16_t acc[DC / 32];
#pragma unroll
  for (int db = 0; db < DC / 32; ++db) acc[db] = zero16();
  const auto product = [&](int slot, const Frag<D> (&p)[2 * KB]) {
#pragma unroll
    for (int st = 0; st < 2 * KB; ++st)
#pragma unroll
      for (int db = 0; db < DC / 32; ++db) acc[db] = mma<D>(rd.column_frag(slot * kTile, st * 16, db), p[st], acc[db]);
  };

  RowState state;
  if (tiles > 0) {
    // Step t reads k of tile t + 1 and v of tile t - 1 and starts the loads of k of tile t + 2 and
    // v of tile t, whose slots step t - 1 read last.  v of tile -1 is zeros.
    load_k(0, 0);
    load_k(1, 1);
    load_v(-1, 1);
    if constexpr (WINDOW) {  // (short walks: not before the first tiles are on their way)
#pragma unroll
      for (int kk = 0; kk < DC / 16; ++kk) flip_frag(qf[kk]);
    }
    wait_vmcnt<2 * Loader::N>();
    barrier_no_fence();
    f32x16_t s0[KB], s1[KB];
    Frag<D> p[2 * KB];
#pragma unroll
    for (int st = 0; st < 2 * KB; ++st)
#pragma unroll
      for (int i = 0; i < Elem<D>::kSize / 2; ++i) p[st].v[i] = make_uint4(0, 0, 0, 0);
    scores(0, s0);
    // WINDOW: whether the wave sees any key of tile t - 1 (was), t (now) and t + 1 (soon).  It leaves out the
    // steps without any: what it holds of such tiles is masked, and their p is 0, before a step reads it.  In
    // float32, whose products are slow (2,000 tokens, 6 / 3 heads of 80, causal: 121 -> 110 us), and at 64 channels, where
    // vector instructions weigh most (four items, 9,371 tokens, 12 heads, 256 keys each way: 54 -> 44 us), of whole tiles alone:
    // elsewhere the branch costs as much (24,576 tokens, 16 heads of 128: 431 us, 437 with it).
    constexpr bool kSkip = WINDOW && KG == 1 && (D == DT::F32 || (DP == 64 && CUT == kNoCut));
    bool was = false, now = true;
    if constexpr (kSkip) now = view.sees_any(walk.key(0), KEYS, walk.end(0));
    const auto step = [&](int t, int slot, f32x16_t (&s)[KB], f32x16_t (&next)[KB]) {
      wait_lgkmcnt0();  // this wave's reads of the slots that are about to be loaded have returned
      wait_vmcnt<0>();
      barrier_no_fence();
      load_k(t + 2, slot);
      load_v(t, slot);
      if constexpr (WINDOW) {
        const int tt = t * KG + part, key = walk.key(tt), end = walk.end(tt);
        if constexpr (kSkip) {
          const bool soon = view.sees_any(walk.key(tt + 1), KEYS, walk.end(tt + 1)), any = was || now || soon;
          was = now;
          now = soon;
          if (!any) return;
        }
        if (!view.sees_all(key, KEYS, end))
          view.template mask<KB>(key, end, lane, [&](int kb, int i) { s[kb][i] = -INFINITY; });
      } else {
        const int key = (t * KG + part) * KEYS;
        if (key + KEYS > left) {  // keys past the end (perhaps all)
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (key + kb * 32 + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3) >= left) s[kb][i] = -INFINITY;
        }
      }
      scores(slot ^ 1, next);
      float shrink;
      const bool moves = softmax_tile<D, KB, WINDOW>(s, c, state, &shrink);
      product(slot ^ 1, p);
      // (p in the storage type, as the matrix cores take it: each off by half a step, of either sign, while the sum
      // that divides has all 32 bits; outputs are 1.2 to 1.45 times as far from 64 bits as one rounding leaves them)
#pragma unroll
      for (int st = 0; st < 2 * KB; ++st) {
        p[st] = to_frag<D>(s[st / 2], st % 2);
        pin<D>(p[st]);
      }
      if (moves) {
#pragma unroll
        for (int db = 0; db < DC / 32; ++db)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[db][i] *= shrink;
      }
    };
    const int steps = (tiles + KG - 1) / KG;
    for (int t = 0;;) {
      step(t, 0, s0, s1);
      if (++t == steps) break;
      step(t, 1, s1, s0);
      if (++t == steps) break;
    }
    wait_lgkmcnt0();
    wait_vmcnt<0>();
    barrier_no_fence();
    product((steps - 1) % 2, p);
  }
  float sum = half_sum(state.sum);
  if constexpr (KG > 1) {
    constexpr int kArea = DC / 32 * 4096;
    static_assert((KG - 1) * W * kArea <= KG * 4 * kTile, "the tiles make room");
    const uint32_t at = lds_offset(s_kv) + wave * kArea;
    wait_lgkmcnt0();
    __syncthreads();  // (every part is done with its tiles)
    if (part > 0) {
      put_acc<DC>(at + (part - 1) * W * kArea, acc, lane);
      s_join[((part - 1) * W + wave) * 64 + lane] = make_float2(state.base, sum);
    }
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int o = 0; o < KG - 1; ++o) {
      const float2 other = s_join[(o * W + wave) * 64 + lane];
      const float base = fmaxf(state.base, other.x);
      const float mine = exp2_fast(state.base - base), theirs = exp2_fast(other.x - base);
      add_acc<DC>(at + o * W * kArea, acc, mine, theirs, lane);
      sum = fmaf(other.y, theirs, sum * mine);
      state.base = base;
    }
  }
  if constexpr (WINDOW) {
    const uint64_t odd = odd_rows<DC>(acc, there && __builtin_isfinite(sum));
    if (odd != 0) forward_again<D, DC, W, KEYS, CUT>(acc, odd, state.base, c, wave, lane);
  }
  if (!there) return;
  if (CUT == kCutAll || (CUT == kCutLast && share.part >= 0)) {
    const int64_t at = (int64_t)share.place * kRows + wave * 32 + (lane & 31);
    if (lane < 32) a.state[at] = make_float2((WINDOW ? tiles > 0 : nk > 0) ? state.base : -INFINITY, sum);
    if (tiles == 0) return;
    float* o = a.part + at * DP;
#pragma unroll
    for (int db = 0; db < DC / 32; ++db)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(o + db * 32 + 8 * i + 4 * (lane >> 5)) =
            make_float4(acc[db][4 * i], acc[db][4 * i + 1], acc[db][4 * i + 2], acc[db][4 * i + 3]);
    return;
  }
  const bool some = WINDOW ? sum != 0.f : tiles > 0;
  store_row<D, DC>(qmap.at<D>(out, row), acc, some ? 1.f / sum : 0.f, a.head_dim, lane);
  if (a.lse != nullptr && lane < 32)
    a.lse[qmap.stat(row, a.heads)] = some ? (state.base + log2f(sum)) * kLn2 : -INFINITY;
}

// Joins the parts of a tile (blockIdx.x of those in parts), DP / 4 threads a row, blockIdx.y the
// rows of the tile.
template <DT D, int DP, int W, bool WINDOW>
__global__ __launch_bounds__(256) void attention_join_kernel(FwdArgs a) {
  constexpr int kThreads = DP / 4, kRows = 32 * W;
  const int group = a.heads / a.kv_heads, parts = a.cut.parts;
  const Share share = tile_share(a.cut, blockIdx.x);
  int item, tile, nq;
  int64_t q0;
  if constexpr (WINDOW) {
    const Item it = find_rows(a, a.window, group, kRows, share.slot);
    item = it.index, tile = it.tile, q0 = it.q0, nq = it.nq;
  } else {
    item = find_item(a.q_offsets, a.nq, a.items, group, kRows, share.slot, &tile);
    item_rows(a.q_offsets, a.nq, item, &q0, &nq);
  }
  const int rows = nq * group;
  const RowMap qmap{q0, share.head * group, group};
  const Heads<D> out = heads_of<D>(a.out);
  const int c = threadIdx.x % kThreads * 4;
  const int r = blockIdx.y * (256 / kThreads) + threadIdx.x / kThreads;
  const int64_t row = (int64_t)tile * kRows + r;
  if (row >= rows) return;
  const int64_t first = (int64_t)share.place * kRows + r;
  // The parts in batches, every load of a batch in flight at once, joined as a running softmax.
  constexpr int kBatch = 8;
  float base = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < parts; s0 += kBatch) {
    float2 st[kBatch];
    float4 p[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t at = first + (int64_t)min(s0 + i, parts - 1) * kRows;
      st[i] = a.state[at];
      p[i] = *reinterpret_cast<const float4*>(a.part + at * DP + c);
    }
    float top = base;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) top = fmaxf(top, st[i].x);
    if (top == -INFINITY) continue;  // (no keys: the same in every part)
    const float shrink = exp2_fast(base - top);
    base = top;
    sum *= shrink;
    o.x *= shrink;
    o.y *= shrink;
    o.z *= shrink;
    o.w *= shrink;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      // a share without keys has a sum of 0 and wrote no part
      const bool some = s0 + i < parts && st[i].y != 0.f;
      const float w = some ? exp2_fast(st[i].x - base) : 0.f;
      sum = fmaf(w, some ? st[i].y : 0.f, sum);
      o.x = fmaf(w, some ? p[i].x : 0.f, o.x);
      o.y = fmaf(w, some ? p[i].y : 0.f, o.y);
      o.z = fmaf(w, some ? p[i].z : 0.f, o.z);
      o.w = fmaf(w, some ? p[i].w : 0.f, o.w);
    }
  }
  const bool none = base == -INFINITY || (WINDOW && sum == 0.f);  // the item has no keys, or the row sees none
  const float f = none ? 0.f : 1.f / sum;
  if (c < a.head_dim) store4<D>(qmap.at<D>(out, (int)row) + c, o.x * f, o.y * f, o.z * f, o.w * f);
  if (a.lse != nullptr && c == 0) a.lse[qmap.stat((int)row, a.heads)] = none ? -INFINITY : (base + log2f(sum)) * kLn2;
}

// The same for few rows in many parts: a workgroup a row (blockIdx.y) of a tile of 32, its parts shared by groups
// of DP / 4 threads, joined through LDS in order.
template <DT D, int DP> __global__ __launch_bounds__(256) void attention_join_rows_kernel(FwdArgs a) {
  constexpr int kThreads = DP / 4, kGroups = 256 / kThreads;
  __shared__ float4 s_part[256];
  __shared__ float2 s_state[kGroups];
  const int group = a.heads / a.kv_heads, parts = a.cut.parts;
  const Share share = tile_share(a.cut, blockIdx.x);
  const Item it = find_rows(a, a.window, group, 32, share.slot);
  const int64_t row = (int64_t)it.tile * 32 + blockIdx.y;
  if (row >= (int64_t)it.nq * group) return;
  const int c = threadIdx.x % kThreads * 4, mine = threadIdx.x / kThreads;
  const int64_t first = (int64_t)share.place * 32 + blockIdx.y;
  constexpr int kBatch = 8;
  float base = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const auto add = [&](float2 st, float4 p, bool some) {  // (base has been raised to st.x)
    const float w = some ? exp2_fast(st.x - base) : 0.f;
    sum = fmaf(w, some ? st.y : 0.f, sum);
    o.x = fmaf(w, some ? p.x : 0.f, o.x);
    o.y = fmaf(w, some ? p.y : 0.f, o.y);
    o.z = fmaf(w, some ? p.z : 0.f, o.z);
    o.w = fmaf(w, some ? p.w : 0.f, o.w);
  };
  const auto raise = [&](float top) {
    const float shrink = exp2_fast(base - top);
    base = top;
    sum *= shrink;
    o = make_float4(o.x * shrink, o.y * shrink, o.z * shrink, o.w * shrink);
  };
  for (int s0 = mine; s0 < parts; s0 += kBatch * kGroups) {
    float2 st[kBatch];
    float4 p[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t at = first + (int64_t)min(s0 + i * kGroups, parts - 1) * 32;
      st[i] = a.state[at];
      p[i] = *reinterpret_cast<const float4*>(a.part + at * DP + c);
    }
    float top = base;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) top = fmaxf(top, st[i].x);
    if (top == -INFINITY) continue;
    raise(top);
    // (a share without keys has a sum of 0 and wrote no part)
#pragma unroll
    for (int i = 0; i < kBatch; ++i) add(st[i], p[i], s0 + i * kGroups < parts && st[i].y != 0.f);
  }
  s_part[threadIdx.x] = o;
  if (c == 0) s_state[mine] = make_float2(base, sum);
  __syncthreads();
  if (mine != 0) return;
#pragma unroll
  for (int k = 1; k < kGroups; ++k) {
    const float2 st = s_state[k];
    if (st.y == 0.f) continue;  // (no parts, or none with keys)
    raise(fmaxf(base, st.x));
    add(st, s_part[k * kThreads + threadIdx.x], true);
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  const RowMap qmap{it.q0, share.head * group, group};
  if (c < a.head_dim) store4<D>(qmap.at<D>(heads_of<D>(a.out), (int)row) + c, o.x * f, o.y * f, o.z * f, o.w * f);
  if (a.lse != nullptr && c == 0) a.lse[qmap.stat((int)row, a.heads)] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * kLn2;
}

template <DT D, int DC, int W, int KG, int CUT, bool WINDOW> hipError_t launch_tiles(const FwdArgs& a, hipStream_t stream) {
  constexpr int KEYS = D == DT::F32 || W == 1 ? 32 : 64;
  constexpr int OCC = D == DT::F32 || (W == 1 && DC > 64) ? 1 : DC <= 64 && KG == 1 && CUT == kNoCut ? 3 : 2;
  const dim3 grid = CUT == kNoCut ? dim3((unsigned)a.cut.slots, (unsigned)a.kv_heads) : dim3((unsigned)cut_blocks(a.cut));
  attention_forward_kernel<D, DC, W, KG, KEYS, OCC, CUT, WINDOW><<<grid, KG * W * 64, 0, stream>>>(a);
  return hipGetLastError();
}

template <DT D, int DC, int W, int CUT, bool WINDOW, int KG = 1> Status launch_cut(FwdArgs a, hipStream_t stream) {
  constexpr int DP = tile_width(DC);
  int dev = 0;
  SUBM_HIP_TRY(hipGetDevice(&dev));
  ScratchLease lease;
  const size_t rows = (size_t)cut_places(a.cut) * 32 * W;
  void* scratch = nullptr;
  Status st = lease.take(dev, stream, rows * (DP * sizeof(float) + sizeof(float2)), &scratch);
  if (!st.ok()) return st;
  a.part = static_cast<float*>(scratch);
  a.state = reinterpret_cast<float2*>(a.part + rows * DP);
  SUBM_HIP_TRY((launch_tiles<D, DC, W, KG, CUT, WINDOW>(a, stream)));
  if constexpr (W == 1) {
    attention_join_rows_kernel<D, DP><<<dim3((unsigned)a.cut.cut, (unsigned)std::min<int64_t>(32, a.nq * (a.heads / a.kv_heads))), 256, 0, stream>>>(a);
  } else {
    attention_join_kernel<D, DP, W, WINDOW><<<dim3((unsigned)a.cut.cut, 32 * W * (DP / 4) / 256), 256, 0, stream>>>(a);
  }
  SUBM_HIP_TRY(hipGetLastError());
  return Status{};
}

// Windows with few rows an item (single tokens of grouped heads): tiles of 32 rows, which one wave holds, and KG
// waves that take every KG-th 32 keys.  Kernel and join, against tiles of 128 rows: one token, 4 / 1 heads of 128,
// 60,000 keys: 19 and 41 us; 3 tokens, 12 heads of 64, 3,000 keys: 15 and 16; 8 tokens, 4 heads of 128, 2,000 keys,
// float32: 39 and 52; 8 tokens, 16 / 4 heads of 128, 4,096 keys each: 22 both, of which 59 MB take 11: a step's loads
// have one step's time to arrive, and with one wave's rows that is less than memory takes.  At 128 channels two
// waves a workgroup where there are many items (17 tokens, 16 / 4 heads, 8,000 keys: 44 us, 52 with four).
template <DT D, int DC, int KG> Status launch_few(FwdArgs a, int64_t rows, hipStream_t stream) {
  constexpr int kTileBytes = KG * 4 * 32 * kRowBytes<D, tile_width(DC)>, kResident = 256 * (kTileBytes > 65536 ? 1 : 2);
  const int64_t slots = rows / 32 + a.items, walked = a.window.walked(a.nk / a.items, 32);
  constexpr int kLeast = D == DT::F32 ? 64 : 128, kWhole = D == DT::F32 ? 64 : 512;
  const int64_t parts = walked <= kWhole ? 1 : std::min<int64_t>(kResident / ((int64_t)a.items * a.kv_heads), walked / kLeast);
  if (parts > 1) {
    a.cut = Cut{(int)slots, 0, (int)(slots * a.kv_heads), (int)parts, parts % 8 == 0 || 8 % parts == 0};
    return launch_cut<D, DC, 1, kCutAll, true, KG>(a, stream);
  }
  a.cut = Cut{(int)slots, (int)(slots * a.kv_heads), 0, 1, false};
  SUBM_HIP_TRY((launch_tiles<D, DC, 1, KG, kNoCut, true>(a, stream)));
  return Status{};
}

template <DT D, int DC, bool WINDOW>
Status launch(FwdArgs a, hipStream_t stream) {
  // 128 channels: 8 waves on one tile stream halve what each row reads of it (24,576 tokens, 16
  // heads, whole tiles: 2.33 ms, 4 waves 2.80), where they fill the compute units.  64 channels: 4
  // waves and three workgroups a compute unit, whose exponentials, the bound there, overlap (9,371
  // rows, 12 heads: 47.9 us, 8 waves 66.7).
  constexpr int kUnits = 256;
  constexpr bool kWide = D != DT::F32 && tile_width(DC) == 128;
  const int64_t rows = a.nq * (a.heads / a.kv_heads), spare = (int64_t)a.items * a.kv_heads;
  // (of a window: those of a tile)
  const int64_t keys = WINDOW ? a.window.walked(a.nk / a.items, 128 / (a.heads / a.kv_heads)) : a.nk / a.items;
  if constexpr (WINDOW) {
    a.window.runs = a.window.in_runs(a.nk / a.items, a.heads / a.kv_heads);
    // Single tokens and the like: a wave holds an item's rows, and the waves of a workgroup share its keys.
    if (rows <= 32 * (int64_t)a.items) {
      if constexpr (D == DT::F32) return launch_few<D, DC, 2>(a, rows, stream);
      else if constexpr (tile_width(DC) == 64) return launch_few<D, DC, 4>(a, rows, stream);
      else return spare < kUnits / 4 ? launch_few<D, DC, 4>(a, rows, stream) : launch_few<D, DC, 2>(a, rows, stream);
    }
  }
  // float32 scores take 8 times as long, so its parts may be short.
  constexpr int kShare = D == DT::F32 ? 32 : WINDOW ? 256 : 512;
  if constexpr (kWide && !WINDOW) {
    const int64_t slots = rows / 256 + a.items;
    if (slots * a.kv_heads >= kUnits && rows / a.items >= 256) {
      a.cut = plan_cut(slots, a.kv_heads, spare, keys, kShare, kUnits, 0, kGainAt128);
      if (a.cut.parts > 1) return launch_cut<D, DC, 8, kCutLast, WINDOW>(a, stream);
      SUBM_HIP_TRY((launch_tiles<D, DC, 8, 1, kNoCut, WINDOW>(a, stream)));
      return Status{};
    }
  }
  // Few tiles: parts for two workgroups a unit (float32: one).  Last tiles in parts: not at 64
  // channels, whose last workgroups speed up as others leave their unit (24,576 tokens, 16 heads: 1.34
  // ms, 1.39 in parts), nor at the short items that are left here at 128.
  const int64_t slots = rows / 128 + a.items, tiles = slots * a.kv_heads;
  constexpr int kFew = kUnits * (D == DT::F32 ? 1 : 2);
  if constexpr (WINDOW) {
    constexpr int64_t kSlots = kUnits * (D == DT::F32 ? 1 : tile_width(DC) == 64 ? 3 : 2);
    a.cut = plan_window_cut(a.window, slots, a.kv_heads, a.nk / a.items, keys, kShare, kSlots, kFew);
  } else {
    a.cut = plan_cut(slots, a.kv_heads, spare, keys, kShare, D == DT::F32 ? kUnits : INT32_MAX, kFew, kGain);
  }
  // Where a compute unit gets one workgroup, two groups of waves on each tile (2,000 tokens, 16 heads
  // of 128: 42 us, 54 in two parts; with fewer than 512 keys the join eats the gain).  float32 waves
  // need the registers of two.
  if constexpr (D != DT::F32) {
    if (tiles <= kUnits && keys >= 512 && a.cut.parts <= 2) {
      SUBM_HIP_TRY((launch_tiles<D, DC, 4, 2, kNoCut, WINDOW>(a, stream)));
      return Status{};
    }
  } else if constexpr (!WINDOW) {
    if (a.cut.parts > 1 && a.cut.whole > 0) return launch_cut<D, DC, 4, kCutLast, WINDOW>(a, stream);
  }
  if (a.cut.parts > 1) return launch_cut<D, DC, 4, kCutAll, WINDOW>(a, stream);
  SUBM_HIP_TRY((launch_tiles<D, DC, 4, 1, kNoCut, WINDOW>(a, stream)));
  return Status{};
}

template <DT D, bool WINDOW> Status launch_dim(const FwdArgs& a, hipStream_t stream) {
  if (a.head_dim <= 32) return launch<D, 32, WINDOW>(a, stream);
  if (a.head_dim <= 64) return launch<D, 64, WINDOW>(a, stream);
  if (a.head_dim <= 96) return launch<D, 96, WINDOW>(a, stream);
  return launch<D, 128, WINDOW>(a, stream);
}

}  // namespace
}  // namespace submconv
