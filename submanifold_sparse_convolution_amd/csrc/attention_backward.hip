// Attention over the items of a sparse tensor, backward pass (include/sparse_transformer.h).
//
//   p = exp(scale q k^T - lse),  dp = dout v^T,  d = sum_c dout out,  e = p (dp - d)
//   dv = p^T dout,  dk = scale e^T q,  dq = scale e k
//
// Two kernels recompute p: one owns blocks of query rows and walks the keys (d, then dq), one owns
// blocks of keys and walks the query rows (dk, dv).  That is 7 products where one kernel with
// atomics on dq would do 5, but every sum has one order, and nothing is written twice.
//
// float16 storage: p spans 2^-24 and below for long items, e is as small as the gradient; both
// would fall among or under the subnormals.  p is scaled by 2^15 (p <= 1), and e by the power of
// two that takes the largest |dout| of its row (for dq) or of its item and head (for dk) to
// [1, 2), or by the smaller one that keeps 2 |dout|_2 max_j |v_j|_2, which no |dp - d| exceeds (d is
// a mean of dp), below 2^15; the results are scaled back in float32.  A kernel before the others
// leaves the norms of v (7,813 tokens, 4 key heads of 64: 4 us on the device, the whole training call
// 371 -> 376 us; 800 tokens, 8 heads of 64: 42 -> 46).  bfloat16 has float32's range and needs none of
// this.
//
// Bound by the matrix cores and, at 64 channels, by the exponentials.  Measured: items of 9,000 and
// 7,384 tokens, 16 heads of 128, bf16: dq 1.40 ms (3 products, 1.19 PFLOP/s, matrix cores busy 65 %),
// dk and dv 2.07 ms (4 products, 1.07 PFLOP/s, 54 %); five items of up to 2,971 tokens, 12 / 4 heads of
// 64, f16: dq 117 us (0.67 PFLOP/s), dk and dv 175 us (0.60).
#include <algorithm>
#include <cmath>

#include "attention_common.h"

namespace submconv {
namespace {

struct BwdArgs {
  subm_heads_t dout, q, k, v, out, dq, dk, dv;
  const float* lse;
  float *norm, *delta;  // [kv_heads, nq * group]: log2 of each packed row's normaliser (less kF16Shift), and d
  // float16 only: [kv_heads, q_slots] the largest |dout| and bound of |dp - d| of each query block,
  // and [kv_heads, v_slots] a bound of |v|_2 over each block of kNormKeys keys
  float2* peak;
  float* v_norm;
  const int64_t *q_offsets, *k_offsets;
  int64_t nq, nk, q_slots, v_slots;
  int items, heads, kv_heads, head_dim;
  float scale;
  int q_rows;  // packed rows of a workgroup of the dq kernel
  // Tiles in parts: float32 sums of dq by the first cut, of dk and dv by the second, [place][rows of
  // a tile][DP], summed by a third kernel.
  Cut q_cut, k_cut;
  float *dq_part, *dk_part, *dv_part;
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
// row; the longest row's norm is between a quarter of the bound and all of it).
template <DT D> __global__ __launch_bounds__(256) void attention_norm_kernel(BwdArgs a) {
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
  for (int i = 0; i < kNormKeys / 16; ++i) top = fmaxf(top, dot_frag<D>(f[i], f[i], 0.f));
  top = fmaxf(top, __shfl_xor(top, 16, 64));
  top = fmaxf(top, __shfl_xor(top, 32, 64));
  if ((threadIdx.x & 63) < 16) s_top[threadIdx.x / 64 * 16 + threadIdx.x % 64] = top;
  __syncthreads();
  if (threadIdx.x != 0) return;
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) sq += fmaxf(fmaxf(s_top[i], s_top[16 + i]), fmaxf(s_top[32 + i], s_top[48 + i]));
  a.v_norm[head * a.v_slots + blockIdx.x] = sqrtf(sq);
}

// d of the own query rows, then dq over the keys, which stream through LDS in tiles of 32.  As in
// the forward pass a step holds independent pieces of work:
//   scores and dp of tile t + 1 (k, v),  e of tile t,  product of tile t - 1 (k).
template <DT D, int DC, int W, int OCC, int CUT>
__global__ __launch_bounds__(W * 64, OCC) void attention_dq_kernel(BwdArgs a) {
  constexpr int DP = tile_width(DC), kRows = 32 * W;
  constexpr int kTile = kStep * kRowBytes<D, DP>;
  using Loader = TileLoader<D, DP, kStep, W>;
  __shared__ __attribute__((aligned(1024))) unsigned char s_kv[6 * kTile];  // four tiles of k, two of v
  __shared__ float2 s_peak[W];
  __shared__ float s_norm[W];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.heads / a.kv_heads;
  const Share share = share_of<CUT>(a.q_cut, blockIdx.x);
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
  if constexpr (D == DT::F16) {
    peak = half_max(peak);
    const float bound = 2.f * sqrtf(half_sum(sq)) * item_norm<W>(a, head, item, k0, nk, s_norm);
    unit = e_scale(peak, bound);
    const float2 top = make_float2(wave_max(peak), wave_max(bound));
    if (lane == 0) s_peak[wave] = top;
    __syncthreads();
    if (first && threadIdx.x == 0) {
      float2 all = top;
#pragma unroll
      for (int w = 0; w < W; ++w) all = make_float2(fmaxf(all.x, s_peak[w].x), fmaxf(all.y, s_peak[w].y));
      a.peak[head * a.q_slots + share.slot] = all;
    }
  }
  const float c = a.scale * kLog2e;

  Loader lk, lv;
  lk.wave = lv.wave = wave;
  lk.lane = lv.lane = lane;
  lk.place(k, a.head_dim, 1, 0, 0);
  lv.place(v, a.head_dim, 1, 0, 0);
  const uint32_t lds = lds_offset(s_kv);
  const TileReader<D, DP> rd(lane, lds, lds);
  int tiles = (nk + kStep - 1) / kStep, left = nk;
  if constexpr (CUT != kNoCut) {
    const int t0 = part_steps(a.q_cut, share.part, &tiles);
    left = min(nk - t0 * kStep, tiles * kStep);
    kp += (int64_t)t0 * kStep * k.row;
    vp += (int64_t)t0 * kStep * v.row;
  }
  const auto load_k = [&](int t, int slot) {
    lk.load(kp + (int64_t)t * kStep * k.row, t < 0 ? 0 : left - t * kStep, lds + slot * kTile);
  };
  const auto load_v = [&](int t, int slot) {
    lv.load(vp + (int64_t)t * kStep * v.row, left - t * kStep, lds + (4 + slot) * kTile);
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
  if (tiles > 0) {
    // Step t reads k and v of tile t + 1 and k of tile t - 1 and starts the loads of tile t + 2.
    load_k(0, 0);
    load_v(0, 0);
    load_k(-1, 3);  // (zeros)
    load_k(1, 1);
    load_v(1, 1);
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
      if ((t + 1) * kStep > left) {  // (a key past the end scores 0, which p need not take to 0)
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
  if (!there) return;
  if (CUT == kCutAll || (CUT == kCutLast && share.part >= 0))
    store_part<DC>(a.dq_part + ((int64_t)share.place * kRows + wave * 32 + (lane & 31)) * DP, acc, a.scale / unit, lane);
  else
    store_row<D, DC>(qmap.at<D>(heads_of<D>(a.dq), row), acc, a.scale / unit, a.head_dim, lane);
}

// The next 32 of `left` floats (zeros past them) straight to LDS, which takes 64 of them.
__device__ __forceinline__ void load_stats(const float* p, int left, uint32_t lds, int lane) {
  const i32x4_t rsrc = make_rsrc(p, kOutOfRange);
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
// and k there is no room for them in 256 registers.
template <DT D, int DC, int W, int OCC, int CUT>
__global__ __launch_bounds__(W * 64, OCC) void attention_dkv_kernel(BwdArgs a) {
  constexpr int DP = tile_width(DC), kKeys = 32 * W;
  constexpr int kTile = kStep * kRowBytes<D, DP>;
  constexpr bool kParked = D != DT::F32 && DP == 128;
  using Loader = TileLoader<D, DP, kStep, W>;
  using Parker = TileLoader<D, DP, kKeys, W>;
  // q, q, dout, dout, own v
  __shared__ __attribute__((aligned(1024))) unsigned char s_qg[4 * kTile + (kParked ? W * kTile : 0)];
  __shared__ __attribute__((aligned(16))) float s_stat[2 * 2 * 64];  // norm and d of two tiles
  __shared__ float2 s_peak[W];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = a.heads / a.kv_heads;
  const Share share = share_of<CUT>(a.k_cut, blockIdx.x);
  const int head = share.head;
  int tile;
  const int item = find_item(a.k_offsets, a.nk, a.items, 1, kKeys, share.slot, &tile);
  int64_t q0, k0;
  int nq, nk;
  item_rows(a.q_offsets, a.nq, item, &q0, &nq);
  item_rows(a.k_offsets, a.nk, item, &k0, &nk);
  const int rows = nq * group;
  if ((int64_t)tile * kKeys >= nk) return;
  const RowMap kmap{k0, head, 1};
  const Heads<D> q = heads_of<D>(a.q), g = heads_of<D>(a.dout), v = heads_of<D>(a.v);
  const typename Elem<D>::T* qp = q.data + q0 * q.row + (int64_t)head * group * q.head;
  const typename Elem<D>::T* gp = g.data + q0 * g.row + (int64_t)head * group * g.head;
  const float* norm = a.norm + head * (a.nq * group) + q0 * group;
  const float* delta = a.delta + head * (a.nq * group) + q0 * group;

  float unit = 1.f;
  if constexpr (D == DT::F16) {  // the largest |dout| and bound of the item and head, from its query blocks
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
  if constexpr (CUT != kNoCut) {
    r0 = part_steps(a.k_cut, share.part, &steps) * kStep;
    end = min(rows, r0 + steps * kStep);
  }
  int tok = r0 / group, rem = r0 - tok * group;  // of the next tile to load
  const int tok_step = kStep / group, rem_step = kStep % group;
  lq.place(q, a.head_dim, group, rem, magic);
  lg.place(g, a.head_dim, group, rem, magic);
  const auto load = [&](int slot) {  // the next tile
    lq.load(qp + (int64_t)tok * q.row, end - r0, lds + slot * kTile);
    lg.load(gp + (int64_t)tok * g.row, end - r0, lds + (2 + slot) * kTile);
    if (wave == 0) load_stats(norm + r0, end - r0, stat + slot * 512, lane);
    if (wave == 1) load_stats(delta + r0, end - r0, stat + slot * 512 + 256, lane);
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
  const auto step = [&](int slot) {
    wait_lgkmcnt0();
    wait_vmcnt<0>();
    barrier_no_fence();
    load(slot ^ 1);
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
    // (rows past the end: q, dout, norm and d read 0, so p is 1 and meets a dout of 0, and e is 0)
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
    for (int t = 0; t < steps; t += 2) {  // (an odd end takes a step of zeros: a second exit costs registers)
      step(0);
      step(1);
    }
  }
  wait_vmcnt<0>();  // (the loads past the end)
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

template <DT D, int DC, int W, int CUT> hipError_t launch_dq(const BwdArgs& a, hipStream_t stream) {
  constexpr int OCC = D == DT::F32 ? 1 : DC <= 64 ? 3 : 2;
  const dim3 grid =
      CUT == kNoCut ? dim3((unsigned)a.q_cut.slots, (unsigned)a.kv_heads) : dim3((unsigned)cut_blocks(a.q_cut));
  attention_dq_kernel<D, DC, W, OCC, CUT><<<grid, W * 64, 0, stream>>>(a);
  return hipGetLastError();
}
template <DT D, int DC, int W, int CUT> hipError_t launch_dkv(const BwdArgs& a, hipStream_t stream) {
  constexpr int OCC = D == DT::F32 ? 1 : DC <= 64 ? 3 : 2;
  const dim3 grid =
      CUT == kNoCut ? dim3((unsigned)a.k_cut.slots, (unsigned)a.kv_heads) : dim3((unsigned)cut_blocks(a.k_cut));
  attention_dkv_kernel<D, DC, W, OCC, CUT><<<grid, W * 64, 0, stream>>>(a);
  return hipGetLastError();
}

// The cuts that plan_cut can give: of 8 waves' tiles, which fill the machine, the last; of 4 waves'
// at 128 channels in 16 bits all (if they filled it, their items would be too short).
template <DT D, int DC, int W> hipError_t launch_dq(const BwdArgs& a, hipStream_t stream) {
  constexpr bool kFull = D != DT::F32 && tile_width(DC) == 128;
  if constexpr (W == 8 || !kFull) {
    if (a.q_cut.parts > 1 && a.q_cut.whole > 0) return launch_dq<D, DC, W, kCutLast>(a, stream);
  }
  if constexpr (W == 4) {
    if (a.q_cut.parts > 1) return launch_dq<D, DC, W, kCutAll>(a, stream);
  }
  return launch_dq<D, DC, W, kNoCut>(a, stream);
}
template <DT D, int DC, int W> hipError_t launch_dkv(const BwdArgs& a, hipStream_t stream) {
  constexpr bool kFull = D != DT::F32 && tile_width(DC) == 128;
  if constexpr (W == 8 || !kFull) {
    if (a.k_cut.parts > 1 && a.k_cut.whole > 0) return launch_dkv<D, DC, W, kCutLast>(a, stream);
  }
  if constexpr (W == 4) {
    if (a.k_cut.parts > 1) return launch_dkv<D, DC, W, kCutAll>(a, stream);
  }
  return launch_dkv<D, DC, W, kNoCut>(a, stream);
}

template <DT D, int DC>
Status launch(BwdArgs a, hipStream_t stream) {
  constexpr int DP = tile_width(DC), kUnits = 256;
  const int group = a.heads / a.kv_heads;
  const int64_t rows = a.nq * group, spare = (int64_t)a.items * a.kv_heads;
  // 128 channels in 16 bits: 8 waves share a tile stream where they fill the compute units.
  constexpr bool kWide = D != DT::F32 && DP == 128;
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
  a.q_cut = plan_cut(a.q_slots, a.kv_heads, spare, a.nk / a.items, kLeast, q_full, kFew, kLess);
  a.k_cut = plan_cut(k_slots, a.kv_heads, spare, rows / a.items, kLeast, k_full, kFew, kLess);

  int dev = 0;
  SUBM_HIP_TRY(hipGetDevice(&dev));
  ScratchLease lease;
  const auto padded = [](size_t bytes) { return (bytes + 255) / 256 * 256; };
  // norm and d of every query row, peaks of query and key blocks, and the parts
  const size_t stat = padded((size_t)rows * a.kv_heads * sizeof(float));
  a.v_slots = a.nk / kNormKeys + a.items;
  const size_t peak = D == DT::F16 ? padded((size_t)a.q_slots * a.kv_heads * sizeof(float2)) : 0;
  const size_t norm = D == DT::F16 ? padded((size_t)a.v_slots * a.kv_heads * sizeof(float)) : 0;
  const size_t part_q = (size_t)cut_places(a.q_cut) * q_rows * DP * sizeof(float);
  const size_t part_k = (size_t)cut_places(a.k_cut) * k_rows * DP * sizeof(float);
  void* scratch = nullptr;
  Status st = lease.take(dev, stream, 2 * stat + peak + norm + part_q + 2 * part_k, &scratch);
  if (!st.ok()) return st;
  unsigned char* p = static_cast<unsigned char*>(scratch);
  a.norm = reinterpret_cast<float*>(p);
  a.delta = reinterpret_cast<float*>(p + stat);
  a.peak = reinterpret_cast<float2*>(p + 2 * stat);
  a.v_norm = reinterpret_cast<float*>(p + 2 * stat + peak);
  p += 2 * stat + peak + norm;
  if (part_q > 0) a.dq_part = reinterpret_cast<float*>(p);
  if (part_k > 0) {
    a.dk_part = reinterpret_cast<float*>(p + part_q);
    a.dv_part = reinterpret_cast<float*>(p + part_q + part_k);
  }
  if constexpr (D == DT::F16) {
    if (a.nk > 0) {
      attention_norm_kernel<D><<<dim3((unsigned)a.v_slots, (unsigned)a.kv_heads), 256, 0, stream>>>(a);
      SUBM_HIP_TRY(hipGetLastError());
    }
  }
  if (a.nq > 0) {
    if constexpr (kWide) {
      if (wide_q) SUBM_HIP_TRY((launch_dq<D, DC, 8>(a, stream)));
    }
    if (!wide_q) SUBM_HIP_TRY((launch_dq<D, DC, 4>(a, stream)));
  }
  if (a.nk > 0) {
    if constexpr (kWide) {
      if (wide_k) SUBM_HIP_TRY((launch_dkv<D, DC, 8>(a, stream)));
    }
    if (!wide_k) SUBM_HIP_TRY((launch_dkv<D, DC, 4>(a, stream)));
  }
  const unsigned jobs = (part_q > 0 ? 1 : 0) + (part_k > 0 ? 2 : 0);
  if (jobs > 0) {
    const dim3 grid((unsigned)std::max(a.q_cut.cut, a.k_cut.cut), std::max(q_rows, k_rows) * (DP / 4) / 256, jobs);
    attention_sum_kernel<D, DP><<<grid, 256, 0, stream>>>(a, q_rows, k_rows);
    SUBM_HIP_TRY(hipGetLastError());
  }
  return Status{};
}

template <DT D> Status launch_dim(const BwdArgs& a, hipStream_t stream) {
  if (a.head_dim <= 32) return launch<D, 32>(a, stream);
  if (a.head_dim <= 64) return launch<D, 64>(a, stream);
  if (a.head_dim <= 96) return launch<D, 96>(a, stream);
  return launch<D, 128>(a, stream);
}

}  // namespace
}  // namespace submconv

using namespace submconv;

extern "C" int sparse_attention_backward(const subm_heads_t* dout, const subm_heads_t* q, const subm_heads_t* k,
                                         const subm_heads_t* v, const subm_heads_t* out, const float* lse, int64_t nq,
                                         int64_t nk, const int64_t* q_offsets, const int64_t* k_offsets, int items,
                                         int heads, int kv_heads, int head_dim, int dtype, float scale,
                                         const subm_heads_t* dq, const subm_heads_t* dk, const subm_heads_t* dv,
                                         hipStream_t stream) {
  return no_throw([&]() -> int {
    clear_error();
    const AttentionShape shape{nq, nk, q_offsets, k_offsets, items, heads, kv_heads, head_dim, dtype, scale};
    Status st = check_attention(shape);
    if (st.ok()) st = check_heads(dout, nq, heads, shape, false, "dout");
    if (st.ok()) st = check_heads(q, nq, heads, shape, false, "q");
    if (st.ok()) st = check_heads(k, nk, kv_heads, shape, false, "k");
    if (st.ok()) st = check_heads(v, nk, kv_heads, shape, false, "v");
    if (st.ok()) st = check_heads(out, nq, heads, shape, false, "out");
    if (st.ok()) st = check_heads(dq, nq, heads, shape, true, "dq");
    if (st.ok()) st = check_heads(dk, nk, kv_heads, shape, true, "dk");
    if (st.ok()) st = check_heads(dv, nk, kv_heads, shape, true, "dv");
    if (!st.ok()) return fail(st);
    if (nq > 0 && lse == nullptr) return fail(SUBM_ERR_INVALID_ARG, "lse is NULL");
    if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return fail(SUBM_ERR_INVALID_ARG, "lse is not 4-byte aligned");
    if (nq == 0 && nk == 0) return SUBM_OK;
    // (the second kernel reads every input after the first has written dq)
    for (const subm_heads_t* w : {dq, dk, dv})
      for (const subm_heads_t* r : {dout, q, k, v, out})
        if (w->data != nullptr && w->data == r->data)
          return fail(SUBM_ERR_INVALID_ARG, "a gradient must not alias an input");
    if (nq > 0 && nk > 0 && (dq->data == dk->data || dq->data == dv->data))
      return fail(SUBM_ERR_INVALID_ARG, "dq, dk and dv must not alias");
    if (nk > 0 && dk->data == dv->data) return fail(SUBM_ERR_INVALID_ARG, "dq, dk and dv must not alias");
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
    a.q_offsets = q_offsets;
    a.k_offsets = k_offsets;
    a.nq = nq;
    a.nk = nk;
    a.items = items;
    a.heads = heads;
    a.kv_heads = kv_heads;
    a.head_dim = head_dim;
    a.scale = scale;
    if (dtype == SUBM_F32) st = launch_dim<DT::F32>(a, stream);
    else if (dtype == SUBM_F16) st = launch_dim<DT::F16>(a, stream);
    else st = launch_dim<DT::BF16>(a, stream);
    if (!st.ok()) return fail(st);
    return SUBM_OK;
  });
}
