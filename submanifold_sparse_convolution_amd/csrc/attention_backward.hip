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
// [1, 2); the results are scaled back in float32.  bfloat16 has float32's range and needs neither.
#include <algorithm>
#include <cmath>

#include "attention_common.h"

namespace submconv {
namespace {

struct BwdArgs {
  subm_heads_t dout, q, k, v, out, dq, dk, dv;
  const float* lse;
  float* delta;     // [nq, heads]: d
  float* peak;      // [kv_heads, slots]: the largest |dout| of each query block (float16 only)
  const int64_t *q_offsets, *k_offsets;
  int64_t nq, nk, q_slots;
  int items, heads, kv_heads, head_dim;
  float scale;
};

constexpr int kBwdWaves = 4;
constexpr int kOwn = 32 * kBwdWaves;  // own rows of a workgroup (query rows or keys), 32 a wave
constexpr int kStep = 32;             // rows of the walked tile

constexpr float kF16Shift = 15.f;  // p is scaled by 2^15 in float16 products

// 2^-floor(log2 x): the power of two that takes x to [1, 2); 1 for 0, subnormal and non-finite x.
__device__ __forceinline__ float unit_scale(float x) {
  const int e = (int)(__float_as_uint(x) >> 23) & 255;
  return e == 0 || e >= 254 ? 1.f : __uint_as_float((uint32_t)(254 - e) << 23);
}

template <DT D> __device__ __forceinline__ float absmax_frag(const Frag<D>& f) {
  float m = 0.f;
  const uint32_t w[4] = {f.v[0].x, f.v[0].y, f.v[0].z, f.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(to_float<D>((uint16_t)w[i])), fabsf(to_float<D>((uint16_t)(w[i] >> 16)))));
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

// d of the own query rows, then dq over the keys.
template <DT D, int DP>
__global__ __launch_bounds__(kBwdWaves * 64) void attention_dq_kernel(BwdArgs a) {
  __shared__ __attribute__((aligned(16))) unsigned char s_k[kStep * kRowBytes<D, DP>];
  __shared__ __attribute__((aligned(16))) unsigned char s_v[kStep * kRowBytes<D, DP>];
  __shared__ float s_peak[kBwdWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int group = a.heads / a.kv_heads, head = blockIdx.y;
  int tile;
  const int item = find_item(a.q_offsets, a.nq, a.items, group, kOwn, blockIdx.x, &tile);
  int64_t q0, k0;
  int nq, nk;
  item_rows(a.q_offsets, a.nq, item, &q0, &nq);
  item_rows(a.k_offsets, a.nk, item, &k0, &nk);
  const int rows = nq * group;
  if ((int64_t)tile * kOwn >= rows) return;
  const RowMap qmap{q0, head * group, group}, kmap{k0, head, 1};
  const Heads<D> k = heads_of<D>(a.k), v = heads_of<D>(a.v);

  const int row = tile * kOwn + wave * 32 + (lane & 31);
  const bool there = row < rows;
  const int safe = there ? row : 0;
  Frag<D> qf[DP / 16], gf[DP / 16];  // own rows of q and dout
  const typename Elem<D>::T* qrow = qmap.at<D>(heads_of<D>(a.q), safe);
  const typename Elem<D>::T* grow = qmap.at<D>(heads_of<D>(a.dout), safe);
  const typename Elem<D>::T* orow = qmap.at<D>(heads_of<D>(a.out), safe);
  float d = 0.f, peak = 0.f;
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk) {
    qf[kk] = own_frag<D>(qrow, there, kk, a.head_dim, lane);
    gf[kk] = own_frag<D>(grow, there, kk, a.head_dim, lane);
    d = dot_frag<D>(gf[kk], own_frag<D>(orow, there, kk, a.head_dim, lane), d);
    if constexpr (D == DT::F16) peak = fmaxf(peak, absmax_frag<D>(gf[kk]));
  }
  d = half_sum(d);
  if (there && lane < 32) a.delta[qmap.stat(row, a.heads)] = d;
  float unit = 1.f;
  if constexpr (D == DT::F16) {
    peak = half_max(peak);
    unit = unit_scale(peak);
#pragma unroll
    for (int mk = 16; mk >= 1; mk >>= 1) peak = fmaxf(peak, __shfl_xor(peak, mk, 64));
    if (lane == 0) s_peak[wave] = peak;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int w = 1; w < kBwdWaves; ++w) peak = fmaxf(peak, s_peak[w]);
      a.peak[head * a.q_slots + blockIdx.x] = peak;
    }
  }
  const float c = a.scale * kLog2e;
  const TileReader<D, DP> rd(lane, lds_offset(s_k), lds_offset(s_k));
  const int to_v = (int)(lds_offset(s_v) - lds_offset(s_k));
  // log2 of the row's normaliser, less the power of two that e is scaled by
  const float base = there ? a.lse[qmap.stat(row, a.heads)] * kLog2e : 0.f;
  f32x16_t acc[DP / 32];
#pragma unroll
  for (int db = 0; db < DP / 32; ++db) acc[db] = zero16();
  for (int key = 0; key < nk; key += kStep) {
    __syncthreads();
    stage_rows<D, DP, kStep, kBwdWaves * 64>(s_k, k, kmap, key, nk, a.head_dim);
    stage_rows<D, DP, kStep, kBwdWaves * 64>(s_v, v, kmap, key, nk, a.head_dim);
    __syncthreads();
    f32x16_t s = zero16(), dp = zero16();
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      s = mma<D>(rd.row_frag(0, 0, kk), qf[kk], s);
      dp = mma<D>(rd.row_frag(to_v, 0, kk), gf[kk], dp);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int j = key + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
      const float e = exp2_fast(fmaf(s[i], c, -base)) * (dp[i] - d) * unit;
      s[i] = j < nk ? e : 0.f;  // (a key past the end scores 0, which p need not take to 0)
    }
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const Frag<D> e = to_frag<D>(s, st);
#pragma unroll
      for (int db = 0; db < DP / 32; ++db) acc[db] = mma<D>(rd.column_frag(0, st * 16, db), e, acc[db]);
    }
  }
  if (there) store_row<D, DP>(qmap.at<D>(heads_of<D>(a.dq), row), acc, a.scale / unit, a.head_dim, lane);
}

// dk and dv of the own keys, over the query rows of all heads that share the key head.
template <DT D, int DP>
__global__ __launch_bounds__(kBwdWaves * 64) void attention_dkv_kernel(BwdArgs a) {
  __shared__ __attribute__((aligned(16))) unsigned char s_q[kStep * kRowBytes<D, DP>];
  __shared__ __attribute__((aligned(16))) unsigned char s_g[kStep * kRowBytes<D, DP>];
  __shared__ __attribute__((aligned(16))) float s_lse[kStep], s_delta[kStep];
  __shared__ float s_peak[kBwdWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int group = a.heads / a.kv_heads, head = blockIdx.y;
  int tile;
  const int item = find_item(a.k_offsets, a.nk, a.items, 1, kOwn, blockIdx.x, &tile);
  int64_t q0, k0;
  int nq, nk;
  item_rows(a.q_offsets, a.nq, item, &q0, &nq);
  item_rows(a.k_offsets, a.nk, item, &k0, &nk);
  const int rows = nq * group;
  if ((int64_t)tile * kOwn >= nk) return;
  const RowMap qmap{q0, head * group, group}, kmap{k0, head, 1};
  const Heads<D> q = heads_of<D>(a.q), g = heads_of<D>(a.dout);

  float unit = 1.f;
  if constexpr (D == DT::F16) {  // the largest |dout| of the item and head, from its query blocks
    const int64_t first = q0 * group / kOwn + item;
    float peak = 0.f;
    for (int t = threadIdx.x; t < (rows + kOwn - 1) / kOwn; t += kBwdWaves * 64)
      peak = fmaxf(peak, a.peak[head * a.q_slots + first + t]);
#pragma unroll
    for (int mk = 32; mk >= 1; mk >>= 1) peak = fmaxf(peak, __shfl_xor(peak, mk, 64));
    if (lane == 0) s_peak[wave] = peak;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kBwdWaves; ++w) peak = fmaxf(peak, s_peak[w]);
    unit = unit_scale(peak);
  }
  const float shift = D == DT::F16 ? kF16Shift : 0.f;
  const float p_unit = D == DT::F16 ? 1.f / 32768.f : 1.f;

  const int key = tile * kOwn + wave * 32 + (lane & 31);
  const bool there = key < nk;
  Frag<D> kf[DP / 16], vf[DP / 16];
  const typename Elem<D>::T* krow = kmap.at<D>(heads_of<D>(a.k), there ? key : 0);
  const typename Elem<D>::T* vrow = kmap.at<D>(heads_of<D>(a.v), there ? key : 0);
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk) {
    kf[kk] = own_frag<D>(krow, there, kk, a.head_dim, lane);
    vf[kk] = own_frag<D>(vrow, there, kk, a.head_dim, lane);
  }
  const float c = a.scale * kLog2e;
  const TileReader<D, DP> rd(lane, lds_offset(s_q), lds_offset(s_q));
  const int to_g = (int)(lds_offset(s_g) - lds_offset(s_q));
  f32x16_t dk[DP / 32], dv[DP / 32];
#pragma unroll
  for (int db = 0; db < DP / 32; ++db) dk[db] = dv[db] = zero16();
  for (int r0 = 0; r0 < rows; r0 += kStep) {
    __syncthreads();
    stage_rows<D, DP, kStep, kBwdWaves * 64>(s_q, q, qmap, r0, rows, a.head_dim);
    stage_rows<D, DP, kStep, kBwdWaves * 64>(s_g, g, qmap, r0, rows, a.head_dim);
    if (threadIdx.x < kStep) {
      const int r = r0 + threadIdx.x;
      const int64_t at = qmap.stat(r < rows ? r : 0, a.heads);
      s_lse[threadIdx.x] = r < rows ? a.lse[at] * kLog2e - shift : INFINITY;  // p = 0 past the last row
      s_delta[threadIdx.x] = r < rows ? a.delta[at] : 0.f;
    }
    __syncthreads();
    f32x16_t s = zero16(), dp = zero16();
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      s = mma<D>(rd.row_frag(0, 0, kk), kf[kk], s);
      dp = mma<D>(rd.row_frag(to_g, 0, kk), vf[kk], dp);
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const float4 ls = *reinterpret_cast<const float4*>(s_lse + 8 * b + 4 * (lane >> 5));
      const float4 dl = *reinterpret_cast<const float4*>(s_delta + 8 * b + 4 * (lane >> 5));
      const float lse4[4] = {ls.x, ls.y, ls.z, ls.w}, del4[4] = {dl.x, dl.y, dl.z, dl.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = exp2_fast(fmaf(s[4 * b + i], c, -lse4[i]));
        s[4 * b + i] = p;
        dp[4 * b + i] = p * (dp[4 * b + i] - del4[i]) * (unit * p_unit);
      }
    }
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      const Frag<D> p = to_frag<D>(s, st), e = to_frag<D>(dp, st);
#pragma unroll
      for (int db = 0; db < DP / 32; ++db) {
        dv[db] = mma<D>(rd.column_frag(to_g, st * 16, db), p, dv[db]);
        dk[db] = mma<D>(rd.column_frag(0, st * 16, db), e, dk[db]);
      }
    }
  }
  if (!there) return;
  store_row<D, DP>(kmap.at<D>(heads_of<D>(a.dk), key), dk, a.scale / unit, a.head_dim, lane);
  store_row<D, DP>(kmap.at<D>(heads_of<D>(a.dv), key), dv, p_unit, a.head_dim, lane);
}

template <DT D, int DP>
hipError_t launch(const BwdArgs& a, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (a.nq > 0) {
    attention_dq_kernel<D, DP><<<dim3((unsigned)a.q_slots, (unsigned)a.kv_heads), kBwdWaves * 64, 0, stream>>>(a);
    e = hipGetLastError();
  }
  if (e == hipSuccess && a.nk > 0) {
    const int64_t slots = a.nk / kOwn + a.items;
    attention_dkv_kernel<D, DP><<<dim3((unsigned)slots, (unsigned)a.kv_heads), kBwdWaves * 64, 0, stream>>>(a);
    e = hipGetLastError();
  }
  return e;
}

template <DT D> hipError_t launch_dim(const BwdArgs& a, hipStream_t stream) {
  return a.head_dim <= 64 ? launch<D, 64>(a, stream) : launch<D, 128>(a, stream);
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
  BwdArgs a{*dout, *q, *k, *v, *out, *dq, *dk, *dv, lse, nullptr, nullptr, q_offsets, k_offsets, nq, nk, 0,
            items, heads, kv_heads, head_dim, scale};
  a.q_slots = nq * (heads / kv_heads) / kOwn + items;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(hip_status(e, "hipGetDevice"));
  const size_t delta_bytes = ((size_t)nq * heads * sizeof(float) + 255) / 256 * 256;
  const size_t peak_bytes = (size_t)a.q_slots * kv_heads * sizeof(float);
  void* scratch = nullptr;
  st = stream_scratch(dev, stream, delta_bytes + peak_bytes, &scratch);
  if (!st.ok()) return fail(st);
  a.delta = static_cast<float*>(scratch);
  a.peak = reinterpret_cast<float*>(static_cast<unsigned char*>(scratch) + delta_bytes);
  if (dtype == SUBM_F32) e = launch_dim<DT::F32>(a, stream);
  else if (dtype == SUBM_F16) e = launch_dim<DT::F16>(a, stream);
  else e = launch_dim<DT::BF16>(a, stream);
  if (e != hipSuccess) return fail(hip_status(e, "sparse_attention_backward launch"));
  return SUBM_OK;
}
