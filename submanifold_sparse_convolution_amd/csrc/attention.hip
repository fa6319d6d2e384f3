// Attention over the items of a sparse tensor, forward pass (include/sparse_transformer.h).
//
//   S = scale q k^T,  m = max_j S,  l = sum_j exp(S - m),  out = (sum_j exp(S - m) v_j) / l,
//   lse = m + log l
// in one pass over the keys with the running m and l of a softmax: when m grows, l and the
// accumulator shrink by exp(m_old - m_new).  Exponentials are powers of two of scores that carry
// scale * log2(e).
//
// Bound by the matrix cores (4 rows keys d operations against rows and keys read once) except for
// a few rows against long caches, which read k and v once at HBM speed.
#include <algorithm>
#include <cmath>

#include "attention_common.h"

namespace submconv {
namespace {

struct FwdArgs {
  subm_heads_t q, k, v, out;
  float* lse;
  const int64_t *q_offsets, *k_offsets;
  int64_t nq, nk;
  int items, heads, kv_heads, head_dim;
  float scale;
};

constexpr int kFwdWaves = 4;
constexpr int kFwdRows = 32 * kFwdWaves;  // packed rows of a workgroup, 32 a wave
constexpr int kFwdKeys = 64;              // keys of a tile

template <DT D, int DP>
__global__ __launch_bounds__(kFwdWaves * 64) void attention_forward_kernel(FwdArgs a) {
  __shared__ __attribute__((aligned(16))) unsigned char s_k[kFwdKeys * kRowBytes<D, DP>];
  __shared__ __attribute__((aligned(16))) unsigned char s_v[kFwdKeys * kRowBytes<D, DP>];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int group = a.heads / a.kv_heads, head = blockIdx.y;
  int tile;
  const int item = find_item(a.q_offsets, a.nq, a.items, group, kFwdRows, blockIdx.x, &tile);
  int64_t q0, k0;
  int nq, nk;
  item_rows(a.q_offsets, a.nq, item, &q0, &nq);
  item_rows(a.k_offsets, a.nk, item, &k0, &nk);
  const int rows = nq * group;
  if ((int64_t)tile * kFwdRows >= rows) return;
  const RowMap qmap{q0, head * group, group}, kmap{k0, head, 1};
  const Heads<D> q = heads_of<D>(a.q), k = heads_of<D>(a.k), v = heads_of<D>(a.v), out = heads_of<D>(a.out);

  const int row = tile * kFwdRows + wave * 32 + (lane & 31);
  const bool there = row < rows;
  Frag<D> qf[DP / 16];
  const typename Elem<D>::T* qrow = qmap.at<D>(q, there ? row : 0);
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk) qf[kk] = own_frag<D>(qrow, there, kk, a.head_dim, lane);

  const float c = a.scale * kLog2e;
  f32x16_t acc[DP / 32];
#pragma unroll
  for (int db = 0; db < DP / 32; ++db) acc[db] = zero16();
  float m = -INFINITY, l = 0.f;  // m: the running maximum of c * score; l: this lane half's sum

  for (int key = 0; key < nk; key += kFwdKeys) {
    __syncthreads();
    stage_rows<D, DP, kFwdKeys, kFwdWaves * 64>(s_k, k, kmap, key, nk, a.head_dim);
    stage_rows<D, DP, kFwdKeys, kFwdWaves * 64>(s_v, v, kmap, key, nk, a.head_dim);
    __syncthreads();
    f32x16_t s[2] = {zero16(), zero16()};
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) s[kb] = mma<D>(row_frag<D, DP>(s_k, kb * 32, kk, lane), qf[kk], s[kb]);
    float top = -INFINITY;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = key + kb * 32 + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
        s[kb][i] = j < nk ? s[kb][i] * c : -INFINITY;
        top = fmaxf(top, s[kb][i]);
      }
    const float m_new = fmaxf(m, fmaxf(top, other_half(top)));
    // (scores that are all -infinity so far: the difference below must not become NaN)
    const float base = m_new == -INFINITY ? 0.f : m_new;
    const float shrink = exp2_fast(m - base);
    m = m_new;
    l *= shrink;
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[db][i] *= shrink;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[kb][i] = exp2_fast(s[kb][i] - base);
        l += s[kb][i];
      }
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const Frag<D> p = to_frag<D>(s[kb], st);
#pragma unroll
        for (int db = 0; db < DP / 32; ++db)
          acc[db] = mma<D>(column_frag<D, DP>(s_v, kb * 32 + st * 16, db, lane), p, acc[db]);
      }
  }
  l += other_half(l);
  if (!there) return;
  store_row<D, DP>(qmap.at<D>(out, row), acc, nk > 0 ? 1.f / l : 0.f, a.head_dim, lane);
  if (a.lse != nullptr && lane < 32) a.lse[qmap.stat(row, a.heads)] = nk > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <DT D, int DP>
hipError_t launch(const FwdArgs& a, hipStream_t stream) {
  const int group = a.heads / a.kv_heads;
  const int64_t slots = a.nq * group / kFwdRows + a.items;
  attention_forward_kernel<D, DP><<<dim3((unsigned)slots, (unsigned)a.kv_heads), kFwdWaves * 64, 0, stream>>>(a);
  return hipGetLastError();
}

template <DT D> hipError_t launch_dim(const FwdArgs& a, hipStream_t stream) {
  return a.head_dim <= 64 ? launch<D, 64>(a, stream) : launch<D, 128>(a, stream);
}

}  // namespace

Status check_attention(const AttentionShape& s) {
  if (s.dtype != SUBM_F32 && s.dtype != SUBM_F16 && s.dtype != SUBM_BF16)
    return make_status(SUBM_ERR_UNSUPPORTED, "dtype must be SUBM_F32, SUBM_F16 or SUBM_BF16");
  if (s.nq < 0 || s.nk < 0 || s.nq > INT32_MAX || s.nk > INT32_MAX)
    return make_status(SUBM_ERR_INVALID_ARG, "nq and nk must be 0 .. 2^31 - 1");
  if (s.items < 1 || s.items > 65535) return make_status(SUBM_ERR_INVALID_ARG, "items must be 1 .. 65535");
  if (s.heads < 1 || s.kv_heads < 1 || s.heads % s.kv_heads != 0)
    return make_status(SUBM_ERR_INVALID_ARG, "heads must be a positive multiple of kv_heads");
  if (s.kv_heads > 65535) return make_status(SUBM_ERR_INVALID_ARG, "kv_heads exceeds 65535");
  if (s.nq * s.heads > INT32_MAX) return make_status(SUBM_ERR_INVALID_ARG, "nq * heads exceeds 2^31 - 1");
  if (s.head_dim < 1) return make_status(SUBM_ERR_INVALID_ARG, "head_dim must be at least 1");
  if (s.head_dim % 8 != 0 || s.head_dim > 128)
    return make_status(SUBM_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 up to 128");
  if (!std::isfinite(s.scale)) return make_status(SUBM_ERR_INVALID_ARG, "scale must be finite");
  if (s.q_offsets == nullptr || s.k_offsets == nullptr) return make_status(SUBM_ERR_INVALID_ARG, "q_offsets or k_offsets is NULL");
  if (((reinterpret_cast<uintptr_t>(s.q_offsets) | reinterpret_cast<uintptr_t>(s.k_offsets)) & 7u) != 0)
    return make_status(SUBM_ERR_INVALID_ARG, "an offsets pointer is not 8-byte aligned");
  return Status{};
}

Status check_heads(const subm_heads_t* t, int64_t rows, int heads, const AttentionShape& s, bool written,
                   const char* what) {
  const std::string name(what);
  if (t == nullptr) return make_status(SUBM_ERR_INVALID_ARG, name + " is NULL");
  if (rows == 0) return Status{};
  if (t->data == nullptr) return make_status(SUBM_ERR_INVALID_ARG, name + ".data is NULL");
  const int64_t size = s.dtype == SUBM_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(t->data) & 15u) != 0 || t->row_stride * size % 16 != 0 || t->head_stride * size % 16 != 0)
    return make_status(SUBM_ERR_UNSUPPORTED, name + ": data and strides must be multiples of 16 bytes");
  const int64_t limit = (int64_t(1) << 22) / size;
  if (t->row_stride < 0 || t->head_stride < 0 || t->row_stride > limit || t->head_stride > limit)
    return make_status(SUBM_ERR_UNSUPPORTED, name + ": strides must be 0 .. 2^22 bytes");
  if (written && ((rows > 1 && t->row_stride == 0) || (heads > 1 && t->head_stride == 0)))
    return make_status(SUBM_ERR_INVALID_ARG, name + " is written and must not overlap itself");
  return Status{};
}

}  // namespace submconv

using namespace submconv;

extern "C" int sparse_attention_forward(const subm_heads_t* q, const subm_heads_t* k, const subm_heads_t* v, int64_t nq,
                                        int64_t nk, const int64_t* q_offsets, const int64_t* k_offsets, int items,
                                        int heads, int kv_heads, int head_dim, int dtype, float scale,
                                        const subm_heads_t* out, float* lse, hipStream_t stream) {
  clear_error();
  const AttentionShape shape{nq, nk, q_offsets, k_offsets, items, heads, kv_heads, head_dim, dtype, scale};
  Status st = check_attention(shape);
  if (st.ok()) st = check_heads(q, nq, heads, shape, false, "q");
  if (st.ok()) st = check_heads(k, nk, kv_heads, shape, false, "k");
  if (st.ok()) st = check_heads(v, nk, kv_heads, shape, false, "v");
  if (st.ok()) st = check_heads(out, nq, heads, shape, true, "out");
  if (!st.ok()) return fail(st);
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return fail(SUBM_ERR_INVALID_ARG, "lse is not 4-byte aligned");
  if (nq == 0) return SUBM_OK;
  const FwdArgs a{*q, *k, *v, *out, lse, q_offsets, k_offsets, nq, nk, items, heads, kv_heads, head_dim, scale};
  hipError_t e;
  if (dtype == SUBM_F32) e = launch_dim<DT::F32>(a, stream);
  else if (dtype == SUBM_F16) e = launch_dim<DT::F16>(a, stream);
  else e = launch_dim<DT::BF16>(a, stream);
  if (e != hipSuccess) return fail(hip_status(e, "sparse_attention_forward launch"));
  return SUBM_OK;
}
