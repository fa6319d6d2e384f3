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
//
// Measured: items of 13,001 and 11,575 tokens, 16 heads of 128, bf16: 2.23 ms, 1.11 PFLOP/s (matrix
// cores busy 58 % of the cycles, at a clock that the power limit holds near 1.8 GHz; in a trace of 30
// calls 2.20 to 2.29 ms); four items of 450 to 4,001 queries and up to 1,374 keys, 12 heads of 64, f16:
// 48 us, 0.53 PFLOP/s (636 workgroups of unequal length at once, each product of 64 channels beside as
// many exponentials); 8 single tokens, up to 32,768 keys each, 16 / 4 heads of 128, bf16: 87 us, 4.9
// TB/s.
#include "attention_forward.h"

namespace submconv {

Status check_attention(const AttentionShape& s) {
  if (s.dtype != SUBM_F32 && s.dtype != SUBM_F16 && s.dtype != SUBM_BF16)
    return make_status(SUBM_ERR_UNSUPPORTED, "dtype must be SUBM_F32, SUBM_F16 or SUBM_BF16");
  // Rows are counted in 32 bits, up to a few tiles past the last, and a launch of 256 threads for each
  // 128 of them (and one more an item) has at most 2^32 - 1.
  constexpr int64_t kMost = (int64_t(1) << 31) - (int64_t(1) << 24);
  if (s.nq < 0 || s.nk < 0 || s.nq > kMost || s.nk > kMost)
    return make_status(SUBM_ERR_INVALID_ARG, "nq and nk must be 0 .. 2^31 - 2^24");
  if (s.items < 1 || s.items > 65535) return make_status(SUBM_ERR_INVALID_ARG, "items must be 1 .. 65535");
  if (s.heads < 1 || s.kv_heads < 1 || s.heads % s.kv_heads != 0)
    return make_status(SUBM_ERR_INVALID_ARG, "heads must be a positive multiple of kv_heads");
  if (s.kv_heads > 65535) return make_status(SUBM_ERR_INVALID_ARG, "kv_heads exceeds 65535");
  if (s.heads / s.kv_heads > 128) return make_status(SUBM_ERR_UNSUPPORTED, "more than 128 query heads a key head");
  if (s.nq * s.heads > kMost) return make_status(SUBM_ERR_INVALID_ARG, "nq * heads exceeds 2^31 - 2^24");
  if (s.head_dim < 1) return make_status(SUBM_ERR_INVALID_ARG, "head_dim must be at least 1");
  if (s.head_dim % 8 != 0 || s.head_dim > 128)
    return make_status(SUBM_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 up to 128");
  if (!std::isfinite(s.scale)) return make_status(SUBM_ERR_INVALID_ARG, "scale must be finite");
  if (s.q_offsets == nullptr || s.k_offsets == nullptr)
    return make_status(SUBM_ERR_INVALID_ARG, "q_offsets or k_offsets is NULL");
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
  // (a tile of 32 rows is addressed with 31 bits from its first token)
  if (t->head_stride * size * (heads / std::max(s.kv_heads, 1)) > (int64_t(1) << 30))
    return make_status(SUBM_ERR_UNSUPPORTED, name + ": the heads of one key head span more than 2^30 bytes");
  if (written && ((rows > 1 && t->row_stride == 0) || (heads > 1 && t->head_stride == 0)))
    return make_status(SUBM_ERR_INVALID_ARG, name + " is written and must not overlap itself");
  return Status{};
}

Status check_forward(const subm_heads_t* q, const subm_heads_t* k, const subm_heads_t* v, const subm_heads_t* out,
                     const float* lse, const AttentionShape& s) {
  Status st = check_heads(q, s.nq, s.heads, s, false, "q");
  if (st.ok()) st = check_heads(k, s.nk, s.kv_heads, s, false, "k");
  if (st.ok()) st = check_heads(v, s.nk, s.kv_heads, s, false, "v");
  if (st.ok()) st = check_heads(out, s.nq, s.heads, s, true, "out");
  if (!st.ok()) return st;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return make_status(SUBM_ERR_INVALID_ARG, "lse is not 4-byte aligned");
  if (s.nq == 0) return Status{};
  if (out->data == k->data || out->data == v->data) return make_status(SUBM_ERR_INVALID_ARG, "out must not alias k or v");
  if (out->data == q->data &&
      ((s.nq > 1 && out->row_stride != q->row_stride) || (s.heads > 1 && out->head_stride != q->head_stride)))
    return make_status(SUBM_ERR_INVALID_ARG, "out over q needs the same strides");
  return Status{};
}

}  // namespace submconv

using namespace submconv;

extern "C" int sparse_attention_forward(const subm_heads_t* q, const subm_heads_t* k, const subm_heads_t* v, int64_t nq,
                                        int64_t nk, const int64_t* q_offsets, const int64_t* k_offsets, int items,
                                        int heads, int kv_heads, int head_dim, int dtype, float scale,
                                        const subm_heads_t* out, float* lse, hipStream_t stream) {
  return no_throw([&]() -> int {
    clear_error();
    const AttentionShape shape{nq, nk, q_offsets, k_offsets, items, heads, kv_heads, head_dim, dtype, scale};
    Status st = check_attention(shape);
    if (st.ok()) st = check_forward(q, k, v, out, lse, shape);
    if (!st.ok()) return fail(st);
    if (nq == 0) return SUBM_OK;
    const FwdArgs a{*q, *k, *v, *out, lse, q_offsets, k_offsets, nq, nk, items, heads, kv_heads,
                    head_dim, scale, Cut{}, nullptr, nullptr, Window{}};
    if (dtype == SUBM_F32) st = launch_dim<DT::F32, false>(a, stream);
    else if (dtype == SUBM_F16) st = launch_dim<DT::F16, false>(a, stream);
    else st = launch_dim<DT::BF16, false>(a, stream);
    if (!st.ok()) return fail(st);
    return SUBM_OK;
  });
}
