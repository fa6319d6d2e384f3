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
#include "attention_gradient.h"

namespace submconv {

Status check_backward(const subm_heads_t* dout, const subm_heads_t* q, const subm_heads_t* k, const subm_heads_t* v,
                      const subm_heads_t* out, const float* lse, const subm_heads_t* dq, const subm_heads_t* dk,
                      const subm_heads_t* dv, const AttentionShape& s) {
  Status st = check_heads(dout, s.nq, s.heads, s, false, "dout");
  if (st.ok()) st = check_heads(q, s.nq, s.heads, s, false, "q");
  if (st.ok()) st = check_heads(k, s.nk, s.kv_heads, s, false, "k");
  if (st.ok()) st = check_heads(v, s.nk, s.kv_heads, s, false, "v");
  if (st.ok()) st = check_heads(out, s.nq, s.heads, s, false, "out");
  if (st.ok()) st = check_heads(dq, s.nq, s.heads, s, true, "dq");
  if (st.ok()) st = check_heads(dk, s.nk, s.kv_heads, s, true, "dk");
  if (st.ok()) st = check_heads(dv, s.nk, s.kv_heads, s, true, "dv");
  if (!st.ok()) return st;
  if (s.nq > 0 && lse == nullptr) return make_status(SUBM_ERR_INVALID_ARG, "lse is NULL");
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return make_status(SUBM_ERR_INVALID_ARG, "lse is not 4-byte aligned");
  if (s.nq == 0 && s.nk == 0) return Status{};
  // (the second kernel reads every input after the first has written dq)
  for (const subm_heads_t* w : {dq, dk, dv})
    for (const subm_heads_t* r : {dout, q, k, v, out})
      if (w->data != nullptr && w->data == r->data)
        return make_status(SUBM_ERR_INVALID_ARG, "a gradient must not alias an input");
  if (s.nq > 0 && s.nk > 0 && (dq->data == dk->data || dq->data == dv->data))
    return make_status(SUBM_ERR_INVALID_ARG, "dq, dk and dv must not alias");
  if (s.nk > 0 && dk->data == dv->data) return make_status(SUBM_ERR_INVALID_ARG, "dq, dk and dv must not alias");
  return Status{};
}

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
    if (st.ok()) st = check_backward(dout, q, k, v, out, lse, dq, dk, dv, shape);
    if (!st.ok()) return fail(st);
    if (nq == 0 && nk == 0) return SUBM_OK;
    const BwdArgs a = backward_args(dout, q, k, v, out, lse, dq, dk, dv, shape);
    if (dtype == SUBM_F32) st = launch_dim<DT::F32, false>(a, stream);
    else if (dtype == SUBM_F16) st = launch_dim<DT::F16, false>(a, stream);
    else st = launch_dim<DT::BF16, false>(a, stream);
    if (!st.ok()) return fail(st);
    return SUBM_OK;
  });
}
