// Attention within a sliding window that keeps an item's first keys visible, backward pass
// (include/sparse_transformer.h).
//
// The kernels of attention_backward.hip over fewer rows: dq walks the keys that the forward pass walks, dk and
// dv of a block of keys the query rows from the first that sees its first key to the last that sees its
// last.  The sinks are seen by nearly every row, which would make their blocks as long as the whole item:
// chunks of rows leave float32 sums for them, which a last kernel adds up in order.
//
// float16: the scale of e (attention_backward.hip) goes by what is seen alone: for a row of dq by its own |dout|
// and the longest v among its keys, for a key of dk by the rows that see it.  A scale that took in a hidden value
// would leave small e among the subnormals (dout of order 2^-7, a hidden |v| of 60,000 in 128 channels).  The kernel
// of v's norms leaves one a key for it, dq a bound a row, and the waves take running maxima over those
// (range_max): forward and backward, five items to 2,971 tokens, 12 / 4 heads of 64, causal: 279 -> 284 us; 9,000
// and 7,384 tokens, 16 heads of 128, 1,024 keys and 4 sinks: 864 -> 875; two items of 4,096, 16 heads a key head, 512
// keys: 197 -> 209.
//
// Measured, with the forward pass: 9,000 and 7,384 tokens, 16 heads of 128, bf16, 1,024 keys and 4 sinks: 790 us
// (177 forward, dq 250, dk and dv 300, the sinks' 38 and 6); five items to 2,971 tokens, 12 / 4 heads of 64, f16,
// causal: 278 us (66 forward, dq 93, dk and dv 111, 13 the sums of parts, 5 the norms of v).  Matrix cores busy 40 %
// and 23 % of the cycles, vector units 26 to 36: nothing is full, a step's parts wait for each other.
#include "attention_gradient.h"

using namespace submconv;

extern "C" int sparse_window_attention_backward(const subm_heads_t* dout, const subm_heads_t* q, const subm_heads_t* k,
                                                const subm_heads_t* v, const subm_heads_t* out, const float* lse,
                                                int64_t nq, int64_t nk, const int64_t* q_offsets,
                                                const int64_t* k_offsets, int items, int heads, int kv_heads,
                                                int head_dim, int dtype, float scale, int64_t left, int64_t right,
                                                int sinks, const subm_heads_t* dq, const subm_heads_t* dk,
                                                const subm_heads_t* dv, hipStream_t stream) {
  return no_throw([&]() -> int {
    clear_error();
    const AttentionShape shape{nq, nk, q_offsets, k_offsets, items, heads, kv_heads, head_dim, dtype, scale};
    Window window{};
    Status st = check_attention(shape);
    if (st.ok()) st = check_window(left, right, sinks, nullptr, &window);
    if (st.ok()) st = check_backward(dout, q, k, v, out, lse, dq, dk, dv, shape);
    if (!st.ok()) return fail(st);
    if (nq == 0 && nk == 0) return SUBM_OK;
    BwdArgs a = backward_args(dout, q, k, v, out, lse, dq, dk, dv, shape);
    a.window = window;
    if (dtype == SUBM_F32) st = launch_dim<DT::F32, true>(a, stream);
    else if (dtype == SUBM_F16) st = launch_dim<DT::F16, true>(a, stream);
    else st = launch_dim<DT::BF16, true>(a, stream);
    if (!st.ok()) return fail(st);
    return SUBM_OK;
  });
}
