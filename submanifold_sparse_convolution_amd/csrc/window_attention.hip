// Attention within a sliding window that keeps an item's first keys visible, forward pass
// (include/sparse_transformer.h).
//
// The kernels of attention.hip over fewer keys: a block of query rows walks the tiles from its first row's
// first key to its last row's last, and those of the sinks before them (attention_window.h).
//
// Bound by products and exponentials in turn (24,576 tokens at 128 channels: matrix cores busy 50 % of the cycles,
// vector units 48; at 64 channels 22 and 47, and 900 tiles on 768 places), and with few rows by the latency of a
// short walk.  Measured: items of 13,001 and 11,575 tokens, 16 heads of 128, bf16, 2,048 keys and 4 sinks: 440 us (0.86
// PFLOP/s of what the rows see, 0.92 of what the tiles compute); four items, 9,371 tokens, 12 heads of 64, f16,
// 256 keys each way: 43 us; 8 single tokens, 16 / 4 heads of 128, bf16, 4,096 keys of caches to 32,768: 23 us, 59 MB.
#include "attention_forward.h"

namespace submconv {

Status check_window(int64_t left, int64_t right, int sinks, const int64_t* k_lengths, Window* w) {
  if (left < 0 || right < 0) return make_status(SUBM_ERR_INVALID_ARG, "left and right must not be negative");
  if (sinks < 0) return make_status(SUBM_ERR_INVALID_ARG, "sinks is negative");
  if (sinks > kMaxSinks) return make_status(SUBM_ERR_UNSUPPORTED, "sinks exceeds 128");
  if ((reinterpret_cast<uintptr_t>(k_lengths) & 7u) != 0)
    return make_status(SUBM_ERR_INVALID_ARG, "k_lengths is not 8-byte aligned");
  *w = Window{std::min(left, kOpen), std::min(right, kOpen), left >= kOpen ? 0 : sinks, k_lengths, false};
  return Status{};
}

}  // namespace submconv

using namespace submconv;

extern "C" int sparse_window_attention_forward(const subm_heads_t* q, const subm_heads_t* k, const subm_heads_t* v,
                                               int64_t nq, int64_t nk, const int64_t* q_offsets,
                                               const int64_t* k_offsets, const int64_t* k_lengths, int items, int heads,
                                               int kv_heads, int head_dim, int dtype, float scale, int64_t left,
                                               int64_t right, int sinks, const subm_heads_t* out, float* lse,
                                               hipStream_t stream) {
  return no_throw([&]() -> int {
    clear_error();
    const AttentionShape shape{nq, nk, q_offsets, k_offsets, items, heads, kv_heads, head_dim, dtype, scale};
    Window window{};
    Status st = check_attention(shape);
    if (st.ok()) st = check_window(left, right, sinks, k_lengths, &window);
    if (st.ok()) st = check_forward(q, k, v, out, lse, shape);
    if (!st.ok()) return fail(st);
    if (nq == 0) return SUBM_OK;
    const FwdArgs a{*q, *k, *v, *out, lse, q_offsets, k_offsets, nq, nk, items, heads, kv_heads,
                    head_dim, scale, Cut{}, nullptr, nullptr, window};
    if (dtype == SUBM_F32) st = launch_dim<DT::F32, true>(a, stream);
    else if (dtype == SUBM_F16) st = launch_dim<DT::F16, true>(a, stream);
    else st = launch_dim<DT::BF16, true>(a, stream);
    if (!st.ok()) return fail(st);
    return SUBM_OK;
  });
}
