// Rows spread over lanes: what the row-wise kernels (norms, embedding) share.
#pragma once

#include "device_common.h"

namespace submconv {

// TPR lanes (a part of a wave, a wave, or a workgroup of TPR threads) hold one row, ITEMS chunks of V
// values each.

template <int CTRL> __device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}

// Sum over aligned groups of LANES lanes, the same in every lane, in VALU instructions alone (an LDS
// permutation a step would cost a row some 12 LDS round trips in the backward pass).
template <int LANES> __device__ __forceinline__ float lanes_sum(float v) {
  static_assert(LANES == 8 || LANES == 16 || LANES == 32 || LANES == 64, "lanes of a row");
  v = dpp_add<0xB1>(v);   // quads: lanes 1 0 3 2
  v = dpp_add<0x4E>(v);   // quads: lanes 2 3 0 1
  v = dpp_add<0x141>(v);  // half rows mirrored
  if constexpr (LANES == 8) return v;
  v = dpp_add<0x140>(v);  // rows of 16 mirrored
  if constexpr (LANES == 16) return v;
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  if constexpr (LANES == 32) return v;
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(h[0]) + __uint_as_float(h[1]);
}

// Sum over the TPR lanes of a row, the same in all of them.  For TPR > 64 every thread of the
// workgroup must call it (it synchronises), with a slot array of its own per call site.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* slots) {
  v = lanes_sum<TPR < 64 ? TPR : 64>(v);
  if constexpr (TPR > 64) {
    __syncthreads();  // the slots' readers of the previous row are done
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) v += slots[w];
  }
  return v;
}

// The largest over aligned groups of `lanes` lanes (4 .. 64, a power of two, the same in the whole
// wave), the same in every lane of a group.  NaN counts for nothing.
template <int CTRL> __device__ __forceinline__ float dpp_max(float v) {
  return fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xf, 0xf, true)));
}
__device__ __forceinline__ float lanes_max(float v, int lanes) {
  v = dpp_max<0xB1>(v);
  v = dpp_max<0x4E>(v);
  if (lanes > 4) v = dpp_max<0x141>(v);
  if (lanes > 8) v = dpp_max<0x140>(v);
  if (lanes > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if (lanes > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}

constexpr int threads_for(int tpr) { return tpr > 256 ? tpr : 256; }

// Lanes of a row: short rows share a wave (179,096 x 48 bf16, forward: 8.1 us, 45 with a wave a row).
inline int short_lanes(int chunks) { return chunks <= 8 ? 8 : chunks <= 16 ? 16 : chunks <= 32 ? 32 : 64; }

}  // namespace submconv
