// 16-byte chunks of a row at element alignment, with element-wise ends: what the row-wise
// kernels (layer norm, rotary positions) load and store.
#pragma once

#include "device_common.h"

namespace submconv {

template <DT D> constexpr int kChunk = 16 / Elem<D>::kSize;  // values of a chunk

// (Global loads and stores need no more than element alignment, so rows of any length and start
// take the wide form.)
template <typename T, int V> struct __attribute__((packed, aligned(sizeof(T)))) Chunk { T v[V]; };

// Values p[c0 .. c0 + V), those at or past `end` zero.  TAIL: `end` may lie inside the chunk, which
// then goes element by element; else it is a multiple of V.
template <DT D, bool TAIL = true>
__device__ __forceinline__ Chunk<typename Elem<D>::T, kChunk<D>> load_raw(const typename Elem<D>::T* p, int c0, int end) {
  using C = Chunk<typename Elem<D>::T, kChunk<D>>;
  if (c0 + kChunk<D> <= end) return *reinterpret_cast<const C*>(p + c0);
  C c;
#pragma unroll
  for (int j = 0; j < kChunk<D>; ++j) c.v[j] = TAIL && c0 + j < end ? p[c0 + j] : (typename Elem<D>::T)0;
  return c;
}

template <DT D, bool TAIL = true>
__device__ __forceinline__ void store_raw(typename Elem<D>::T* p, int c0, int end,
                                          const Chunk<typename Elem<D>::T, kChunk<D>>& c) {
  using C = Chunk<typename Elem<D>::T, kChunk<D>>;
  if (c0 + kChunk<D> <= end) {
    *reinterpret_cast<C*>(p + c0) = c;
  } else if constexpr (TAIL) {
#pragma unroll
    for (int j = 0; j < kChunk<D>; ++j)
      if (c0 + j < end) p[c0 + j] = c.v[j];
  }
}

template <DT D, bool TAIL = true>
__device__ __forceinline__ void load_chunk(const typename Elem<D>::T* p, int c0, int end, float (&out)[kChunk<D>]) {
  const auto c = load_raw<D, TAIL>(p, c0, end);
#pragma unroll
  for (int j = 0; j < kChunk<D>; ++j) out[j] = to_float<D>(c.v[j]);
}

// float -> storage of a whole chunk, to nearest even (hardware conversions of pairs).
template <DT D> __device__ __forceinline__ Chunk<typename Elem<D>::T, kChunk<D>> pack_chunk(const float (&in)[kChunk<D>]) {
  Chunk<typename Elem<D>::T, kChunk<D>> c;
  if constexpr (D == DT::F32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c.v[j] = in[j];
  } else {
    const uint2 lo = pack4<D>(in[0], in[1], in[2], in[3]), hi = pack4<D>(in[4], in[5], in[6], in[7]);
    const uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
    for (int j = 0; j < 8; ++j) c.v[j] = (uint16_t)(w[j / 2] >> (j % 2 * 16));
  }
  return c;
}

template <DT D, bool TAIL = true>
__device__ __forceinline__ void store_chunk(typename Elem<D>::T* p, int c0, int end, const float (&in)[kChunk<D>]) {
  store_raw<D, TAIL>(p, c0, end, pack_chunk<D>(in));
}

}  // namespace submconv
