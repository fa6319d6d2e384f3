// 16-byte chunks of a row at element alignment, with element-wise ends: what the row-wise
// kernels (layer norm, rotary positions) load and store.
#pragma once

#include "device_common.h"

namespace submconv {

template <DT D> constexpr int kChunk = 16 / Elem<D>::kSize;  // values of a chunk

// (Global loads and stores need no more than element alignment, so rows of any length and start
// take the wide form.)
template <typename T, int V> struct __attribute__((packed, aligned(sizeof(T)))) Chunk { T v[V]; };

// Values p[c0 .. c0 + V), those at or past `end` zero.
template <DT D>
__device__ __forceinline__ Chunk<typename Elem<D>::T, kChunk<D>> load_raw(const typename Elem<D>::T* p, int c0, int end) {
  using C = Chunk<typename Elem<D>::T, kChunk<D>>;
  if (c0 + kChunk<D> <= end) return *reinterpret_cast<const C*>(p + c0);
  C c;
#pragma unroll
  for (int j = 0; j < kChunk<D>; ++j) c.v[j] = c0 + j < end ? p[c0 + j] : (typename Elem<D>::T)0;
  return c;
}

template <DT D>
__device__ __forceinline__ void store_raw(typename Elem<D>::T* p, int c0, int end,
                                          const Chunk<typename Elem<D>::T, kChunk<D>>& c) {
  using C = Chunk<typename Elem<D>::T, kChunk<D>>;
  if (c0 + kChunk<D> <= end) {
    *reinterpret_cast<C*>(p + c0) = c;
  } else {
#pragma unroll
    for (int j = 0; j < kChunk<D>; ++j)
      if (c0 + j < end) p[c0 + j] = c.v[j];
  }
}

template <DT D>
__device__ __forceinline__ void load_chunk(const typename Elem<D>::T* p, int c0, int end, float (&out)[kChunk<D>]) {
  const auto c = load_raw<D>(p, c0, end);
#pragma unroll
  for (int j = 0; j < kChunk<D>; ++j) out[j] = to_float<D>(c.v[j]);
}

template <DT D>
__device__ __forceinline__ void store_chunk(typename Elem<D>::T* p, int c0, int end, const float (&in)[kChunk<D>]) {
  Chunk<typename Elem<D>::T, kChunk<D>> c;
#pragma unroll
  for (int j = 0; j < kChunk<D>; ++j) c.v[j] = from_float<D>(in[j]);
  store_raw<D>(p, c0, end, c);
}

}  // namespace submconv
