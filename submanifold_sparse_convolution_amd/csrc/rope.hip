// Rotary positions (include/sparse_transformer.h): pair i of a head's `pairs` channel pairs turns
// by t = position[axis i / num_freq] * freq[i % num_freq],
//   (u, v) -> m (u cos t - v sin t, v cos t + u sin t);
// the gradient is the same rotation by -t.  The other channels are copied.
//
// Bound by HBM: 2 values an element, 3 operations.  A thread takes one 16-byte unit of a row's
// head, computes its sines once and then walks the heads, so the sines cost 1 / heads of what
// they would cost an element.
#include <algorithm>
#include <cmath>

#include "chunk.h"
#include "device_common.h"
#include "internal.h"
#include "sparse_transformer.h"

namespace submconv {
namespace {

struct RopeArgs {
  const void* x;
  void* y;
  int64_t n, x_row, x_head, y_row, y_head;
  const int32_t* positions;
  int64_t pos_row;
  const float* freq;
  int heads, head_dim, pairs, num_freq, heads_per_group;
  float magnitude, sign;
};

// magnitude * (cos, sin) of one pair's angle.  The turns are position * freq / (2 pi), formed and
// reduced in float64: float32 would keep only 24 bits of an angle that passes 2^13 radians.
__device__ __forceinline__ float2 rotation(const RopeArgs& a, int64_t row, int pair) {
  const double inv_2pi = 0.15915494309189533577;
  double turns = (double)a.positions[row * a.pos_row + pair / a.num_freq] * (double)a.freq[pair % a.num_freq] * inv_2pi;
  turns -= rint(turns);
  float s, c;
  sincospif(2.f * (float)turns, &s, &c);
  return make_float2(c * a.magnitude, s * a.magnitude * a.sign);
}

// One thread: unit `unit` of row `row`, heads [group * heads_per_group, ...).  Units of a head:
//   interleaved: the chunks of its channels (pairs never straddle two);
//   half-split:  the chunks of the first channels of its pairs, each with its partner chunk
//                `pairs` further on, then the chunks of the channels past the pairs (copied).
template <DT D, bool HALF>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, int units, int groups) {
  using T = typename Elem<D>::T;
  constexpr int V = kChunk<D>;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t rg = id / units;
  const int unit = (int)(id - rg * units);
  const int64_t row = rg / groups;
  const int group = (int)(rg - row * groups);
  if (row >= a.n) return;
  const int h0 = group * a.heads_per_group;
  const int h1 = min(a.heads, h0 + a.heads_per_group);
  const T* x = static_cast<const T*>(a.x) + row * a.x_row;
  T* y = static_cast<T*>(a.y) + row * a.y_row;
  const int rotated = 2 * a.pairs;
  if constexpr (HALF) {
    const int turning = (a.pairs + V - 1) / V;
    if (unit >= turning) {
      const int c = rotated + (unit - turning) * V;
      for (int h = h0; h < h1; ++h) store_raw<D>(y + h * a.y_head, c, a.head_dim, load_raw<D>(x + h * a.x_head, c, a.head_dim));
      return;
    }
    const int c = unit * V;
    float2 cs[V];
#pragma unroll
    for (int j = 0; j < V; ++j) cs[j] = c + j < a.pairs ? rotation(a, row, c + j) : make_float2(1.f, 0.f);
    for (int h = h0; h < h1; ++h) {
      float u[V], v[V], ou[V], ov[V];
      load_chunk<D>(x + h * a.x_head, c, a.pairs, u);
      load_chunk<D>(x + h * a.x_head + a.pairs, c, a.pairs, v);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        ou[j] = u[j] * cs[j].x - v[j] * cs[j].y;
        ov[j] = v[j] * cs[j].x + u[j] * cs[j].y;
      }
      store_chunk<D>(y + h * a.y_head, c, a.pairs, ou);
      store_chunk<D>(y + h * a.y_head + a.pairs, c, a.pairs, ov);
    }
  } else {
    const int c = unit * V;
    float2 cs[V / 2];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) cs[j] = c + 2 * j < rotated ? rotation(a, row, c / 2 + j) : make_float2(1.f, 0.f);
    for (int h = h0; h < h1; ++h) {
      auto w = load_raw<D>(x + h * a.x_head, c, a.head_dim);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        if (c + 2 * j < rotated) {  // (channels past the pairs are copied bit for bit)
          const float u = to_float<D>(w.v[2 * j]), v = to_float<D>(w.v[2 * j + 1]);
          w.v[2 * j] = from_float<D>(u * cs[j].x - v * cs[j].y);
          w.v[2 * j + 1] = from_float<D>(v * cs[j].x + u * cs[j].y);
        }
      }
      store_raw<D>(y + h * a.y_head, c, a.head_dim, w);
    }
  }
}

template <DT D, bool HALF>
hipError_t launch(RopeArgs a, hipStream_t stream) {
  constexpr int V = kChunk<D>;
  const int units = HALF ? (a.pairs + V - 1) / V + (a.head_dim - 2 * a.pairs + V - 1) / V : (a.head_dim + V - 1) / V;
  // Heads split into groups only while the rows alone leave compute units without a workgroup:
  // each further group computes the sines of its pairs again.
  int groups = 1;
  while (groups * 2 <= a.heads && a.n * units * groups < 256 * 256) groups *= 2;
  a.heads_per_group = (a.heads + groups - 1) / groups;
  groups = (a.heads + a.heads_per_group - 1) / a.heads_per_group;
  const int64_t blocks = (a.n * units * groups + 255) / 256;
  if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
  rope_kernel<D, HALF><<<(unsigned)blocks, 256, 0, stream>>>(a, units, groups);
  return hipGetLastError();
}

int rope(const subm_heads_t* x, int64_t n, int heads, int head_dim, int dtype, const int32_t* positions,
         int64_t position_stride, int axes, const float* freq, int num_freq, int layout, float magnitude, float sign,
         const subm_heads_t* y, hipStream_t stream, const char* what) {
  clear_error();
  if (dtype != SUBM_F32 && dtype != SUBM_F16 && dtype != SUBM_BF16)
    return fail(SUBM_ERR_UNSUPPORTED, "dtype must be SUBM_F32, SUBM_F16 or SUBM_BF16");
  if (layout != SUBM_ROPE_INTERLEAVED && layout != SUBM_ROPE_HALF)
    return fail(SUBM_ERR_INVALID_ARG, "layout must be SUBM_ROPE_INTERLEAVED or SUBM_ROPE_HALF");
  if (n < 0 || n > INT32_MAX) return fail(SUBM_ERR_INVALID_ARG, "n must be 0 .. 2^31 - 1");
  if (heads < 1 || heads > 65535) return fail(SUBM_ERR_INVALID_ARG, "heads must be 1 .. 65535");
  if (head_dim < 1 || head_dim > 4096) return fail(SUBM_ERR_INVALID_ARG, "head_dim must be 1 .. 4096");
  if (axes < 1 || num_freq < 1 || (int64_t)axes * num_freq * 2 > head_dim)
    return fail(SUBM_ERR_INVALID_ARG, "2 axes num_freq must be 2 .. head_dim");
  if (!std::isfinite(magnitude)) return fail(SUBM_ERR_INVALID_ARG, "magnitude must be finite");
  if (n == 0) return SUBM_OK;
  if (x == nullptr || y == nullptr || x->data == nullptr || y->data == nullptr || positions == nullptr || freq == nullptr)
    return fail(SUBM_ERR_INVALID_ARG, "x, y, positions or freq is NULL");
  const int size = dtype == SUBM_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x->data) % size != 0 || reinterpret_cast<uintptr_t>(y->data) % size != 0 ||
      reinterpret_cast<uintptr_t>(positions) % 4 != 0 || reinterpret_cast<uintptr_t>(freq) % 4 != 0)
    return fail(SUBM_ERR_INVALID_ARG, "a pointer is not aligned to its element");
  if (x->data == y->data && (x->row_stride != y->row_stride || x->head_stride != y->head_stride))
    return fail(SUBM_ERR_INVALID_ARG, "in place needs the same strides");
  if ((n > 1 && y->row_stride == 0) || (heads > 1 && y->head_stride == 0))
    return fail(SUBM_ERR_INVALID_ARG, "y is written and must not overlap itself");
  RopeArgs a{};
  a.x = x->data;
  a.y = y->data;
  a.n = n;
  a.x_row = x->row_stride;
  a.x_head = x->head_stride;
  a.y_row = y->row_stride;
  a.y_head = y->head_stride;
  a.positions = positions;
  a.pos_row = position_stride;
  a.freq = freq;
  a.heads = heads;
  a.head_dim = head_dim;
  a.pairs = axes * num_freq;
  a.num_freq = num_freq;
  a.magnitude = magnitude;
  a.sign = sign;
  hipError_t e;
  const bool half = layout == SUBM_ROPE_HALF;
  if (dtype == SUBM_F32) e = half ? launch<DT::F32, true>(a, stream) : launch<DT::F32, false>(a, stream);
  else if (dtype == SUBM_F16) e = half ? launch<DT::F16, true>(a, stream) : launch<DT::F16, false>(a, stream);
  else e = half ? launch<DT::BF16, true>(a, stream) : launch<DT::BF16, false>(a, stream);
  if (e != hipSuccess) return fail(hip_status(e, what));
  return SUBM_OK;
}

}  // namespace
}  // namespace submconv

using namespace submconv;

extern "C" int sparse_rope_frequencies(int count, double base, int scaling, double factor, double trained_length,
                                       float* freq, float* magnitude) {
  clear_error();
  if (count < 1) return fail(SUBM_ERR_INVALID_ARG, "count must be at least 1");
  if (!(base > 1.0) || !std::isfinite(base)) return fail(SUBM_ERR_INVALID_ARG, "base must be above 1 and finite");
  if (scaling < SUBM_ROPE_PLAIN || scaling > SUBM_ROPE_PARTS) return fail(SUBM_ERR_INVALID_ARG, "unknown scaling");
  if (!(factor >= 1.0) || !std::isfinite(factor)) return fail(SUBM_ERR_INVALID_ARG, "factor must be at least 1 and finite");
  if (scaling == SUBM_ROPE_PARTS && (!(trained_length > 0.0) || !std::isfinite(trained_length)))
    return fail(SUBM_ERR_INVALID_ARG, "trained_length must be positive and finite");
  if (freq == nullptr) return fail(SUBM_ERR_INVALID_ARG, "freq is NULL");
  if (scaling == SUBM_ROPE_BASE && count > 1) base *= std::pow(factor, (double)count / (count - 1));
  for (int i = 0; i < count; ++i) {
    double f = std::pow(base, -(double)i / count);
    if (scaling == SUBM_ROPE_LINEAR) f /= factor;
    if (scaling == SUBM_ROPE_PARTS) {
      const double turns = trained_length * f / (2.0 * 3.14159265358979323846);
      const double keep = std::min(1.0, std::max(0.0, (turns - 1.0) / 31.0));
      f = f * keep + f / factor * (1.0 - keep);
    }
    freq[i] = (float)f;
  }
  if (magnitude != nullptr) *magnitude = scaling == SUBM_ROPE_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return SUBM_OK;
}

extern "C" int sparse_rope_forward(const subm_heads_t* x, int64_t n, int heads, int head_dim, int dtype,
                                   const int32_t* positions, int64_t position_stride, int axes, const float* freq,
                                   int num_freq, int layout, float magnitude, const subm_heads_t* y,
                                   hipStream_t stream) {
  return rope(x, n, heads, head_dim, dtype, positions, position_stride, axes, freq, num_freq, layout, magnitude, 1.f,
              y, stream, "sparse_rope_forward launch");
}

extern "C" int sparse_rope_backward(const subm_heads_t* dy, int64_t n, int heads, int head_dim, int dtype,
                                    const int32_t* positions, int64_t position_stride, int axes, const float* freq,
                                    int num_freq, int layout, float magnitude, const subm_heads_t* dx,
                                    hipStream_t stream) {
  return rope(dy, n, heads, head_dim, dtype, positions, position_stride, axes, freq, num_freq, layout, magnitude,
              -1.f, dx, stream, "sparse_rope_backward launch");
}
