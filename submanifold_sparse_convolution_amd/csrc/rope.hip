// Rotary positions (include/sparse_transformer.h): pair i of a head's `pairs` channel pairs turns
// by t = position[axis i / num_freq] * freq[i % num_freq],
//   (u, v) -> m (u cos t - v sin t, v cos t + u sin t);
// the gradient is the same rotation by -t.  The other channels are copied.
//
// Bound by HBM: 2 values an element, 3 operations.  A workgroup first computes the sines of its
// rows into LDS, once for all heads (each costs some 40 instructions), and then walks the rows'
// 16-byte units in storage order (65,536 tokens, 20 heads of 128, bf16: 159 us, 4.2 TB/s; 238 with the
// sines computed at each use).
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
  int heads, head_dim, pairs, num_freq;
  float magnitude, sign;
  // a workgroup takes `rows` rows of `group` heads, `units` units a head (see rope_kernel)
  int rows, group, units;
  uint32_t unit_magic, group_magic;  // ceil(2^32 / units), ceil(2^32 / group)
};

// i / d for i < 2^16 and magic = ceil(2^32 / d), d < 2^16 (magic 0: d is 1).
__device__ __forceinline__ int divide(int i, uint32_t magic) { return magic == 0 ? i : (int)__umulhi((uint32_t)i, magic); }

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

constexpr int kThreads = 256;
constexpr int kBatch = 2;               // units a thread has in flight
constexpr int kSines = 4096;            // LDS: float2 of rows * pairs, 32 KB

// Units of a head:
//   interleaved: the chunks of its channels (pairs never straddle two);
//   half-split:  the chunks of the first channels of its pairs, each with its partner chunk
//                `pairs` further on, then the chunks of the channels past the pairs (copied).
template <DT D, bool HALF>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a) {
  using T = typename Elem<D>::T;
  constexpr int V = kChunk<D>;
  extern __shared__ float2 s_turn[];  // [rows, pairs]
  const int64_t row0 = (int64_t)blockIdx.x * a.rows;
  const int rows = (int)(a.n - row0 < a.rows ? a.n - row0 : a.rows);
  const int head0 = blockIdx.y * a.group, group = min(a.group, a.heads - head0);
  for (int i = threadIdx.x; i < rows * a.pairs; i += kThreads) {
    const int r = i / a.pairs;
    s_turn[i] = rotation(a, row0 + r, i - r * a.pairs);
  }
  __syncthreads();
  const T* x = static_cast<const T*>(a.x) + row0 * a.x_row + head0 * a.x_head;
  T* y = static_cast<T*>(a.y) + row0 * a.y_row + head0 * a.y_head;
  const int rotated = 2 * a.pairs, turning = HALF ? (a.pairs + V - 1) / V : 0;
  const int total = rows * a.group * a.units;
  for (int i0 = threadIdx.x; i0 < total; i0 += kThreads * kBatch) {
    Chunk<T, V> u[kBatch], v[kBatch];
    const T* px[kBatch];
    T* py[kBatch];
    const float2* turn[kBatch];
    int c[kBatch], end[kBatch];  // first channel and the end of its kind (0: no unit)
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int i = i0 + b * kThreads;
      const int rh = divide(i, a.unit_magic), unit = i - rh * a.units;
      const int r = divide(rh, a.group_magic), h = rh - r * a.group;
      px[b] = x + r * a.x_row + h * a.x_head;
      py[b] = y + r * a.y_row + h * a.y_head;
      turn[b] = s_turn + r * a.pairs;
      const bool copied = HALF && unit >= turning;
      c[b] = HALF && copied ? rotated + (unit - turning) * V : unit * V;
      end[b] = i < total && h < group ? (HALF && !copied ? a.pairs : a.head_dim) : 0;
      if (end[b] != 0) {
        u[b] = load_raw<D>(px[b], c[b], end[b]);
        if (HALF && !copied) v[b] = load_raw<D>(px[b] + a.pairs, c[b], end[b]);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (end[b] == 0) continue;
      if constexpr (HALF) {
        if (c[b] < rotated) {
          float fu[V], fv[V];
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float2 t = c[b] + j < a.pairs ? turn[b][c[b] + j] : make_float2(1.f, 0.f);
            const float p = to_float<D>(u[b].v[j]), q = to_float<D>(v[b].v[j]);
            fu[j] = p * t.x - q * t.y;
            fv[j] = q * t.x + p * t.y;
          }
          u[b] = pack_chunk<D>(fu);
          store_raw<D>(py[b] + a.pairs, c[b], end[b], pack_chunk<D>(fv));
        }
      } else {
        float f[V];
#pragma unroll
        for (int j = 0; j < V; j += 2) {
          const float2 t = c[b] + j < rotated ? turn[b][(c[b] + j) / 2] : make_float2(1.f, 0.f);
          const float p = to_float<D>(u[b].v[j]), q = to_float<D>(u[b].v[j + 1]);
          f[j] = p * t.x - q * t.y;
          f[j + 1] = q * t.x + p * t.y;
        }
        const Chunk<T, V> turned = pack_chunk<D>(f);
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (c[b] + j < rotated) u[b].v[j] = turned.v[j];  // (channels past the pairs are copied bit for bit)
      }
      store_raw<D>(py[b], c[b], end[b], u[b]);
    }
  }
}

uint32_t magic(int d) { return d == 1 ? 0u : (uint32_t)((0x100000000ull + d - 1) / d); }

template <DT D, bool HALF>
hipError_t launch(RopeArgs a, hipStream_t stream) {
  constexpr int V = kChunk<D>;
  a.units = HALF ? (a.pairs + V - 1) / V + (a.head_dim - 2 * a.pairs + V - 1) / V : (a.head_dim + V - 1) / V;
  // Heads of a workgroup: all, up to 2^13 units.  Rows: some 2,048 units a workgroup, fewer while
  // that leaves compute units without one, and no more than the sines of LDS.
  a.group = std::min(a.heads, std::max(1, 8192 / a.units));
  const int groups = (a.heads + a.group - 1) / a.group;
  int64_t rows = std::max<int64_t>(1, 2048 / (a.group * a.units));
  rows = std::min<int64_t>(rows, std::max<int64_t>(1, a.n * groups / 1024));
  rows = std::min<int64_t>(rows, std::max(1, kSines / a.pairs));
  a.rows = (int)rows;
  a.unit_magic = magic(a.units);
  a.group_magic = magic(a.group);
  const int64_t blocks = (a.n + a.rows - 1) / a.rows;
  const size_t lds = (size_t)a.rows * a.pairs * sizeof(float2);
  rope_kernel<D, HALF><<<dim3((unsigned)blocks, (unsigned)groups), kThreads, lds, stream>>>(a);
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
  return no_throw([&]() -> int {
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
  });
}

extern "C" int sparse_rope_forward(const subm_heads_t* x, int64_t n, int heads, int head_dim, int dtype,
                                   const int32_t* positions, int64_t position_stride, int axes, const float* freq,
                                   int num_freq, int layout, float magnitude, const subm_heads_t* y,
                                   hipStream_t stream) {
  return no_throw([&]() -> int {
    return rope(x, n, heads, head_dim, dtype, positions, position_stride, axes, freq, num_freq, layout, magnitude, 1.f,
                y, stream, "sparse_rope_forward launch");
  });
}

extern "C" int sparse_rope_backward(const subm_heads_t* dy, int64_t n, int heads, int head_dim, int dtype,
                                    const int32_t* positions, int64_t position_stride, int axes, const float* freq,
                                    int num_freq, int layout, float magnitude, const subm_heads_t* dx,
                                    hipStream_t stream) {
  return no_throw([&]() -> int {
    return rope(dy, n, heads, head_dim, dtype, positions, position_stride, axes, freq, num_freq, layout, magnitude,
                -1.f, dx, stream, "sparse_rope_backward launch");
  });
}
