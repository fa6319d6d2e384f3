// Root-mean-square norm of the rows of x + residual, forward (also to 8 bits with scales) and backward
// (include/sparse_transformer.h).
//
//   t = x + residual,  r = 1 / sqrt(sum t^2 / C + eps),  y = t r g
//   8 bits: s = max |y| / 448 over a group of channels (448: the largest e4m3 number),  q = y / s
//   h = t r,  a = dy g,  dx = r (a - h mean(a h)) + dt,  dg = sum_rows dy h
//
// Bound by HBM: a row is read once and stays in registers, spread over TPR lanes in 16-byte chunks,
// from its loads to its stores.  The norm is of the float32 sum, not of its rounding that is stored.
//
// Measured: 135,826 rows of 1,024 channels, bf16, with a residual: to 8 bits in groups 178 us (973 MB, 5.5 TB/s),
// backward with both gradients 207 us (1,113 MB, 5.4 TB/s); a 1 GiB copy reaches 5.49 TB/s.  4,099 rows of 675,
// float32, backward: 10 us and 4 for the weight's gradient, latency; 450 rows of 768, f16: 3.7 us.
#include <algorithm>
#include <cmath>

#include "chunk.h"
#include "device_common.h"
#include "internal.h"
#include "row_lanes.h"
#include "sparse_transformer.h"

namespace submconv {
namespace {

constexpr float kMostE4m3 = 448.f;
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126, which a group of zeros gets

struct RmsForward {
  const void *x, *residual, *gamma;
  void *total, *y;  // y: not with 8 bits
  uint8_t* q;
  float *scales, *rstd;
  float eps;
  int group;  // channels of a scale; 0: a row
};
struct RmsBackward {
  const void *dy, *total, *dtotal, *gamma;
  const float* rstd;
  void* dx;
  float* part;
};

// Eight or four values to e4m3, to nearest even.
template <int V> __device__ __forceinline__ Chunk<uint8_t, V> pack_e4m3(const float (&v)[V]) {
  Chunk<uint8_t, V> c;
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[i], v[i + 1], w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[i + 2], v[i + 3], w, true);
#pragma unroll
    for (int j = 0; j < 4; ++j) c.v[i + j] = (uint8_t)((uint32_t)w >> (8 * j));
  }
  return c;
}

// (x, residual, total and y may be one memory: none is declared free of aliases.)
template <DT D, int TPR, int ITEMS, bool TAIL, bool QUANT>
__global__ __launch_bounds__(threads_for(TPR)) void rms_norm_forward_kernel(RmsForward a, int64_t n, int channels) {
  using T = typename Elem<D>::T;
  constexpr int V = kChunk<D>;
  constexpr int kRows = threads_for(TPR) / TPR;  // rows of a workgroup at once
  __shared__ float s_sum[16], s_top[16];
  const int lane = threadIdx.x % TPR;
  const float inv_c = 1.f / (float)channels;
  const T* gamma = static_cast<const T*>(a.gamma);
  float g[ITEMS][V];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    if (gamma != nullptr) load_chunk<D, TAIL>(gamma, (i * TPR + lane) * V, channels, g[i]);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (gamma == nullptr) g[i][j] = 1.f;
  }
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR; row < n; row += (int64_t)gridDim.x * kRows) {
    const int64_t at = row * channels;
    Chunk<T, V> cx[ITEMS], cr[ITEMS];  // (every load before the first use)
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      cx[i] = load_raw<D, TAIL>(static_cast<const T*>(a.x) + at, (i * TPR + lane) * V, channels);
      if (a.residual != nullptr)
        cr[i] = load_raw<D, TAIL>(static_cast<const T*>(a.residual) + at, (i * TPR + lane) * V, channels);
    }
    float v[ITEMS][V];
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[i][j] = to_float<D>(cx[i].v[j]);
        if (a.residual != nullptr) v[i][j] += to_float<D>(cr[i].v[j]);
        sq = fmaf(v[i][j], v[i][j], sq);  // (zeros beyond the row)
      }
      if (a.total != nullptr) store_chunk<D, TAIL>(static_cast<T*>(a.total) + at, (i * TPR + lane) * V, channels, v[i]);
    }
    const float r = 1.f / sqrtf(row_sum<TPR>(sq, s_sum) * inv_c + a.eps);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = v[i][j] * r * g[i][j];
    if constexpr (!QUANT) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) store_chunk<D, TAIL>(static_cast<T*>(a.y) + at, (i * TPR + lane) * V, channels, v[i]);
    } else {
      float top[ITEMS];
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        top[i] = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) top[i] = fmaxf(top[i], fabsf(v[i][j]));
      }
      if (a.group == 0) {
#pragma unroll
        for (int i = 1; i < ITEMS; ++i) top[0] = fmaxf(top[0], top[i]);
        top[0] = lanes_max(top[0], TPR < 64 ? TPR : 64);
        if constexpr (TPR > 64) {
          __syncthreads();
          if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top[0];
          __syncthreads();
#pragma unroll
          for (int w = 0; w < TPR / 64; ++w) top[0] = fmaxf(top[0], s_top[w]);
        }
#pragma unroll
        for (int i = 1; i < ITEMS; ++i) top[i] = top[0];
      } else {
        const int lanes = min(a.group / V, TPR);  // (a row shorter than a group has no more)
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) top[i] = lanes_max(top[i], lanes);
      }
      const int per = a.group == 0 ? channels : a.group;
      const int64_t groups = (channels + per - 1) / per;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int c0 = (i * TPR + lane) * V;
        const float s = fmaxf(top[i] / kMostE4m3, kLeastScale), inv = 1.f / s;
        const float by = __builtin_isfinite(s) ? s : 0.f;  // (an infinite scale: no correction, and 0)
        if (c0 < channels && c0 % per == 0) a.scales[row * groups + c0 / per] = s;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          // v / s: the product with the reciprocal, whose roundings would move values next to a tie, and its
          // remainder once more (135,826 x 1,024 bf16: 178 us, without 176, divisions 190)
          const float quotient = v[i][j] * inv;
          v[i][j] = fmaf(fmaf(-quotient, by, v[i][j]), inv, quotient);
        }
        const Chunk<uint8_t, V> c = pack_e4m3<V>(v[i]);
        uint8_t* q = a.q + at;
        if (c0 + V <= channels) {
          *reinterpret_cast<Chunk<uint8_t, V>*>(q + c0) = c;
        } else if constexpr (TAIL) {
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (c0 + j < channels) q[c0 + j] = c.v[j];
        }
      }
    }
    if (a.rstd != nullptr && lane == 0) a.rstd[row] = r;
  }
}

// dx, and this workgroup's partial row sums of dy h into part[blockIdx.x][channels] (part may be NULL:
// no weight gradient).
template <DT D, int TPR, int ITEMS, bool TAIL>
__global__ __launch_bounds__(threads_for(TPR)) void rms_norm_backward_kernel(RmsBackward b, int64_t n, int channels) {
  using T = typename Elem<D>::T;
  constexpr int V = kChunk<D>;
  constexpr int kRows = threads_for(TPR) / TPR;
  __shared__ float s_sum[16];
  __shared__ float s_part[kRows > 1 ? ITEMS * TPR * V : 1];
  const int lane = threadIdx.x % TPR;
  const float inv_c = 1.f / (float)channels;
  const T* gamma = static_cast<const T*>(b.gamma);
  float g[ITEMS][V], dg[ITEMS][V];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    if (gamma != nullptr) load_chunk<D, TAIL>(gamma, (i * TPR + lane) * V, channels, g[i]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (gamma == nullptr) g[i][j] = 1.f;
      dg[i][j] = 0.f;
    }
  }
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR; row < n; row += (int64_t)gridDim.x * kRows) {
    const int64_t at = row * channels;
    Chunk<T, V> ct[ITEMS], cdy[ITEMS], cdt[ITEMS];  // (every load before the first use)
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c0 = (i * TPR + lane) * V;
      ct[i] = load_raw<D, TAIL>(static_cast<const T*>(b.total) + at, c0, channels);
      cdy[i] = load_raw<D, TAIL>(static_cast<const T*>(b.dy) + at, c0, channels);  // (zeros beyond the row)
      if (b.dtotal != nullptr) cdt[i] = load_raw<D, TAIL>(static_cast<const T*>(b.dtotal) + at, c0, channels);
    }
    const float r = b.rstd[row];
    float h[ITEMS][V], a[ITEMS][V];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        h[i][j] = to_float<D>(ct[i].v[j]) * r;
        a[i][j] = to_float<D>(cdy[i].v[j]);
        dg[i][j] = fmaf(a[i][j], h[i][j], dg[i][j]);
        a[i][j] *= g[i][j];
        sum = fmaf(a[i][j], h[i][j], sum);
      }
    const float mean = row_sum<TPR>(sum, s_sum) * inv_c;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        a[i][j] = r * fmaf(-h[i][j], mean, a[i][j]);
        if (b.dtotal != nullptr) a[i][j] += to_float<D>(cdt[i].v[j]);
      }
      store_chunk<D, TAIL>(static_cast<T*>(b.dx) + at, (i * TPR + lane) * V, channels, a[i]);
    }
  }
  if (b.part == nullptr) return;
  float* out = b.part + (int64_t)blockIdx.x * channels;
  // The rows of a wave are summed across its lanes, those of the workgroup in LDS, wave by wave (one
  // order).
  if constexpr (kRows > 1) {
    for (int m = TPR; m < 64; m *= 2) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) dg[i][j] += __shfl_xor(dg[i][j], m, 64);
    }
    for (int w = 0; w < threads_for(TPR) / 64; ++w) {
      if ((int)(threadIdx.x / 64) == w && (int)(threadIdx.x % 64) < TPR) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            float* s = s_part + (i * TPR + lane) * V + j;
            *s = w == 0 ? dg[i][j] : *s + dg[i][j];
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < channels; c += blockDim.x) out[c] = s_part[c];
  } else {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (i * TPR + lane) * V + j;
        if (c < channels) out[c] = dg[i][j];
      }
  }
}

// Workgroups of either pass: the four a compute unit that are resident.
constexpr int kGridLimit = 256 * 4;

// Sums of the workgroups' partial rows: 16 columns a workgroup, 64 threads a column each taking every
// 64th partial row, then those 64 in halves.
constexpr int kSumColumns = 16, kSumRows = 64;
template <DT D>
__global__ __launch_bounds__(kSumColumns * kSumRows) void rms_norm_weight_grad_kernel(const float* __restrict__ part, int parts,
                                                                                      int channels,
                                                                                      typename Elem<D>::T* __restrict__ dgamma) {
  __shared__ float s[kSumRows][kSumColumns];
  const int col = threadIdx.x % kSumColumns, k = threadIdx.x / kSumColumns;
  const int c = blockIdx.x * kSumColumns + col;
  float sum = 0.f;
  if (c < channels) {
    float v[kGridLimit / kSumRows];
#pragma unroll
    for (int i = 0; i < kGridLimit / kSumRows; ++i)
      v[i] = k + i * kSumRows < parts ? part[(int64_t)(k + i * kSumRows) * channels + c] : 0.f;
#pragma unroll
    for (int i = 0; i < kGridLimit / kSumRows; ++i) sum += v[i];
  }
  s[k][col] = sum;
  __syncthreads();
#pragma unroll
  for (int half = kSumRows / 2; half >= 1; half /= 2) {
    if (k < half) s[k][col] += s[k + half][col];
    __syncthreads();
  }
  if (k == 0 && c < channels) dgamma[c] = from_float<D>(s[0][col]);
}

template <DT D, int TPR, int ITEMS, bool TAIL>
void launch(const RmsForward& f, int64_t n, int channels, int blocks, hipStream_t stream) {
  if (f.q != nullptr) rms_norm_forward_kernel<D, TPR, ITEMS, TAIL, true><<<blocks, threads_for(TPR), 0, stream>>>(f, n, channels);
  else rms_norm_forward_kernel<D, TPR, ITEMS, TAIL, false><<<blocks, threads_for(TPR), 0, stream>>>(f, n, channels);
}
template <DT D, int TPR, int ITEMS, bool TAIL>
void launch(const RmsBackward& b, int64_t n, int channels, int blocks, hipStream_t stream) {
  rms_norm_backward_kernel<D, TPR, ITEMS, TAIL><<<blocks, threads_for(TPR), 0, stream>>>(b, n, channels);
}

// Lanes of a row.  A lane holds up to 4 chunks in the forward pass and up to 3 in the backward pass, whose
// gradients and weights stay in registers too; up to 16,384 channels, beyond which float32 rows would not
// fit.
int lanes_for(const RmsForward&, int chunks) {
  return chunks <= 64 ? short_lanes(chunks) : chunks <= 256 ? 64 : chunks <= 1024 ? 256 : 1024;
}
int lanes_for(const RmsBackward&, int chunks) {
  return chunks <= 64 ? short_lanes(chunks) : chunks <= 192 ? 64 : chunks <= 512 ? 256 : 1024;
}

template <DT D, bool TAIL>
void launch_rows(const RmsForward& a, int64_t n, int channels, int chunks, int blocks, hipStream_t stream) {
  if (chunks <= 8) launch<D, 8, 1, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 16) launch<D, 16, 1, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 32) launch<D, 32, 1, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 64) launch<D, 64, 1, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 128) launch<D, 64, 2, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 256) launch<D, 64, 4, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 512) launch<D, 256, 2, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 1024) launch<D, 256, 4, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 2048) launch<D, 1024, 2, TAIL>(a, n, channels, blocks, stream);
  else if constexpr (D == DT::F32) launch<D, 1024, 4, TAIL>(a, n, channels, blocks, stream);
}
template <DT D, bool TAIL>
void launch_rows(const RmsBackward& a, int64_t n, int channels, int chunks, int blocks, hipStream_t stream) {
  if (chunks <= 8) launch<D, 8, 1, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 16) launch<D, 16, 1, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 32) launch<D, 32, 1, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 64) launch<D, 64, 1, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 128) launch<D, 64, 2, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 192) launch<D, 64, 3, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 256) launch<D, 256, 1, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 512) launch<D, 256, 2, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 1024) launch<D, 1024, 1, TAIL>(a, n, channels, blocks, stream);
  else if (chunks <= 2048) launch<D, 1024, 2, TAIL>(a, n, channels, blocks, stream);
  else if constexpr (D == DT::F32) launch<D, 1024, 4, TAIL>(a, n, channels, blocks, stream);
}

// (whole chunks: no element-wise ends in the kernel, whose branches part the loads of a row)
template <DT D, typename A> void launch_ends(const A& a, int64_t n, int channels, int blocks, hipStream_t stream) {
  const int chunks = (channels + kChunk<D> - 1) / kChunk<D>;
  if (channels % kChunk<D> == 0) launch_rows<D, false>(a, n, channels, chunks, blocks, stream);
  else launch_rows<D, true>(a, n, channels, chunks, blocks, stream);
}

template <typename A> hipError_t launch_dtype(const A& a, int64_t n, int channels, int dtype, int blocks, hipStream_t stream) {
  if (dtype == SUBM_F32) launch_ends<DT::F32>(a, n, channels, blocks, stream);
  else if (dtype == SUBM_F16) launch_ends<DT::F16>(a, n, channels, blocks, stream);
  else launch_ends<DT::BF16>(a, n, channels, blocks, stream);
  return hipGetLastError();
}

template <typename A> int blocks_for(const A& a, int64_t n, int channels, int dtype) {
  const int chunk = dtype == SUBM_F32 ? 4 : 8, tpr = lanes_for(a, (channels + chunk - 1) / chunk);
  const int rows = threads_for(tpr) / tpr;
  return (int)std::min<int64_t>((n + rows - 1) / rows, kGridLimit);
}

Status check_rms_norm(int64_t n, int channels, int dtype) {
  if (dtype != SUBM_F32 && dtype != SUBM_F16 && dtype != SUBM_BF16)
    return make_status(SUBM_ERR_UNSUPPORTED, "dtype must be SUBM_F32, SUBM_F16 or SUBM_BF16");
  if (n < 0) return make_status(SUBM_ERR_INVALID_ARG, "n is negative");
  if (n > INT32_MAX) return make_status(SUBM_ERR_INVALID_ARG, "n exceeds 2^31 - 1");
  if (channels < 1) return make_status(SUBM_ERR_INVALID_ARG, "channels must be at least 1");
  if (channels > 16384) return make_status(SUBM_ERR_UNSUPPORTED, "channels exceeds 16384");
  return Status{};
}

bool misaligned(const void* p, int size) { return reinterpret_cast<uintptr_t>(p) % size != 0; }

int forward(const RmsForward& f, int64_t n, int channels, int dtype, hipStream_t stream, const char* what) {
  Status st = check_rms_norm(n, channels, dtype);
  if (!st.ok()) return fail(st);
  if (!(f.eps > 0.f) || !std::isfinite(f.eps)) return fail(SUBM_ERR_INVALID_ARG, "eps must be positive and finite");
  if (n == 0) return SUBM_OK;
  if (f.x == nullptr) return fail(SUBM_ERR_INVALID_ARG, "x is NULL");
  if (f.residual != nullptr && f.total == nullptr) return fail(SUBM_ERR_INVALID_ARG, "total is NULL with a residual");
  const int elem = dtype == SUBM_F32 ? 4 : 2;
  if (misaligned(f.x, elem) || misaligned(f.residual, elem) || misaligned(f.gamma, elem) || misaligned(f.total, elem) ||
      misaligned(f.y, elem) || misaligned(f.scales, 4) || misaligned(f.rstd, 4))
    return fail(SUBM_ERR_INVALID_ARG, "a pointer is not aligned to its element");
  if (f.total != nullptr && f.total == f.y) return fail(SUBM_ERR_INVALID_ARG, "total and y must not alias");
  if (f.q != nullptr && (f.q == f.x || f.q == f.residual || f.q == f.total))
    return fail(SUBM_ERR_INVALID_ARG, "q must not alias x, residual or total");
  const hipError_t e = launch_dtype(f, n, channels, dtype, blocks_for(f, n, channels, dtype), stream);
  if (e != hipSuccess) return fail(hip_status(e, what));
  return SUBM_OK;
}

}  // namespace
}  // namespace submconv

using namespace submconv;

extern "C" int sparse_rms_norm_forward(const void* x, const void* residual, int64_t n, int channels, int dtype,
                                       const void* gamma, float eps, void* y, void* total, float* rstd, hipStream_t stream) {
  return no_throw([&]() -> int {
    clear_error();
    if (n > 0 && y == nullptr) return fail(SUBM_ERR_INVALID_ARG, "y is NULL");
    const RmsForward f{x, residual, gamma, total, y, nullptr, nullptr, rstd, eps, 0};
    return forward(f, n, channels, dtype, stream, "sparse_rms_norm_forward launch");
  });
}

extern "C" int sparse_rms_norm_quantize_forward(const void* x, const void* residual, int64_t n, int channels, int dtype,
                                                const void* gamma, float eps, int group, void* q, float* scales, void* total,
                                                float* rstd, hipStream_t stream) {
  return no_throw([&]() -> int {
    clear_error();
    if (group != 0 && group != 32 && group != 64 && group != 128)
      return fail(SUBM_ERR_INVALID_ARG, "group must be 0, 32, 64 or 128");
    if (n > 0 && (q == nullptr || scales == nullptr)) return fail(SUBM_ERR_INVALID_ARG, "q or scales is NULL");
    const RmsForward f{x, residual, gamma, total, nullptr, static_cast<uint8_t*>(q), scales, rstd, eps, group};
    return forward(f, n, channels, dtype, stream, "sparse_rms_norm_quantize_forward launch");
  });
}

extern "C" int sparse_rms_norm_backward(const void* dy, const void* total, const void* dtotal, int64_t n, int channels,
                                        int dtype, const void* gamma, const float* rstd, void* dx, void* dgamma,
                                        hipStream_t stream) {
  return no_throw([&]() -> int {
    clear_error();
    Status st = check_rms_norm(n, channels, dtype);
    if (!st.ok()) return fail(st);
    const int elem = dtype == SUBM_F32 ? 4 : 2;
    if (n > 0 && (dy == nullptr || total == nullptr || rstd == nullptr || dx == nullptr))
      return fail(SUBM_ERR_INVALID_ARG, "dy, total, rstd or dx is NULL");
    if (misaligned(dy, elem) || misaligned(total, elem) || misaligned(dtotal, elem) || misaligned(gamma, elem) ||
        misaligned(dx, elem) || misaligned(dgamma, elem) || misaligned(rstd, 4))
      return fail(SUBM_ERR_INVALID_ARG, "a pointer is not aligned to its element");
    if (dx != nullptr && dx == total) return fail(SUBM_ERR_INVALID_ARG, "dx must not alias total");
    if (n == 0 && dgamma == nullptr) return SUBM_OK;
    RmsBackward b{dy, total, dtotal, gamma, rstd, dx, nullptr};
    const int blocks = blocks_for(b, n, channels, dtype);
    ScratchLease lease;
    if (dgamma != nullptr) {
      int dev = 0;
      hipError_t e = hipGetDevice(&dev);
      if (e != hipSuccess) return fail(hip_status(e, "hipGetDevice"));
      void* scratch = nullptr;
      st = lease.take(dev, stream, std::max<size_t>((size_t)blocks * channels * sizeof(float), 16), &scratch);
      if (!st.ok()) return fail(st);
      b.part = static_cast<float*>(scratch);
    }
    hipError_t e = hipSuccess;
    if (n > 0) e = launch_dtype(b, n, channels, dtype, blocks, stream);
    if (e == hipSuccess && dgamma != nullptr) {
      const int grid = (channels + kSumColumns - 1) / kSumColumns;
      if (dtype == SUBM_F32)
        rms_norm_weight_grad_kernel<DT::F32><<<grid, kSumColumns * kSumRows, 0, stream>>>(b.part, blocks, channels, static_cast<float*>(dgamma));
      else if (dtype == SUBM_F16)
        rms_norm_weight_grad_kernel<DT::F16><<<grid, kSumColumns * kSumRows, 0, stream>>>(b.part, blocks, channels, static_cast<uint16_t*>(dgamma));
      else
        rms_norm_weight_grad_kernel<DT::BF16><<<grid, kSumColumns * kSumRows, 0, stream>>>(b.part, blocks, channels, static_cast<uint16_t*>(dgamma));
      e = hipGetLastError();
    }
    if (e != hipSuccess) return fail(hip_status(e, "sparse_rms_norm_backward launch"));
    return SUBM_OK;
  });
}
