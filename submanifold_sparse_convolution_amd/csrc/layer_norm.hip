// Layer norm over the channels of each row, forward and backward (include/sparse_transformer.h).
//
//   mu = sum x / C,  r = 1 / sqrt(sum (x - mu)^2 / C + eps),  h = (x - mu) r,  y = h g + b
//   a = dy g,  dx = r (a - mean(a) - h mean(a h)),  dg = sum_rows dy h,  db = sum_rows dy
//
// Both are bound by HBM: the forward pass moves 2 and the backward pass 3 values an element and
// neither reuses any.  A row therefore stays in registers between its one load and its one store
// (the variance is taken of the centred values there), spread over TPR lanes in 16-byte chunks.
// Rows of any length and alignment take the same path; the last chunk of a row goes element by
// element when C is not a multiple of the chunk.
//
// Measured: 135,826 x 1,024 bf16: forward 102 us (5.5 TB/s), backward 160 us (5.2 TB/s); 4,099 x 675
// float32, backward: 15 us, two launches; 450 x 768 f16, forward: 3.4 us on the device, 6.2 a call.
#include <algorithm>
#include <cmath>

#include "chunk.h"
#include "device_common.h"
#include "internal.h"
#include "row_lanes.h"
#include "sparse_transformer.h"

namespace submconv {
namespace {

// Workgroups of the backward pass, each a partial weight gradient: the four a compute unit that are
// resident (1,024 16-bit channels, 135,826 rows: 160 us; two 238, three 180, eight 170), two with
// three chunks a lane (60,000 x 700 float32: 95 us, four 103).
constexpr int kPartsLimit = 256 * 4;
int parts_limit(int chunks) { return chunks > 128 && chunks <= 192 ? 256 * 2 : kPartsLimit; }

// (x may be y: neither is declared free of aliases.)
template <DT D, int TPR, int ITEMS, bool TAIL>
__global__ __launch_bounds__(threads_for(TPR)) void layer_norm_forward_kernel(
    const typename Elem<D>::T* x, int64_t n, int channels, const typename Elem<D>::T* __restrict__ gamma,
    const typename Elem<D>::T* __restrict__ beta, float eps, typename Elem<D>::T* y, float* __restrict__ mean,
    float* __restrict__ rstd) {
  constexpr int V = kChunk<D>;
  constexpr int kRows = threads_for(TPR) / TPR;  // rows of a workgroup at once
  __shared__ float s_a[16], s_b[16];
  const int lane = threadIdx.x % TPR;
  const float inv_c = 1.f / (float)channels;
  float g[ITEMS][V], b[ITEMS][V];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c0 = (i * TPR + lane) * V;
    if (gamma != nullptr) load_chunk<D, TAIL>(gamma, c0, channels, g[i]);
    if (beta != nullptr) load_chunk<D, TAIL>(beta, c0, channels, b[i]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (gamma == nullptr) g[i][j] = 1.f;
      if (beta == nullptr) b[i][j] = 0.f;
    }
  }
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR; row < n; row += (int64_t)gridDim.x * kRows) {
    const typename Elem<D>::T* px = x + row * channels;
    float v[ITEMS][V];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      load_chunk<D, TAIL>(px, (i * TPR + lane) * V, channels, v[i]);
#pragma unroll
      for (int j = 0; j < V; ++j) sum += v[i][j];
    }
    const float mu = row_sum<TPR>(sum, s_a) * inv_c;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[i][j] -= mu;
        sq += (i * TPR + lane) * V + j < channels ? v[i][j] * v[i][j] : 0.f;
      }
    const float r = 1.f / sqrtf(row_sum<TPR>(sq, s_b) * inv_c + eps);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = fmaf(v[i][j] * r, g[i][j], b[i][j]);
      store_chunk<D, TAIL>(y + row * channels, (i * TPR + lane) * V, channels, v[i]);
    }
    if (mean != nullptr && lane == 0) {
      mean[row] = mu;
      rstd[row] = r;
    }
  }
}

// dx, and this workgroup's partial row sums of dy h and dy into part[blockIdx.x][2][channels]
// (part may be NULL: no weight gradients).
template <DT D, int TPR, int ITEMS, bool TAIL>
__global__ __launch_bounds__(threads_for(TPR)) void layer_norm_backward_kernel(
    const typename Elem<D>::T* dy, const typename Elem<D>::T* __restrict__ x, int64_t n, int channels,
    const typename Elem<D>::T* __restrict__ gamma, const float* __restrict__ mean, const float* __restrict__ rstd,
    typename Elem<D>::T* dx, float* __restrict__ part) {
  constexpr int V = kChunk<D>;
  constexpr int kRows = threads_for(TPR) / TPR;
  __shared__ float s_a[16], s_b[16];
  __shared__ float s_part[kRows > 1 ? 2 * ITEMS * TPR * V : 1];
  const int lane = threadIdx.x % TPR;
  const float inv_c = 1.f / (float)channels;
  float g[ITEMS][V], dg[ITEMS][V], db[ITEMS][V];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    if (gamma != nullptr) load_chunk<D, TAIL>(gamma, (i * TPR + lane) * V, channels, g[i]);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (gamma == nullptr) g[i][j] = 1.f;
      dg[i][j] = 0.f;
      db[i][j] = 0.f;
    }
  }
  // (Waves of other rows hide a row's memory latency: prefetching the next row into registers takes
  // a resident workgroup away; when there were three of them it measured 186 us for 155.)
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR; row < n; row += (int64_t)gridDim.x * kRows) {
    Chunk<typename Elem<D>::T, V> cx[ITEMS], cdy[ITEMS];  // (every load before the first use)
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      cx[i] = load_raw<D, TAIL>(x + row * channels, (i * TPR + lane) * V, channels);
      cdy[i] = load_raw<D, TAIL>(dy + row * channels, (i * TPR + lane) * V, channels);  // (zeros beyond the row)
    }
    const float mu = mean[row], r = rstd[row];
    float h[ITEMS][V], a[ITEMS][V];
    float sa = 0.f, sah = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        h[i][j] = (to_float<D>(cx[i].v[j]) - mu) * r;
        a[i][j] = to_float<D>(cdy[i].v[j]);
      }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        dg[i][j] = fmaf(a[i][j], h[i][j], dg[i][j]);
        db[i][j] += a[i][j];
        a[i][j] *= g[i][j];
        sa += a[i][j];
        sah = fmaf(a[i][j], h[i][j], sah);
      }
    const float ma = row_sum<TPR>(sa, s_a) * inv_c;
    const float mah = row_sum<TPR>(sah, s_b) * inv_c;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
      for (int j = 0; j < V; ++j) a[i][j] = r * (a[i][j] - ma - h[i][j] * mah);
      store_chunk<D, TAIL>(dx + row * channels, (i * TPR + lane) * V, channels, a[i]);
    }
  }
  if (part == nullptr) return;
  // The rows of a wave are summed across its lanes, those of the workgroup in LDS, wave by wave (one
  // order).
  if constexpr (kRows > 1) {
    for (int m = TPR; m < 64; m *= 2) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          dg[i][j] += __shfl_xor(dg[i][j], m, 64);
          db[i][j] += __shfl_xor(db[i][j], m, 64);
        }
    }
    for (int w = 0; w < threads_for(TPR) / 64; ++w) {
      if ((int)(threadIdx.x / 64) == w && (int)(threadIdx.x % 64) < TPR) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const int c = (i * TPR + lane) * V + j;
            float* sg = s_part + c;
            float* sb = s_part + ITEMS * TPR * V + c;
            *sg = w == 0 ? dg[i][j] : *sg + dg[i][j];
            *sb = w == 0 ? db[i][j] : *sb + db[i][j];
          }
      }
      __syncthreads();
    }
    float* out = part + (int64_t)blockIdx.x * 2 * channels;
    for (int c = threadIdx.x; c < channels; c += blockDim.x) {
      out[c] = s_part[c];
      out[channels + c] = s_part[ITEMS * TPR * V + c];
    }
  } else {
    float* out = part + (int64_t)blockIdx.x * 2 * channels;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (i * TPR + lane) * V + j;
        if (c < channels) {
          out[c] = dg[i][j];
          out[channels + c] = db[i][j];
        }
      }
  }
}

// Sums of the workgroups' partial rows: 16 columns of dgamma | dbeta (2 channels in all) a
// workgroup, 64 threads a column each taking every 64th partial row, then those 64 in halves.
constexpr int kSumColumns = 16, kSumRows = 64;
template <DT D>
__global__ __launch_bounds__(kSumColumns * kSumRows) void layer_norm_weight_grad_kernel(
    const float* __restrict__ part, int parts, int channels, typename Elem<D>::T* __restrict__ dgamma,
    typename Elem<D>::T* __restrict__ dbeta) {
  __shared__ float s[kSumRows][kSumColumns];
  const int col = threadIdx.x % kSumColumns, k = threadIdx.x / kSumColumns;
  const int c = blockIdx.x * kSumColumns + col;
  float sum = 0.f;
  if (c < 2 * channels) {
    float v[kPartsLimit / kSumRows];
#pragma unroll
    for (int i = 0; i < kPartsLimit / kSumRows; ++i)
      v[i] = k + i * kSumRows < parts ? part[(int64_t)(k + i * kSumRows) * 2 * channels + c] : 0.f;
#pragma unroll
    for (int i = 0; i < kPartsLimit / kSumRows; ++i) sum += v[i];
  }
  s[k][col] = sum;
  __syncthreads();
#pragma unroll
  for (int half = kSumRows / 2; half >= 1; half /= 2) {
    if (k < half) s[k][col] += s[k + half][col];
    __syncthreads();
  }
  if (k != 0 || c >= 2 * channels) return;
  if (c < channels) dgamma[c] = from_float<D>(s[0][col]);
  else dbeta[c - channels] = from_float<D>(s[0][col]);
}

constexpr int kMaxChannels = 16384;
// workgroups of the forward pass (135,826 x 1024 bf16: 101 us; eight a compute unit 119)
constexpr int kGridLimit = 256 * 4;

struct Forward {
  const void *x, *gamma, *beta;
  void* y;
  float *mean, *rstd;
  float eps;
};
struct Backward {
  const void *dy, *x, *gamma;
  const float *mean, *rstd;
  void* dx;
  float* part;
};

int rows_per_block(int tpr) { return threads_for(tpr) / tpr; }

template <DT D, int TPR, int ITEMS, bool TAIL>
void launch(const Forward& f, int64_t n, int channels, int blocks, hipStream_t stream) {
  using T = typename Elem<D>::T;
  layer_norm_forward_kernel<D, TPR, ITEMS, TAIL><<<blocks, threads_for(TPR), 0, stream>>>(
      static_cast<const T*>(f.x), n, channels, static_cast<const T*>(f.gamma), static_cast<const T*>(f.beta), f.eps,
      static_cast<T*>(f.y), f.mean, f.rstd);
}
template <DT D, int TPR, int ITEMS, bool TAIL>
void launch(const Backward& b, int64_t n, int channels, int blocks, hipStream_t stream) {
  using T = typename Elem<D>::T;
  layer_norm_backward_kernel<D, TPR, ITEMS, TAIL><<<blocks, threads_for(TPR), 0, stream>>>(
      static_cast<const T*>(b.dy), static_cast<const T*>(b.x), n, channels, static_cast<const T*>(b.gamma), b.mean,
      b.rstd, static_cast<T*>(b.dx), b.part);
}

// A lane holds up to 4 chunks in the forward pass and 2 in the backward pass,
// whose gradients and weights stay in registers too, or 3 where a wave then spares a row its
// barriers (60,000 x 700 float32: 95 us, four waves a row 107); up to 16,384 channels, beyond which
// float32 rows would not fit.
int lanes_for(const Forward&, int chunks) {
  return chunks <= 64 ? short_lanes(chunks) : chunks <= 256 ? 64 : chunks <= 1024 ? 256 : 1024;
}
int lanes_for(const Backward&, int chunks) {
  return chunks <= 64 ? short_lanes(chunks) : chunks <= 192 ? 64 : chunks <= 512 ? 256 : 1024;
}

int limit_for(const Forward&, int) { return kGridLimit; }
int limit_for(const Backward&, int chunks) { return parts_limit(chunks); }

template <DT D, bool TAIL>
hipError_t launch_rows(const Forward& a, int64_t n, int channels, int chunks, int blocks, hipStream_t stream) {
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
  return hipGetLastError();
}
template <DT D, bool TAIL>
hipError_t launch_rows(const Backward& a, int64_t n, int channels, int chunks, int blocks, hipStream_t stream) {
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
  return hipGetLastError();
}

// (whole chunks: no element-wise ends in the kernel, whose branches part the loads of a row)
template <DT D, typename A>
hipError_t launch_ends(const A& a, int64_t n, int channels, int blocks, hipStream_t stream) {
  const int chunks = (channels + kChunk<D> - 1) / kChunk<D>;
  return channels % kChunk<D> == 0 ? launch_rows<D, false>(a, n, channels, chunks, blocks, stream)
                                   : launch_rows<D, true>(a, n, channels, chunks, blocks, stream);
}

template <typename A>
hipError_t launch_dtype(const A& a, int64_t n, int channels, int dtype, int blocks, hipStream_t stream) {
  if (dtype == SUBM_F32) return launch_ends<DT::F32>(a, n, channels, blocks, stream);
  if (dtype == SUBM_F16) return launch_ends<DT::F16>(a, n, channels, blocks, stream);
  return launch_ends<DT::BF16>(a, n, channels, blocks, stream);
}

template <typename A> int blocks_for(const A& a, int64_t n, int channels, int dtype) {
  const int chunk = dtype == SUBM_F32 ? 4 : 8, chunks = (channels + chunk - 1) / chunk;
  const int rows = rows_per_block(lanes_for(a, chunks));
  return (int)std::min<int64_t>((n + rows - 1) / rows, limit_for(a, chunks));
}

Status check_layer_norm(int64_t n, int channels, int dtype) {
  if (dtype != SUBM_F32 && dtype != SUBM_F16 && dtype != SUBM_BF16)
    return make_status(SUBM_ERR_UNSUPPORTED, "dtype must be SUBM_F32, SUBM_F16 or SUBM_BF16");
  if (n < 0) return make_status(SUBM_ERR_INVALID_ARG, "n is negative");
  if (n > INT32_MAX) return make_status(SUBM_ERR_INVALID_ARG, "n exceeds 2^31 - 1");
  if (channels < 1) return make_status(SUBM_ERR_INVALID_ARG, "channels must be at least 1");
  if (channels > kMaxChannels) return make_status(SUBM_ERR_UNSUPPORTED, "channels exceeds 16384");
  return Status{};
}

bool misaligned(const void* p, int size) { return reinterpret_cast<uintptr_t>(p) % size != 0; }

}  // namespace
}  // namespace submconv

using namespace submconv;

extern "C" int sparse_layer_norm_forward(const void* x, int64_t n, int channels, int dtype, const void* gamma,
                                         const void* beta, float eps, void* y, float* mean, float* rstd,
                                         hipStream_t stream) {
  return no_throw([&]() -> int {
    clear_error();
    Status st = check_layer_norm(n, channels, dtype);
    if (!st.ok()) return fail(st);
    if (!(eps > 0.f) || !std::isfinite(eps)) return fail(SUBM_ERR_INVALID_ARG, "eps must be positive and finite");
    if ((mean == nullptr) != (rstd == nullptr)) return fail(SUBM_ERR_INVALID_ARG, "mean and rstd go together");
    if (n == 0) return SUBM_OK;
    if (x == nullptr || y == nullptr) return fail(SUBM_ERR_INVALID_ARG, "x or y is NULL");
    const int elem = dtype == SUBM_F32 ? 4 : 2;
    if (misaligned(x, elem) || misaligned(y, elem) || misaligned(gamma, elem) || misaligned(beta, elem) ||
        misaligned(mean, 4) || misaligned(rstd, 4))
      return fail(SUBM_ERR_INVALID_ARG, "a pointer is not aligned to its element");
    const Forward f{x, gamma, beta, y, mean, rstd, eps};
    const hipError_t e = launch_dtype(f, n, channels, dtype, blocks_for(f, n, channels, dtype), stream);
    if (e != hipSuccess) return fail(hip_status(e, "sparse_layer_norm_forward launch"));
    return SUBM_OK;
  });
}

extern "C" int sparse_layer_norm_backward(const void* dy, const void* x, int64_t n, int channels, int dtype,
                                          const void* gamma, const float* mean, const float* rstd, void* dx,
                                          void* dgamma, void* dbeta, hipStream_t stream) {
  return no_throw([&]() -> int {
    clear_error();
    Status st = check_layer_norm(n, channels, dtype);
    if (!st.ok()) return fail(st);
    if ((dgamma == nullptr) != (dbeta == nullptr)) return fail(SUBM_ERR_INVALID_ARG, "dgamma and dbeta go together");
    const int elem = dtype == SUBM_F32 ? 4 : 2;
    if (n > 0 && (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr || dx == nullptr))
      return fail(SUBM_ERR_INVALID_ARG, "dy, x, mean, rstd or dx is NULL");
    if (misaligned(dy, elem) || misaligned(x, elem) || misaligned(gamma, elem) || misaligned(dx, elem) ||
        misaligned(dgamma, elem) || misaligned(dbeta, elem) || misaligned(mean, 4) || misaligned(rstd, 4))
      return fail(SUBM_ERR_INVALID_ARG, "a pointer is not aligned to its element");
    if (n == 0 && dgamma == nullptr) return SUBM_OK;
    Backward b{dy, x, gamma, mean, rstd, dx, nullptr};
    const int blocks = blocks_for(b, n, channels, dtype);
    ScratchLease lease;
    if (dgamma != nullptr) {
      int dev = 0;
      hipError_t e = hipGetDevice(&dev);
      if (e != hipSuccess) return fail(hip_status(e, "hipGetDevice"));
      void* scratch = nullptr;
      st = lease.take(dev, stream, std::max<size_t>((size_t)blocks * 2 * channels * sizeof(float), 16), &scratch);
      if (!st.ok()) return fail(st);
      b.part = static_cast<float*>(scratch);
    }
    hipError_t e = hipSuccess;
    if (n > 0) {
      e = launch_dtype(b, n, channels, dtype, blocks, stream);
    }
    if (e == hipSuccess && dgamma != nullptr) {
      const int grid = (2 * channels + kSumColumns - 1) / kSumColumns;
      if (dtype == SUBM_F32)
        layer_norm_weight_grad_kernel<DT::F32><<<grid, kSumColumns * kSumRows, 0, stream>>>(b.part, blocks, channels, static_cast<float*>(dgamma),
                                                                         static_cast<float*>(dbeta));
      else if (dtype == SUBM_F16)
        layer_norm_weight_grad_kernel<DT::F16><<<grid, kSumColumns * kSumRows, 0, stream>>>(
            b.part, blocks, channels, static_cast<uint16_t*>(dgamma), static_cast<uint16_t*>(dbeta));
      else
        layer_norm_weight_grad_kernel<DT::BF16><<<grid, kSumColumns * kSumRows, 0, stream>>>(
            b.part, blocks, channels, static_cast<uint16_t*>(dgamma), static_cast<uint16_t*>(dbeta));
      e = hipGetLastError();
    }
    if (e != hipSuccess) return fail(hip_status(e, "sparse_layer_norm_backward launch"));
    return SUBM_OK;
  });
}
