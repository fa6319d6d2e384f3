// Attention over the items of a sparse tensor, forward pass (include/sparse_transformer.h).
//
//   S = scale q k^T,  m = max_j S,  l = sum_j exp(S - m),  out = (sum_j exp(S - m) v_j) / l,
//   lse = m + log l
// in one pass over the keys with the running m and l of a softmax: when m grows, l and the
// accumulator shrink by exp(m_old - m_new).  Exponentials are powers of two of scores that carry
// scale * log2(e).
//
// Bound by the matrix cores (4 rows keys d operations against rows and keys read once) except for
// a few rows against long caches, which read k and v once at HBM speed.
//
// Measured: items of 13,001 and 11,575 tokens, 16 heads of 128, bf16: 2.23 ms, 1.11 PFLOP/s (matrix
// cores busy 58 % of the cycles, at a clock that the power limit holds near 1.8 GHz; in a trace of 30
// calls 2.20 to 2.29 ms); four items of 450 to 4,001 queries and up to 1,374 keys, 12 heads of 64, f16:
// 48 us, 0.53 PFLOP/s (636 workgroups of unequal length at once, each product of 64 channels beside as
// many exponentials); 8 single tokens, up to 32,768 keys each, 16 / 4 heads of 128, bf16: 87 us, 4.9
// TB/s.
#include <algorithm>
#include <cmath>

#include "attention_common.h"

namespace submconv {
namespace {

struct FwdArgs {
  subm_heads_t q, k, v, out;
  float* lse;
  const int64_t *q_offsets, *k_offsets;
  int64_t nq, nk;
  int items, heads, kv_heads, head_dim;
  float scale;
  // Tiles in parts: what a part leaves, [place][rows of a tile][DP] unnormalised sums and their
  // (base, sum).
  Cut cut;
  float* part;
  float2* state;
};

// (fmaxf would first quiet every operand)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// Keeps the values computed here: the compiler would sink them past the next branch, away from the
// matrix products that they overlap with.
template <DT D> __device__ __forceinline__ void pin(Frag<D>& f) {
#pragma unroll
  for (int i = 0; i < Elem<D>::kSize / 2; ++i)
    asm volatile("" : "+v"(f.v[i].x), "+v"(f.v[i].y), "+v"(f.v[i].z), "+v"(f.v[i].w));
}

constexpr float kNone = -1.7e38f;  // a running maximum before any score (finite: differences stay numbers)

// The running softmax of one own row (held by the lanes l and l + 32, half its scores each):
// scores are kept as c * s - base in powers of two; base is a maximum, less kLift, that may lag behind
// the true one by kSlack, so that most tiles do not rescale the accumulator.  p stays below
// 2^(kLift + kSlack), which the storage type holds.  float16 rounds what is below 2^-25 to zero, and
// thousands of such keys beside one large score are not nothing (60,000 at 2^-25.5 of it are a
// thousandth): there p starts from 2^11, and what vanishes is below 2^-36 of the largest.
template <DT D> constexpr float kLift = D == DT::F16 ? 11.f : 0.f;
template <DT D> constexpr float kSlack = D == DT::F16 ? 4.f : 8.f;
struct RowState {
  float base = kNone;
  float sum = 0.f;  // of this lane's half
};

// Scores (raw) -> probabilities in place; returns the factor that earlier sums shrink by, and
// whether any row of the wave does shrink.
template <DT D, int KB>
__device__ __forceinline__ bool softmax_tile(f32x16_t (&s)[KB], float c, RowState& st, float* shrink) {
  float top = s[0][0];
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 16; i += 2) top = max3(top, s[kb][i], s[kb][i + 1]);
  top = half_max(top);
  top = kLift<D> == 0.f ? top * c : fmaf(top, c, -kLift<D>);
  const bool moves = __builtin_amdgcn_ballot_w64(top > st.base + kSlack<D>) != 0;
  // (a scalar gate instead of a branch, which would part the matrix products from the exponentials)
  const float base = fmaxf(st.base, top + (moves ? 0.f : -INFINITY));
  *shrink = exp2_fast(st.base - base);
  st.base = base;
  float sum = 0.f;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[kb][i] = exp2_fast(fmaf(s[kb][i], c, -base));
      sum += s[kb][i];
    }
  st.sum = fmaf(st.sum, *shrink, sum);
  return moves;
}

// Streams the keys through LDS in tiles of KEYS, two of k and two of v; one step of the loop holds
// three independent pieces of work, so that the matrix cores run while the exponentials do:
//   scores of tile t + 1 (k),  softmax of tile t,  product of tile t - 1 (v).
// (Four tiles of each in flight: the same time.)
//
// KG = 2: two groups of W waves hold the same rows and take every other tile of keys, joined through
// LDS at the end: where a compute unit gets one workgroup, a lone wave a SIMD would wait for each
// instruction's result in turn.
template <DT D, int DC, int W, int KG, int KEYS, int OCC, int CUT>
__global__ __launch_bounds__(KG * W * 64, OCC) void attention_forward_kernel(FwdArgs a) {
  constexpr int DP = tile_width(DC), KB = KEYS / 32;
  constexpr int kTile = KEYS * kRowBytes<D, DP>;
  constexpr int kRows = 32 * W;
  using Loader = TileLoader<D, DP, KEYS, W>;
  __shared__ __attribute__((aligned(1024))) unsigned char s_kv[KG * 4 * kTile];
  __shared__ float2 s_join[KG == 1 ? 1 : W * 64];
  const int lane = threadIdx.x & 63, every = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = KG == 1 ? 0 : every / W, wave = KG == 1 ? every : every % W;
  const int group = a.heads / a.kv_heads;
  const Share share = share_of<CUT>(a.cut, blockIdx.x);
  const int head = share.head;
  int tile;
  const int item = find_item(a.q_offsets, a.nq, a.items, group, kRows, share.slot, &tile);
  int64_t q0, k0;
  int nq, nk;
  item_rows(a.q_offsets, a.nq, item, &q0, &nq);
  item_rows(a.k_offsets, a.nk, item, &k0, &nk);
  const int rows = nq * group;
  if ((int64_t)tile * kRows >= rows) return;
  const RowMap qmap{q0, head * group, group};
  const Heads<D> q = heads_of<D>(a.q), k = heads_of<D>(a.k), v = heads_of<D>(a.v), out = heads_of<D>(a.out);
  const typename Elem<D>::T* kp = k.data + k0 * k.row + (int64_t)head * k.head;
  const typename Elem<D>::T* vp = v.data + k0 * v.row + (int64_t)head * v.head;

  const int row = tile * kRows + wave * 32 + (lane & 31);
  const bool there = row < rows;
  Frag<D> qf[DC / 16];
  const typename Elem<D>::T* qrow = qmap.at<D>(q, there ? row : 0);
  // a negative scale goes into q, so that the largest score is the largest product
  const uint32_t flip = a.scale < 0.f ? (D == DT::F32 ? 0x80000000u : 0x80008000u) : 0u;
#pragma unroll
  for (int kk = 0; kk < DC / 16; ++kk) {
    qf[kk] = own_frag<D>(qrow, there, kk, a.head_dim, lane);
#pragma unroll
    for (int i = 0; i < Elem<D>::kSize / 2; ++i) {
      qf[kk].v[i].x ^= flip;
      qf[kk].v[i].y ^= flip;
      qf[kk].v[i].z ^= flip;
      qf[kk].v[i].w ^= flip;
    }
  }
  // (a scale of 0 becomes tiny: a key past the end must still score -infinity)
  const float c = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);

  Loader lk, lv;
  lk.wave = lv.wave = wave;
  lk.lane = lv.lane = lane;
  lk.place(k, a.head_dim, 1, 0, 0);
  lv.place(v, a.head_dim, 1, 0, 0);
  const uint32_t lds = lds_offset(s_kv) + part * 4 * kTile;
  const TileReader<D, DP> rd(lane, lds, lds + 2 * kTile);
  // this workgroup's keys: all, or its share of whole tiles (a share may be empty)
  int tiles = (nk + KEYS - 1) / KEYS, left = nk;
  if constexpr (CUT != kNoCut) {
    const int first = part_steps(a.cut, share.part, &tiles);
    left = min(nk - first * KEYS, tiles * KEYS);
    kp += (int64_t)first * KEYS * k.row;
    vp += (int64_t)first * KEYS * v.row;
  }
  // (t counts this part's tiles; t and slot apart: inside the loop the slot is a constant)
  const auto load_k = [&](int t, int slot) {
    const int key = (t * KG + part) * KEYS;
    lk.load(kp + (int64_t)key * k.row, left - key, lds + slot * kTile);
  };
  const auto load_v = [&](int t, int slot) {
    const int key = (t * KG + part) * KEYS;
    lv.load(vp + (int64_t)key * v.row, t < 0 ? 0 : left - key, lds + (2 + slot) * kTile);
  };
  const auto scores = [&](int slot, f32x16_t (&s)[KB]) {
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      s[kb] = zero16();
#pragma unroll
      for (int kk = 0; kk < DC / 16; ++kk) s[kb] = mma<D>(rd.row_frag(slot * kTile, kb * 32, kk), qf[kk], s[kb]);
    }
  };
  f32x16_t acc[DC / 32];
#pragma unroll
  for (int db = 0; db < DC / 32; ++db) acc[db] = zero16();
  const auto product = [&](int slot, const Frag<D> (&p)[2 * KB]) {
#pragma unroll
    for (int st = 0; st < 2 * KB; ++st)
#pragma unroll
      for (int db = 0; db < DC / 32; ++db) acc[db] = mma<D>(rd.column_frag(slot * kTile, st * 16, db), p[st], acc[db]);
  };

  RowState state;
  if (tiles > 0) {
    // Step t reads k of tile t + 1 and v of tile t - 1 and starts the loads of k of tile t + 2 and
    // v of tile t, whose slots step t - 1 read last.  v of tile -1 is zeros.
    load_k(0, 0);
    load_k(1, 1);
    load_v(-1, 1);
    wait_vmcnt<2 * Loader::N>();
    barrier_no_fence();
    f32x16_t s0[KB], s1[KB];
    Frag<D> p[2 * KB];
#pragma unroll
    for (int st = 0; st < 2 * KB; ++st)
#pragma unroll
      for (int i = 0; i < Elem<D>::kSize / 2; ++i) p[st].v[i] = make_uint4(0, 0, 0, 0);
    scores(0, s0);
    const auto step = [&](int t, int slot, f32x16_t (&s)[KB], f32x16_t (&next)[KB]) {
      wait_lgkmcnt0();  // this wave's reads of the slots that are about to be loaded have returned
      wait_vmcnt<0>();
      barrier_no_fence();
      load_k(t + 2, slot);
      load_v(t, slot);
      const int key = (t * KG + part) * KEYS;
      if (key + KEYS > left) {  // keys past the end (perhaps all)
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (key + kb * 32 + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3) >= left) s[kb][i] = -INFINITY;
      }
      scores(slot ^ 1, next);
      float shrink;
      const bool moves = softmax_tile<D, KB>(s, c, state, &shrink);
      product(slot ^ 1, p);
#pragma unroll
      for (int st = 0; st < 2 * KB; ++st) {
        p[st] = to_frag<D>(s[st / 2], st % 2);
        pin<D>(p[st]);
      }
      if (moves) {
#pragma unroll
        for (int db = 0; db < DC / 32; ++db)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[db][i] *= shrink;
      }
    };
    const int steps = (tiles + KG - 1) / KG;
    for (int t = 0;;) {
      step(t, 0, s0, s1);
      if (++t == steps) break;
      step(t, 1, s1, s0);
      if (++t == steps) break;
    }
    wait_lgkmcnt0();
    wait_vmcnt<0>();
    barrier_no_fence();
    product((steps - 1) % 2, p);
  }
  float sum = half_sum(state.sum);
  if constexpr (KG == 2) {
    const uint32_t at = lds_offset(s_kv) + wave * (DC / 32 * 4096);
    wait_lgkmcnt0();
    __syncthreads();  // (every part is done with its tiles)
    if (part == 1) {
      put_acc<DC>(at, acc, lane);
      s_join[wave * 64 + lane] = make_float2(state.base, sum);
    }
    __syncthreads();
    if (part == 1) return;
    const float2 other = s_join[wave * 64 + lane];
    const float base = fmaxf(state.base, other.x);
    const float mine = exp2_fast(state.base - base), theirs = exp2_fast(other.x - base);
    add_acc<DC>(at, acc, mine, theirs, lane);
    sum = fmaf(other.y, theirs, sum * mine);
    state.base = base;
  }
  if (!there) return;
  if (CUT == kCutAll || (CUT == kCutLast && share.part >= 0)) {
    const int64_t at = (int64_t)share.place * kRows + wave * 32 + (lane & 31);
    if (lane < 32) a.state[at] = make_float2(nk > 0 ? state.base : -INFINITY, sum);
    if (tiles == 0) return;
    float* o = a.part + at * DP;
#pragma unroll
    for (int db = 0; db < DC / 32; ++db)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(o + db * 32 + 8 * i + 4 * (lane >> 5)) =
            make_float4(acc[db][4 * i], acc[db][4 * i + 1], acc[db][4 * i + 2], acc[db][4 * i + 3]);
    return;
  }
  store_row<D, DC>(qmap.at<D>(out, row), acc, tiles > 0 ? 1.f / sum : 0.f, a.head_dim, lane);
  if (a.lse != nullptr && lane < 32)
    a.lse[qmap.stat(row, a.heads)] = tiles > 0 ? (state.base + log2f(sum)) * kLn2 : -INFINITY;
}

// Joins the parts of a tile (blockIdx.x of those in parts), DP / 4 threads a row, blockIdx.y the
// rows of the tile.
template <DT D, int DP, int W>
__global__ __launch_bounds__(256) void attention_join_kernel(FwdArgs a) {
  constexpr int kThreads = DP / 4, kRows = 32 * W;
  const int group = a.heads / a.kv_heads, parts = a.cut.parts;
  const Share share = tile_share(a.cut, blockIdx.x);
  int tile;
  const int item = find_item(a.q_offsets, a.nq, a.items, group, kRows, share.slot, &tile);
  int64_t q0;
  int nq;
  item_rows(a.q_offsets, a.nq, item, &q0, &nq);
  const int rows = nq * group;
  const RowMap qmap{q0, share.head * group, group};
  const Heads<D> out = heads_of<D>(a.out);
  const int c = threadIdx.x % kThreads * 4;
  const int r = blockIdx.y * (256 / kThreads) + threadIdx.x / kThreads;
  const int64_t row = (int64_t)tile * kRows + r;
  if (row >= rows) return;
  const int64_t first = (int64_t)share.place * kRows + r;
  // The parts in batches, every load of a batch in flight at once, joined as a running softmax.
  constexpr int kBatch = 8;
  float base = -INFINITY, sum = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < parts; s0 += kBatch) {
    float2 st[kBatch];
    float4 p[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t at = first + (int64_t)min(s0 + i, parts - 1) * kRows;
      st[i] = a.state[at];
      p[i] = *reinterpret_cast<const float4*>(a.part + at * DP + c);
    }
    float top = base;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) top = fmaxf(top, st[i].x);
    if (top == -INFINITY) continue;  // (no keys: the same in every part)
    const float shrink = exp2_fast(base - top);
    base = top;
    sum *= shrink;
    o.x *= shrink;
    o.y *= shrink;
    o.z *= shrink;
    o.w *= shrink;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      // a share without keys has a sum of 0 and wrote no part
      const bool some = s0 + i < parts && st[i].y != 0.f;
      const float w = some ? exp2_fast(st[i].x - base) : 0.f;
      sum = fmaf(w, some ? st[i].y : 0.f, sum);
      o.x = fmaf(w, some ? p[i].x : 0.f, o.x);
      o.y = fmaf(w, some ? p[i].y : 0.f, o.y);
      o.z = fmaf(w, some ? p[i].z : 0.f, o.z);
      o.w = fmaf(w, some ? p[i].w : 0.f, o.w);
    }
  }
  const bool none = base == -INFINITY;  // the item has no keys
  const float f = none ? 0.f : 1.f / sum;
  if (c < a.head_dim) store4<D>(qmap.at<D>(out, (int)row) + c, o.x * f, o.y * f, o.z * f, o.w * f);
  if (a.lse != nullptr && c == 0) a.lse[qmap.stat((int)row, a.heads)] = none ? -INFINITY : (base + log2f(sum)) * kLn2;
}

template <DT D, int DC, int W, int KG, int CUT> hipError_t launch_tiles(const FwdArgs& a, hipStream_t stream) {
  constexpr int KEYS = D == DT::F32 ? 32 : 64, OCC = D == DT::F32 ? 1 : DC <= 64 && KG == 1 && CUT == kNoCut ? 3 : 2;
  const dim3 grid = CUT == kNoCut ? dim3((unsigned)a.cut.slots, (unsigned)a.kv_heads) : dim3((unsigned)cut_blocks(a.cut));
  attention_forward_kernel<D, DC, W, KG, KEYS, OCC, CUT><<<grid, KG * W * 64, 0, stream>>>(a);
  return hipGetLastError();
}

template <DT D, int DC, int W, int CUT> Status launch_cut(FwdArgs a, hipStream_t stream) {
  constexpr int DP = tile_width(DC);
  int dev = 0;
  SUBM_HIP_TRY(hipGetDevice(&dev));
  ScratchLease lease;
  const size_t rows = (size_t)cut_places(a.cut) * 32 * W;
  void* scratch = nullptr;
  Status st = lease.take(dev, stream, rows * (DP * sizeof(float) + sizeof(float2)), &scratch);
  if (!st.ok()) return st;
  a.part = static_cast<float*>(scratch);
  a.state = reinterpret_cast<float2*>(a.part + rows * DP);
  SUBM_HIP_TRY((launch_tiles<D, DC, W, 1, CUT>(a, stream)));
  attention_join_kernel<D, DP, W><<<dim3((unsigned)a.cut.cut, 32 * W * (DP / 4) / 256), 256, 0, stream>>>(a);
  SUBM_HIP_TRY(hipGetLastError());
  return Status{};
}

template <DT D, int DC>
Status launch(FwdArgs a, hipStream_t stream) {
  // 128 channels: 8 waves on one tile stream halve what each row reads of it (24,576 tokens, 16
  // heads, whole tiles: 2.33 ms, 4 waves 2.80), where they fill the compute units.  64 channels: 4
  // waves and three workgroups a compute unit, whose exponentials, the bound there, overlap (9,371
  // rows, 12 heads: 47.9 us, 8 waves 66.7).
  constexpr int kUnits = 256;
  constexpr bool kWide = D != DT::F32 && tile_width(DC) == 128;
  const int64_t rows = a.nq * (a.heads / a.kv_heads), keys = a.nk / a.items, spare = (int64_t)a.items * a.kv_heads;
  // float32 scores take 8 times as long, so its parts may be short.
  constexpr int kShare = D == DT::F32 ? 32 : 512;
  if constexpr (kWide) {
    const int64_t slots = rows / 256 + a.items;
    if (slots * a.kv_heads >= kUnits && rows / a.items >= 256) {
      a.cut = plan_cut(slots, a.kv_heads, spare, keys, kShare, kUnits, 0, kGainAt128);
      if (a.cut.parts > 1) return launch_cut<D, DC, 8, kCutLast>(a, stream);
      SUBM_HIP_TRY((launch_tiles<D, DC, 8, 1, kNoCut>(a, stream)));
      return Status{};
    }
  }
  // Few tiles: parts for two workgroups a unit (float32: one).  Last tiles in parts: not at 64
  // channels, whose last workgroups speed up as others leave their unit (24,576 tokens, 16 heads: 1.34
  // ms, 1.39 in parts), nor at the short items that are left here at 128.
  const int64_t slots = rows / 128 + a.items, tiles = slots * a.kv_heads;
  constexpr int kFew = kUnits * (D == DT::F32 ? 1 : 2);
  a.cut = plan_cut(slots, a.kv_heads, spare, keys, kShare, D == DT::F32 ? kUnits : INT32_MAX, kFew, kGain);
  // Where a compute unit gets one workgroup, two groups of waves on each tile (2,000 tokens, 16 heads
  // of 128: 42 us, 54 in two parts; with fewer than 512 keys the join eats the gain).  float32 waves
  // need the registers of two.
  if constexpr (D != DT::F32) {
    if (tiles <= kUnits && keys >= 512 && a.cut.parts <= 2) {
      SUBM_HIP_TRY((launch_tiles<D, DC, 4, 2, kNoCut>(a, stream)));
      return Status{};
    }
  } else {
    if (a.cut.parts > 1 && a.cut.whole > 0) return launch_cut<D, DC, 4, kCutLast>(a, stream);
  }
  if (a.cut.parts > 1) return launch_cut<D, DC, 4, kCutAll>(a, stream);
  SUBM_HIP_TRY((launch_tiles<D, DC, 4, 1, kNoCut>(a, stream)));
  return Status{};
}

template <DT D> Status launch_dim(const FwdArgs& a, hipStream_t stream) {
  if (a.head_dim <= 32) return launch<D, 32>(a, stream);
  if (a.head_dim <= 64) return launch<D, 64>(a, stream);
  if (a.head_dim <= 96) return launch<D, 96>(a, stream);
  return launch<D, 128>(a, stream);
}

}  // namespace

Status check_attention(const AttentionShape& s) {
  if (s.dtype != SUBM_F32 && s.dtype != SUBM_F16 && s.dtype != SUBM_BF16)
    return make_status(SUBM_ERR_UNSUPPORTED, "dtype must be SUBM_F32, SUBM_F16 or SUBM_BF16");
  // Rows are counted in 32 bits, up to a few tiles past the last, and a launch of 256 threads for each
  // 128 of them (and one more an item) has at most 2^32 - 1.
  constexpr int64_t kMost = (int64_t(1) << 31) - (int64_t(1) << 24);
  if (s.nq < 0 || s.nk < 0 || s.nq > kMost || s.nk > kMost)
    return make_status(SUBM_ERR_INVALID_ARG, "nq and nk must be 0 .. 2^31 - 2^24");
  if (s.items < 1 || s.items > 65535) return make_status(SUBM_ERR_INVALID_ARG, "items must be 1 .. 65535");
  if (s.heads < 1 || s.kv_heads < 1 || s.heads % s.kv_heads != 0)
    return make_status(SUBM_ERR_INVALID_ARG, "heads must be a positive multiple of kv_heads");
  if (s.kv_heads > 65535) return make_status(SUBM_ERR_INVALID_ARG, "kv_heads exceeds 65535");
  if (s.heads / s.kv_heads > 128) return make_status(SUBM_ERR_UNSUPPORTED, "more than 128 query heads a key head");
  if (s.nq * s.heads > kMost) return make_status(SUBM_ERR_INVALID_ARG, "nq * heads exceeds 2^31 - 2^24");
  if (s.head_dim < 1) return make_status(SUBM_ERR_INVALID_ARG, "head_dim must be at least 1");
  if (s.head_dim % 8 != 0 || s.head_dim > 128)
    return make_status(SUBM_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 up to 128");
  if (!std::isfinite(s.scale)) return make_status(SUBM_ERR_INVALID_ARG, "scale must be finite");
  if (s.q_offsets == nullptr || s.k_offsets == nullptr)
    return make_status(SUBM_ERR_INVALID_ARG, "q_offsets or k_offsets is NULL");
  if (((reinterpret_cast<uintptr_t>(s.q_offsets) | reinterpret_cast<uintptr_t>(s.k_offsets)) & 7u) != 0)
    return make_status(SUBM_ERR_INVALID_ARG, "an offsets pointer is not 8-byte aligned");
  return Status{};
}

Status check_heads(const subm_heads_t* t, int64_t rows, int heads, const AttentionShape& s, bool written,
                   const char* what) {
  const std::string name(what);
  if (t == nullptr) return make_status(SUBM_ERR_INVALID_ARG, name + " is NULL");
  if (rows == 0) return Status{};
  if (t->data == nullptr) return make_status(SUBM_ERR_INVALID_ARG, name + ".data is NULL");
  const int64_t size = s.dtype == SUBM_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(t->data) & 15u) != 0 || t->row_stride * size % 16 != 0 || t->head_stride * size % 16 != 0)
    return make_status(SUBM_ERR_UNSUPPORTED, name + ": data and strides must be multiples of 16 bytes");
  const int64_t limit = (int64_t(1) << 22) / size;
  if (t->row_stride < 0 || t->head_stride < 0 || t->row_stride > limit || t->head_stride > limit)
    return make_status(SUBM_ERR_UNSUPPORTED, name + ": strides must be 0 .. 2^22 bytes");
  // (a tile of 32 rows is addressed with 31 bits from its first token)
  if (t->head_stride * size * (heads / std::max(s.kv_heads, 1)) > (int64_t(1) << 30))
    return make_status(SUBM_ERR_UNSUPPORTED, name + ": the heads of one key head span more than 2^30 bytes");
  if (written && ((rows > 1 && t->row_stride == 0) || (heads > 1 && t->head_stride == 0)))
    return make_status(SUBM_ERR_INVALID_ARG, name + " is written and must not overlap itself");
  return Status{};
}

}  // namespace submconv

using namespace submconv;

extern "C" int sparse_attention_forward(const subm_heads_t* q, const subm_heads_t* k, const subm_heads_t* v, int64_t nq,
                                        int64_t nk, const int64_t* q_offsets, const int64_t* k_offsets, int items,
                                        int heads, int kv_heads, int head_dim, int dtype, float scale,
                                        const subm_heads_t* out, float* lse, hipStream_t stream) {
  return no_throw([&]() -> int {
    clear_error();
    const AttentionShape shape{nq, nk, q_offsets, k_offsets, items, heads, kv_heads, head_dim, dtype, scale};
    Status st = check_attention(shape);
    if (st.ok()) st = check_heads(q, nq, heads, shape, false, "q");
    if (st.ok()) st = check_heads(k, nk, kv_heads, shape, false, "k");
    if (st.ok()) st = check_heads(v, nk, kv_heads, shape, false, "v");
    if (st.ok()) st = check_heads(out, nq, heads, shape, true, "out");
    if (!st.ok()) return fail(st);
    if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return fail(SUBM_ERR_INVALID_ARG, "lse is not 4-byte aligned");
    if (nq == 0) return SUBM_OK;
    if (out->data == k->data || out->data == v->data) return fail(SUBM_ERR_INVALID_ARG, "out must not alias k or v");
    if (out->data == q->data && ((nq > 1 && out->row_stride != q->row_stride) || (heads > 1 && out->head_stride != q->head_stride)))
      return fail(SUBM_ERR_INVALID_ARG, "out over q needs the same strides");
    const FwdArgs a{*q, *k, *v, *out, lse, q_offsets, k_offsets, nq, nk, items, heads, kv_heads,
                    head_dim, scale, Cut{}, nullptr, nullptr};
    if (dtype == SUBM_F32) st = launch_dim<DT::F32>(a, stream);
    else if (dtype == SUBM_F16) st = launch_dim<DT::F16>(a, stream);
    else st = launch_dim<DT::BF16>(a, stream);
    if (!st.ok()) return fail(st);
    return SUBM_OK;
  });
}
