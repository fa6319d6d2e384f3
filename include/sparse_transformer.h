/*
 * sparse_transformer.h -- C ABI of the operators of a sparse transformer block: norms, embeddings,
 * rotary positions and attention over the items of a sparse tensor, each with its backward pass.
 * Part of libsubmconv.so; status codes, dtypes, pointer and stream conventions are those of
 * submconv.h.
 *
 * These are the per-token layers of the flow models and cross blocks that the sparse decoders
 * belong to: attention in its full mode over the voxels of an item (lato.2_mrp_mlx README, scope
 * table, the attention row), rotary phases from voxel coordinates (trellis_sparse_mrp_mlx commit
 * log, the rope_phases_from_coords commit) and layer norms with and without affine weights
 * (the same log, the cross-block commit: norm1 / norm3 non-affine, norm2 affine).
 *
 * Rows (tokens) of all items are concatenated; item b holds rows offsets[b] .. offsets[b+1] - 1.
 * No call synchronises.  Every result is bitwise reproducible from run to run: no sum goes
 * through atomics.
 *
 * The backward passes of the norms (with weight gradients) and of the embedding, and attention forward
 * and backward may keep partial results in scratch memory of the stream, which grows
 * to the largest call so far and is given back by subm_release_cached_memory.  It cannot grow
 * under graph capture (SUBM_ERR_UNSUPPORTED): make the call once on the capturing stream before.
 * The scratch memory of captured calls is kept apart from that of other calls: a captured call stays
 * valid until subm_release_cached_memory, and its graph may be replayed on any stream.  Calls that
 * were captured on one stream share their scratch memory, so replays of different graphs from one
 * stream must not overlap.
 */
#ifndef SPARSE_TRANSFORMER_H
#define SPARSE_TRANSFORMER_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "submconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * One tensor of token rows split into heads: element c of head h of row r is at
 * data[r * row_stride + h * head_stride + c], strides in elements.  A packed projection is read
 * and written in place through it (queries, keys and values of one [n, heads, head_dim] buffer
 * are three views with one row stride).
 */
typedef struct {
  void* data; /* device pointer; an input is not written */
  int64_t row_stride;
  int64_t head_stride;
} subm_heads_t;

/* ------------------------------------------------------------------------------ layer norm */

/*
 * sparse_layer_norm_forward -- y = (x - mean) * rstd * gamma + beta over the channels of each
 * row, mean and the biased variance in float32, rstd = 1 / sqrt(var + eps).
 *   x, y         device [n, channels] in `dtype` (SUBM_F32 / SUBM_F16 / SUBM_BF16), aligned to
 *                their element; y may be x (in place), any other overlap is undefined.
 *   n            0 <= n <= 2^31 - 1; n == 0 returns SUBM_OK with no launch.
 *   channels     1 .. 16384, any value.
 *   gamma, beta  device [channels] in `dtype`, each may be NULL for 1 and 0.
 *   eps          > 0 and finite.
 *   mean, rstd   device float32 [n], both or neither NULL: what the backward pass needs.
 * The variance is taken of the centred values (two passes over registers), so a mean far from
 * zero costs no digits.  Errors: SUBM_ERR_INVALID_ARG, SUBM_ERR_UNSUPPORTED, SUBM_ERR_HIP.
 */
int sparse_layer_norm_forward(const void* x, int64_t n, int channels, int dtype, const void* gamma,
                              const void* beta, float eps, void* y, float* mean, float* rstd,
                              hipStream_t stream);

/*
 * sparse_layer_norm_backward -- gradients of sparse_layer_norm_forward.  With
 * h = (x - mean) rstd and a = dy gamma:
 *   dx = rstd (a - mean_c(a) - h mean_c(a h)),  dgamma = sum_r dy h,  dbeta = sum_r dy.
 *   dy, x          device [n, channels] in `dtype`.
 *   gamma          as in the forward pass (NULL for 1).
 *   mean, rstd     the forward pass's statistics.
 *   dx             device [n, channels] in `dtype`; may be dy (in place).
 *   dgamma, dbeta  device [channels] in `dtype`, overwritten; both or neither NULL (no weight
 *                  gradients).  n == 0 writes zeros.
 * The row sums of dgamma and dbeta are float32, per workgroup and then over workgroups in a
 * fixed order, rounded once.  Errors: as the forward pass, and SUBM_ERR_OUT_OF_MEMORY.
 */
int sparse_layer_norm_backward(const void* dy, const void* x, int64_t n, int channels, int dtype,
                               const void* gamma, const float* mean, const float* rstd, void* dx, void* dgamma,
                               void* dbeta, hipStream_t stream);

/* ------------------------------------------------------------------ root-mean-square norm */

/*
 * sparse_rms_norm_forward -- with t = x + residual,
 *   y = t * rstd * gamma,   rstd = 1 / sqrt(mean_c(t^2) + eps),   total = t,
 * the step between two layers of a block: the layer's output x joins the residual stream, which is
 * normalised for the next layer.  t and its square sum are float32; y is of t before total rounds it.
 *   x, residual  device [n, channels] in `dtype`, aligned to their element; residual may be NULL (t = x).
 *   n            0 <= n <= 2^31 - 1; n == 0 returns SUBM_OK with no launch.
 *   channels     1 .. 16384, any value.
 *   gamma        device [channels] in `dtype`, may be NULL for 1.
 *   eps          > 0 and finite.
 *   y            device [n, channels] in `dtype`; may be x or residual (in place).
 *   total        device [n, channels] in `dtype`, required with a residual, else it may be NULL; may be x or
 *                residual (in place) but not y.  Any other overlap is undefined.
 *   rstd         device float32 [n], or NULL: what the backward pass needs beside total.
 * Errors: SUBM_ERR_INVALID_ARG, SUBM_ERR_UNSUPPORTED, SUBM_ERR_HIP.
 */
int sparse_rms_norm_forward(const void* x, const void* residual, int64_t n, int channels, int dtype, const void* gamma,
                            float eps, void* y, void* total, float* rstd, hipStream_t stream);

/*
 * sparse_rms_norm_quantize_forward -- sparse_rms_norm_forward with y in 8 bits, for a linear layer in 8
 * bits: y = q * scale with one scale for `group` consecutive channels of a row,
 *   scale = max(max |y| / 448, 2^-126),   q = y / scale rounded to nearest even (e4m3, largest 448).
 *   group   32, 64 or 128 channels (the last group of a row may be shorter), or 0 for the whole row.
 *   q       device [n, channels] bytes, e4m3 without infinities; it must not overlap another argument.
 *   scales  device float32 [n, ceil(channels / group)] ([n] for group 0).
 * The maximum is of the values that are numbers: NaN comes out as NaN, and leaves its group's scale alone;
 * an infinite value makes the scale infinite, the value NaN and the rest of its group 0.
 * The other arguments and errors are those of sparse_rms_norm_forward.  y has no gradient of its own: the
 * backward pass takes that of the 16- or 32-bit y (q / scale taken as y).
 */
int sparse_rms_norm_quantize_forward(const void* x, const void* residual, int64_t n, int channels, int dtype,
                                     const void* gamma, float eps, int group, void* q, float* scales, void* total,
                                     float* rstd, hipStream_t stream);

/*
 * sparse_rms_norm_backward -- gradients of sparse_rms_norm_forward.  With h = total * rstd and a = dy gamma:
 *   dx = rstd (a - h mean_c(a h)) + dtotal,   dgamma = sum_r dy h;
 * dx is the gradient of x and of residual alike.
 *   dy, total  device [n, channels] in `dtype`; total is the forward pass's (x without a residual).
 *   dtotal     the gradient of total, [n, channels], or NULL for none.
 *   gamma, rstd  as in the forward pass.
 *   dx         device [n, channels] in `dtype`; may be dy or dtotal (in place).
 *   dgamma     device [channels] in `dtype`, overwritten, or NULL (no weight gradient).  n == 0 writes zeros.
 * The row sums of dgamma are float32, per workgroup and then over workgroups in a fixed order, rounded
 * once.  Errors: as the forward pass, and SUBM_ERR_OUT_OF_MEMORY.
 */
int sparse_rms_norm_backward(const void* dy, const void* total, const void* dtotal, int64_t n, int channels, int dtype,
                             const void* gamma, const float* rstd, void* dx, void* dgamma, hipStream_t stream);

/* -------------------------------------------------------------------------------- embedding */

/*
 * sparse_embedding_forward -- out_i = scale * table[tokens_i], rounded once: rows of a learned table for
 * tokens that name them (codebook entries of voxels, words of a prompt).
 *   table        device [rows, channels] in `dtype`, aligned to its element.
 *   rows         1 .. 2^21.
 *   channels     1 .. 16384, any value.
 *   tokens       device [n], integers of token_bytes (4 or 8) bytes.  A token outside 0 .. rows - 1 (padding,
 *                -1) gives a row of zeros.
 *   n            0 <= n <= 2^31 - 1; n == 0 returns SUBM_OK with no launch.
 *   scale        finite.
 *   out          device [n, channels] in `dtype`; it must not overlap the table.
 * Errors: SUBM_ERR_INVALID_ARG, SUBM_ERR_UNSUPPORTED, SUBM_ERR_HIP.
 */
int sparse_embedding_forward(const void* table, int rows, int channels, int dtype, const void* tokens, int token_bytes,
                             int64_t n, float scale, void* out, hipStream_t stream);

/*
 * sparse_embedding_backward -- dtable_t = scale * sum of dout_i over the tokens_i that are t, every row of
 * dtable [rows, channels] overwritten (zeros where no token names it).  The tokens are sorted by row and
 * position, so each float32 sum has one order; it is rounded once.  dtable must not overlap dout.  Other
 * arguments as in the forward pass.  Errors: as the forward pass, and SUBM_ERR_OUT_OF_MEMORY.
 */
int sparse_embedding_backward(const void* dout, int rows, int channels, int dtype, const void* tokens, int token_bytes,
                              int64_t n, float scale, void* dtable, hipStream_t stream);

/* ------------------------------------------------------------------------- rotary positions */

/* Which two channels of a head form pair i of `pairs` pairs. */
typedef enum {
  SUBM_ROPE_INTERLEAVED = 0, /* 2i and 2i + 1 */
  SUBM_ROPE_HALF = 1         /* i and i + pairs */
} subm_rope_layout_t;

/* How the frequencies stretch to a context `factor` times the one that was trained on. */
typedef enum {
  SUBM_ROPE_PLAIN = 0,  /* base^(-i / count) */
  SUBM_ROPE_LINEAR = 1, /* all divided by factor */
  SUBM_ROPE_BASE = 2,   /* a larger base: the highest is kept, the lowest divided by factor */
  SUBM_ROPE_PARTS = 3   /* by turns over the trained length: above 32 kept, below 1 divided, blended between */
} subm_rope_scaling_t;

/*
 * sparse_rope_frequencies -- the `count` frequencies of one axis, on the host (double arithmetic,
 * rounded to float32), and the factor that the rotated channels are multiplied by.
 *   count           >= 1 pairs of an axis; frequency i starts from base^(-i / count).
 *   base            > 1.
 *   scaling         a subm_rope_scaling_t.
 *   factor          >= 1 (1 leaves every scaling plain).
 *   trained_length  > 0, positions of the trained context (SUBM_ROPE_PARTS only).
 *   freq            host float [count].
 *   magnitude       host float: 0.1 ln(factor) + 1 for SUBM_ROPE_PARTS, else 1; may be NULL.
 * Touches no device.  Errors: SUBM_ERR_INVALID_ARG.
 */
int sparse_rope_frequencies(int count, double base, int scaling, double factor, double trained_length,
                            float* freq, float* magnitude);

/*
 * sparse_rope_forward -- rotates `axes * num_freq` channel pairs of every head of every row:
 * pair i turns by t = positions[r, i / num_freq] * freq[i % num_freq],
 *   (u, v) -> magnitude (u cos t - v sin t, v cos t + u sin t),
 * and copies the head's other channels.
 *   x, y             n rows of `heads` heads; the pairs take 2 axes num_freq <= head_dim
 *                    channels.  y may be x (same strides, in place); any other overlap is undefined.
 *   n                0 <= n <= 2^31 - 1; n == 0 returns SUBM_OK with no launch.
 *   heads, head_dim  1 .. 65535 and 1 .. 4096.
 *   positions        device int32, row r at positions + r * position_stride, `axes` values; voxel
 *                    coordinates (b, z, y, x) are passed as coords + 1 with stride 4 and 3 axes.
 *   freq             device float32 [num_freq].
 *   layout           a subm_rope_layout_t.
 * The angle is the exact product reduced to one turn in float64, so long positions lose no
 * digits; sine and cosine are computed once for all heads of a row.
 * Errors: SUBM_ERR_INVALID_ARG, SUBM_ERR_UNSUPPORTED, SUBM_ERR_HIP.
 */
int sparse_rope_forward(const subm_heads_t* x, int64_t n, int heads, int head_dim, int dtype,
                        const int32_t* positions, int64_t position_stride, int axes, const float* freq, int num_freq,
                        int layout, float magnitude, const subm_heads_t* y, hipStream_t stream);

/* sparse_rope_backward -- dx from dy: the rotation by -t with the same magnitude. */
int sparse_rope_backward(const subm_heads_t* dy, int64_t n, int heads, int head_dim, int dtype,
                         const int32_t* positions, int64_t position_stride, int axes, const float* freq, int num_freq,
                         int layout, float magnitude, const subm_heads_t* dx, hipStream_t stream);

/* -------------------------------------------------------------------------------- attention */

/*
 * sparse_attention_forward -- for every item and head,
 *   out = softmax(scale * q k^T) v,   lse = log sum_j exp(scale * q . k_j).
 *   q, out       nq rows of `heads` heads;  k, v  nk rows of `kv_heads` heads, `heads` a multiple
 *                of `kv_heads`: query head h reads key head h / (heads / kv_heads).
 *   q_offsets    device int64 [items + 1], non-decreasing from 0 to nq;  k_offsets  the same to
 *                nk (the same pointer for self attention).  They are not checked on the device:
 *                other values give unspecified results, but every access stays inside the tensors.
 *   items        1 .. 65535.  Items without queries or without keys are allowed: a query without
 *                keys gets out = 0 and lse = -infinity.
 *   nq, nk       0 .. 2^31 - 2^24, and nq * heads <= 2^31 - 2^24.
 *   heads        at most 128 a key head.
 *   head_dim     a multiple of 8, 8 .. 128.  data 16-byte aligned, strides multiples of 16 bytes
 *                (else SUBM_ERR_UNSUPPORTED); row strides of at most 2^22 bytes, head strides of at
 *                most 2^22 bytes.
 *   scale        finite; the forward pass takes magnitudes below 7e-31 as that.
 *   lse          device float32 [nq, heads], or NULL.
 *   out          may be q (same strides); it must not overlap k or v.
 * Scores, the running maximum and sum, and out accumulate in float32.  With 16-bit storage the
 * probabilities are rounded to it for the product with v (SUBM_F16: from 2^11 for the largest score
 * down, so that many small ones beside it keep their weight).  Rows of one item never meet values of
 * another, whatever they hold.  Where query rows do not fill the compute units evenly, keys are split
 * over workgroups and joined by a second kernel, with float32 partial results in the stream's scratch
 * memory.
 * Errors: SUBM_ERR_INVALID_ARG, SUBM_ERR_UNSUPPORTED, SUBM_ERR_OUT_OF_MEMORY, SUBM_ERR_HIP.
 */
int sparse_attention_forward(const subm_heads_t* q, const subm_heads_t* k, const subm_heads_t* v, int64_t nq,
                             int64_t nk, const int64_t* q_offsets, const int64_t* k_offsets, int items, int heads,
                             int kv_heads, int head_dim, int dtype, float scale, const subm_heads_t* out, float* lse,
                             hipStream_t stream);

/*
 * sparse_attention_backward -- gradients of sparse_attention_forward.  With
 * p = exp(scale q k^T - lse) recomputed from lse, dp = dout v^T and d = sum_c dout out:
 *   ds = scale p (dp - d),  dq = ds k,  dk = ds^T q,  dv = p^T dout,
 * dk and dv summed over the query heads that share a key head.
 *   dout, out, dq  nq rows of `heads` heads;  dk, dv  nk rows of `kv_heads` heads, overwritten.
 *                  The gradients must not overlap an input or each other.
 *   lse            the forward pass's, required.
 * A query without keys gets dq = 0, a key without queries dk = dv = 0.  With 16-bit storage p and
 * ds are rounded to it for their products; with SUBM_F16 both are scaled by powers of two first
 * (ds by the largest |dout| of its row for dq, of its item and head for dk, or by what the item's
 * longest row of v leaves room for), so that small gradients keep their digits and none overflows
 * before the products.  Other arguments and errors as in the forward pass.
 */
int sparse_attention_backward(const subm_heads_t* dout, const subm_heads_t* q, const subm_heads_t* k,
                              const subm_heads_t* v, const subm_heads_t* out, const float* lse, int64_t nq,
                              int64_t nk, const int64_t* q_offsets, const int64_t* k_offsets, int items, int heads,
                              int kv_heads, int head_dim, int dtype, float scale, const subm_heads_t* dq,
                              const subm_heads_t* dk, const subm_heads_t* dv, hipStream_t stream);

/* ------------------------------------------------------------ attention in a sliding window */

/*
 * sparse_window_attention_forward -- sparse_attention_forward where a query sees a part of its item's keys:
 * those next to its own position, and the first `sinks`.  Query i of an item with nq queries and nk keys stands
 * at key position p = i + nk - nq (the queries are the last tokens of a sequence whose keys are all its
 * tokens: a whole prompt, a chunk of one after a cache, or one new token) and sees key j if
 *   j <= p + right  and  (j >= p - left  or  j < sinks).
 *   left, right  >= 0; 2^31 or more leaves that end open (left open and right 0 is causal attention).
 *   sinks        0 .. 128 (else SUBM_ERR_UNSUPPORTED).  They are not seen before p + right reaches them.
 *   k_lengths    device int64 [items], or NULL: how many of an item's key rows are there (a cache with room
 *                behind its tokens); values outside 0 .. its rows are taken as the nearest.  Rows past it are not read.
 * A query that sees no key (p + right < 0, or an item without keys) gets out = 0 and lse = -infinity.  A key or
 * value that a query does not see, NaN and infinities included, does not change the query's result (a tile in
 * which such a value meets other rows is computed again row by row, which is slow; where a row
 * that sees such a value itself is not finite, infinity and NaN may stand for each other).  Only the tiles
 * of keys that some row of a block sees are read.  How the work is split goes by the items' mean lengths, which the
 * host knows: a batch of single tokens and one long prompt, or of one long cache among short ones, gives the same
 * results but takes longer than a call for each kind (bf16, 8 heads of 128: 255 tokens of 1,000 keys and a prompt of
 * 7,900 432 us, apart 379; 15 tokens of 200 keys and one of 60,000 201 us, apart 62).  All other arguments,
 * limits and errors are those of
 * sparse_attention_forward, and SUBM_ERR_INVALID_ARG for a negative left, right or sinks.
 */
int sparse_window_attention_forward(const subm_heads_t* q, const subm_heads_t* k, const subm_heads_t* v, int64_t nq,
                                    int64_t nk, const int64_t* q_offsets, const int64_t* k_offsets,
                                    const int64_t* k_lengths, int items, int heads, int kv_heads, int head_dim,
                                    int dtype, float scale, int64_t left, int64_t right, int sinks,
                                    const subm_heads_t* out, float* lse, hipStream_t stream);

/*
 * sparse_window_attention_backward -- gradients of sparse_window_attention_forward without k_lengths: those of
 * sparse_attention_backward, each sum over the keys that a query sees or the queries that see a key.  A key
 * that no query sees gets dk = dv = 0, and a query that sees no key dq = 0; what a query does not see changes
 * neither its dq nor, through it, other keys' gradients (SUBM_F16: ds is scaled for dq by what its row sees, for
 * dk by the rows that see its key).  The sinks' sums go through float32 partial results in
 * scratch memory, one a chunk of query rows and at least one an item: with many short items they take 8 bytes times
 * items, kv_heads, sinks and head_dim (rounded up to 64 or 128).
 */
int sparse_window_attention_backward(const subm_heads_t* dout, const subm_heads_t* q, const subm_heads_t* k,
                                     const subm_heads_t* v, const subm_heads_t* out, const float* lse, int64_t nq,
                                     int64_t nk, const int64_t* q_offsets, const int64_t* k_offsets, int items,
                                     int heads, int kv_heads, int head_dim, int dtype, float scale, int64_t left,
                                     int64_t right, int sinks, const subm_heads_t* dq, const subm_heads_t* dk,
                                     const subm_heads_t* dv, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_TRANSFORMER_H */
