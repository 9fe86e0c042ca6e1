/*
 * conv_gb300_attention.h -- C ABI of libconvgb300.so: the attention that
 * stands between the convolutions of a text-conditioned image model.
 *
 *  - cross_attention_fwd / cross_attention_bwd: softmax attention of queries
 *    to an encoder's states of another length;
 *  - qk_norm_rope_fwd / qk_norm_rope_bwd: the root-mean-square norm of
 *    queries and keys for each head, with the position rotation.
 *
 * A feature map [n][h][w][heads * d] of the convolutions is a query tensor
 * [n][h * w][heads][d] as it stands: nothing is copied between them.
 *
 * The conventions of conv_gb300.h hold: device pointers, 16-byte aligned; the
 * caller owns all memory; calls are asynchronous on `stream`; validation
 * failures return before any launch and write nothing; workspaces start with
 * the CONV_STATUS_BYTES status region, zeroed once by the caller and read by
 * conv_check_device_status.  Calls that may overlap on the GPU need separate
 * workspaces; calls that follow one another, the convolutions' among them, may
 * share one.  Lengths and the batch may be zero here.
 */
#ifndef CONV_GB300_ATTENTION_H
#define CONV_GB300_ATTENTION_H

#include <stddef.h>

#include "conv_gb300.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Cross attention.  For batch b, query head h, query i and key j, with the
 * key head g = h / (heads / kv_heads):
 *   s_ij = scale * sum_d q[b][i][h][d] * k[b][j][g][d]
 *   lse_i = log sum_j exp(s_ij),  p_ij = exp(s_ij - lse_i)
 *   out[b][i][h][d] = sum_j p_ij * v[b][j][g][d]
 * over the pairs (i, j) that take part: j < kv_lengths[b] (when given) and
 * mask[b][h][i][j] != 0 (when given).  A query with no key gives out = 0 and
 * lse = -inf, and its gradients are 0.  Keys that no query may attend, and in
 * the backward pass queries that attend no key, are never multiplied: their
 * rows may hold anything, infinities and NaN among them.  (A row that some
 * query attends is used in products with whole tiles of queries, so it has to
 * be finite for those that do not attend it, too.)
 * Backward, with dout of out:
 *   dv_j = sum_i p_ij dout_i,  delta_i = sum_d dout_i[d] out_i[d]  (of the
 *   rounded out that is passed in, or summed anew where all keys are one tile)
 *   ds_ij = p_ij (dout_i . v_j - delta_i)
 *   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
 * dk and dv sum over the query heads that share the key head.  Sums run in a
 * fixed order: equal calls give equal bits.
 *
 * Scores, sums and statistics are fp32; probabilities and ds are rounded to
 * `dtype` for the products that take them; results are rounded once.  F16:
 * probabilities are rounded after a scaling by 2^7 (backward 2^15), ds after one
 * by a power of two from the norms of dout and v: for dq each query's own, for
 * dk one for a part of a request's and key head's queries, where what is below
 * 2^-29 of the largest 2 |dout| |v| is rounded in steps of 2^-40 of it.
 *
 * Layouts: [batch][length][heads][head_dim] with any strides (in elements,
 * {batch, token, head}; the innermost stride is 1).  Strides are multiples of
 * 8; strides of inputs may be 0 along batch and heads (a broadcast); strides
 * along dimensions of extent 1 are ignored.  lse is dense [batch][heads]
 * [q_len].  mask is bytes (0 = left out) with any strides, 0 among them.
 *
 * Gates (CONV_ERR_NOT_SUPPORTED): dtype BF16 or F16; head_dim a multiple of 8
 * up to 128; batch * heads * (q_len + 128) and batch * kv_heads * (kv_len +
 * 128) below 2^31.  CONV_ERR_INVALID_VALUE: null pointers, negative sizes,
 * heads not a multiple of kv_heads, negative strides, zero strides of outputs
 * or along tokens, a scale that is not finite and positive.
 * CONV_ERR_MISALIGNED: a pointer off 16 bytes (lse and kv_lengths: 4) or a
 * stride that is no multiple of 8.  CONV_ERR_DEVICE_TIMEOUT, by
 * conv_check_device_status: a wait inside a kernel ran out.
 * kv_lengths values are taken as clamped to [0, kv_len].
 * ------------------------------------------------------------------------ */
typedef struct {
  int dtype; /* conv_dtype_t */
  int batch, heads, kv_heads, q_len, kv_len, head_dim;
  float scale;
  const void* q;
  const void* k;
  const void* v;
  void* out;              /* written by the forward pass, read by the backward pass */
  float* lse;             /* as out; may be NULL in the forward pass */
  const int* kv_lengths;  /* [batch], or NULL */
  const unsigned char* mask; /* or NULL */
  const void* dout;       /* the rest: backward pass only */
  void* dq;
  void* dk;
  void* dv;
  long long q_stride[3], k_stride[3], v_stride[3], out_stride[3]; /* batch, token, head */
  long long dout_stride[3], dq_stride[3], dk_stride[3], dv_stride[3];
  long long mask_stride[4]; /* batch, head, query, key */
} cross_attention_args_t;

/* Workspace bytes of a call on the current device (the status region
 * included): packed mask bits, partial results of work split along the keys
 * (forward) or the queries (backward), row sums (backward).  With `backward`
 * they serve both passes.  Of `args` only the sizes, the dtype, whether mask
 * is NULL and its strides are read. */
size_t cross_attention_workspace_size(const cross_attention_args_t* args, int backward);

conv_status_t cross_attention_fwd(const cross_attention_args_t* args, void* workspace,
                                  size_t workspace_bytes, void* stream);

conv_status_t cross_attention_bwd(const cross_attention_args_t* args, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Norm of queries and keys with the position rotation.  For every row x of a
 * head (head_dim = D elements), with weight w and the row's position t:
 *   r = 1 / sqrt(mean(x^2) + eps),  y = x * r * w
 * then each pair (a, b) = (y[i0], y[i1]), i < rot_dim / 2, becomes
 *   (a cos - b sin, b cos + a sin),  cos, sin = tables[t][i]
 * with (i0, i1) = (i, i + rot_dim / 2), or (2i, 2i + 1) when adjacent_pairs.
 * Elements from rot_dim on are not rotated.  Backward, with g the gradient
 * rotated back: dw = sum over rows of g * x * r (fp32),
 *   dx = r * (g w - x r * mean(g w x r)).
 * Both tensors go through one launch; either may be left out (NULL x).
 * The weight gradient sums in a fixed order.
 *
 * x, y, dy, dx: [batch][length][heads][D] of `dtype` (BF16 or F16), strides
 * {batch, token, head} in elements, multiples of 8 (ignored for extents of
 * 1; nonzero for outputs).  weight: [D], fp32 or `dtype`.  cos, sin: dense
 * fp32 [table_rows][rot_dim / 2].  positions: int32 [batch][length] with
 * batch stride position_stride (0: shared by the batch), or NULL for
 * 0 .. length-1; they are clamped to [0, table_rows - 1].
 * Gates: D a multiple of 8 up to 256; rot_dim a multiple of 8 up to D, or 0;
 * batch * length * heads up to 0x7FFF0000, strides below 2^35
 * (CONV_ERR_NOT_SUPPORTED).
 * ------------------------------------------------------------------------ */
typedef struct {
  const void* x;
  const void* weight;
  const int* positions;
  void* y;               /* forward */
  const void* dy;        /* backward, as the next two */
  void* dx;
  float* dweight;        /* [D] */
  int length, heads;
  int weight_f32;        /* weight is fp32, not `dtype` */
  long long position_stride;
  long long x_stride[3], y_stride[3], dy_stride[3], dx_stride[3];
} qk_norm_rope_tensor_t;

typedef struct {
  int dtype; /* conv_dtype_t */
  int batch, head_dim, rot_dim, table_rows;
  int adjacent_pairs;
  float eps;
  const float* cos;
  const float* sin;
  qk_norm_rope_tensor_t q, k;
} qk_norm_rope_args_t;

conv_status_t qk_norm_rope_fwd(const qk_norm_rope_args_t* args, void* stream);

/* Workspace bytes of the backward pass on the current device. */
size_t qk_norm_rope_workspace_size(int head_dim);

conv_status_t qk_norm_rope_bwd(const qk_norm_rope_args_t* args, void* workspace,
                               size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONV_GB300_ATTENTION_H */
