/*
 * conv_gb300_decoder.h -- C ABI of libconvgb300.so: what a text decoder
 * between the convolutions needs beside conv_gb300_attention.h.
 *
 *  - layer_norm_fwd / layer_norm_bwd: the norm in front of the projections;
 *  - kv_cache_write / kv_cache_read: keys and values in pages and in 8 bits;
 *  - tree_attention_fwd: the attention of drafted tokens to that cache.
 *
 * The conventions of conv_gb300_attention.h hold: device pointers; the caller
 * owns all memory; calls are asynchronous on `stream`; validation failures
 * return before any launch and write nothing; workspaces start with the
 * CONV_STATUS_BYTES status region and may be shared by calls that follow one
 * another.  Batches, lengths and rows may be zero.
 */
#ifndef CONV_GB300_DECODER_H
#define CONV_GB300_DECODER_H

#include <stddef.h>

#include "conv_gb300_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Layer norm.  For every row x of C = channels elements:
 *   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps)
 *   y = (x - mean) * rstd * weight + bias
 * Backward, with xhat = (x - mean) * rstd and g = dy * weight:
 *   dx = rstd * (g - sum g / C - xhat * sum(g xhat) / C)
 *   dweight = sum over rows of dy * xhat,  dbias = sum over rows of dy
 * Sums are fp32, the forward pass's deviations are taken from the row's own
 * mean, and every sum runs in a fixed order: equal calls give equal bits.  A
 * finite row's squares and sum may pass fp32's range.  With eps = 0 a row of one
 * value has rstd = infinity (and y, as in the formula, is not a number).
 *
 * x, y, dy, dx: [batch][length][C] of `dtype` (BF16 or F16), strides {batch,
 * token} in elements (ignored for extents of 1; inputs may repeat a row with
 * a stride of 0; outputs may not).  y may be x, and dx may be dy or x, with
 * the same strides.  A feature map [n][h][w][C] is [n][h * w][C] as it stands.
 * weight, bias: [C], fp32 or `dtype`, either may be NULL (1 and 0); the
 * backward pass does not read bias.  mean, rstd: dense fp32 [batch][length],
 * written by the forward pass where not NULL, read by the backward pass.
 * dweight, dbias: dense fp32 [C], either may be NULL.
 * Gates (CONV_ERR_NOT_SUPPORTED): other dtypes; C above 16384; batch * length
 * above 0x7F000000; strides from 2^40 on.  CONV_ERR_INVALID_VALUE: negative
 * sizes or strides, eps negative or not finite, outputs with strides of 0,
 * missing tensors.  CONV_ERR_MISALIGNED: a pointer off its element's size.
 * (Rows are read 16 bytes at a time: fastest with C and strides multiples of 8
 * and tensors on 16-byte boundaries, then with any others up to C = 8185; beyond,
 * those go element by element.)
 * ------------------------------------------------------------------------ */
typedef struct {
  int dtype; /* conv_dtype_t */
  int batch, length, channels;
  int weight_f32; /* weight and bias are fp32, not `dtype` */
  float eps;
  const void* x;
  const void* weight;
  const void* bias;
  void* y;
  float* mean;
  float* rstd;
  const void* dy; /* the rest: backward pass only */
  void* dx;
  float* dweight;
  float* dbias;
  long long x_stride[2], y_stride[2], dy_stride[2], dx_stride[2]; /* batch, token */
} layer_norm_args_t;

conv_status_t layer_norm_fwd(const layer_norm_args_t* args, void* stream);

/* Workspace bytes of the backward pass on the current device (with neither
 * dweight nor dbias the status region's CONV_STATUS_BYTES do). */
size_t layer_norm_workspace_size(int channels);

conv_status_t layer_norm_bwd(const layer_norm_args_t* args, void* workspace,
                             size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * The cache.  Keys and values of kv_heads heads of D = head_dim elements lie
 * in pages of page_size tokens: k_cache and v_cache, e4m3 codes [pages]
 * [page_size][kv_heads][D] with any strides {page, token, head} (bytes,
 * multiples of 16; the innermost is 1), so also with the heads outside the
 * tokens.  scales: dense bytes [pages][kv_heads][page_size][2], for each row
 * the exponents, plus 127, of its key (first) and of its value:
 *   row = code * 2^(byte - 127)
 * A key's byte of 0 says that nothing was written there, whatever the value's
 * byte is: attention leaves such a token out (a cache whose scales start at zero
 * is empty).  Other bytes lie in [63, 247], as kv_cache_write gives them.
 * block_table: int32 [batch][table_width] with rows table_stride apart: token
 * p of request b is token p % page_size of page block_table[b][p / page_size].
 * Page numbers outside [0, pages) stand for no page: nothing is written
 * there, reading gives zeros, and attention leaves their tokens out.
 *
 * kv_cache_write quantises rows of k and v, [batch][length][kv_heads][D] of
 * `dtype` (BF16 or F16; strides {batch, token, head} in elements, multiples
 * of 8), as tokens starts[b] .. of request b.  The exponent is the smallest
 * (-64 at least) with which the row's largest finite element is at most 448,
 * 0 for rows of zeros; elements are rounded to nearest, ties to even, after
 * that exact scaling; infinities become +-448, NaN stays NaN.  With lengths
 * (int32 [batch]) only the first lengths[b] tokens are taken.  Tokens in front
 * of 0 or behind the table are left out.  No two tokens of a call may go to
 * the same place (requests that share a page only read it).
 *
 * kv_cache_read is the way back: k and v are written with the rows' values in
 * `dtype`, rounded to nearest, and limited to its largest finite number;
 * tokens from lengths[b] on keep what they hold.  Tokens outside the table
 * read as zeros.
 *
 * Gates (CONV_ERR_NOT_SUPPORTED): other dtypes; D no multiple of 16 or above
 * 128; page_size no multiple of 16; table_width * page_size or batch * length
 * * kv_heads above 0x7FFF0000.  CONV_ERR_INVALID_VALUE: missing tensors, a
 * cache without pages, negative sizes or strides, strides of 0 of what is
 * written.
 * CONV_ERR_MISALIGNED: pointers off 16 bytes (int32: 4), other strides.
 * ------------------------------------------------------------------------ */
typedef struct {
  int dtype; /* conv_dtype_t of k and v */
  int batch, length, kv_heads, head_dim;
  int pages, page_size, table_width;
  void* k; /* read by kv_cache_write, written by kv_cache_read, as v */
  void* v;
  void* k_cache; /* the other way round, as the next two */
  void* v_cache;
  unsigned char* scales;
  const int* block_table;
  const int* starts;  /* [batch], or NULL: 0 */
  const int* lengths; /* [batch], or NULL: length */
  long long table_stride;
  long long k_stride[3], v_stride[3];             /* batch, token, head */
  long long k_cache_stride[3], v_cache_stride[3]; /* page, token, head */
} kv_cache_args_t;

conv_status_t kv_cache_write(const kv_cache_args_t* args, void* stream);
conv_status_t kv_cache_read(const kv_cache_args_t* args, void* stream);

/* ------------------------------------------------------------------------
 * Attention of drafted tokens to the cache.  Request b has n = kv_lengths[b]
 * tokens in the cache, the last t = draft_lengths[b] of which (q_len without
 * draft_lengths) are drafts: they are written there before the call.  Draft
 * i, query i of q, attends the n - t tokens in front of the drafts, itself,
 * and the drafts on its way to the root of the tree:
 *   parents[b][i] is the draft in front of draft i, one of 0 .. i - 1;
 *   any other number says that the context is.
 * Without parents the drafts are a chain: draft i attends all drafts up to i
 * (with q_len = 1, decoding of single tokens).
 *   s_ij = scale * sum_d q[b][i][h][d] * K_j[d],  lse_i = log sum_j exp(s_ij)
 *   out[b][i][h][d] = sum_j exp(s_ij - lse_i) * V_j[d]
 * over the key head h / (heads / kv_heads) of the cache, K and V the rows'
 * values as above.  Rows of drafts from t on (t is taken within [0, min(q_len,
 * n)], n within [0, table_width * page_size]) keep what they hold.  A query
 * without keys (its pages are none, its tokens empty) gives 0 and lse = -inf.
 * Tokens that no draft attends may hold anything; a draft is multiplied with
 * zero for the others, so its rows have to be finite.
 *
 * Scores, sums and statistics are fp32.  Codes, queries and probabilities
 * meet in the products as fp16: codes are exact there, a query's row is held
 * times a power of two (elements below 2^-28 of the row's largest are rounded
 * in steps of 2^-39 of it), and probabilities times their value's scale and a
 * power of two that holds the row's largest of these at 2^4 at least (small
 * ones are rounded in steps of 2^-28 of it).  With more than 64 rows (drafts
 * times query heads of a key head) that scale is the largest of 16 neighbouring
 * tokens, and codes are held relative to it: elements of keys are rounded in
 * steps of 2^-24, of values in steps of 2^-31, of it.  Results are rounded once.
 * Sums run in a fixed order: equal calls give equal bits.
 *
 * q and out: [batch][q_len][heads][D] of `dtype`, strides {batch, token,
 * head} in elements, multiples of 8; lse: dense fp32 [batch][heads][q_len], or
 * NULL.  parents: int32, rows parent_stride apart (0: one tree for all).
 * Gates: those of the cache; q_len up to 256; heads a multiple of kv_heads;
 * batch * heads * q_len up to 0x7FFF0000.  A scale that is not finite and
 * positive is CONV_ERR_INVALID_VALUE.
 * ------------------------------------------------------------------------ */
typedef struct {
  int dtype; /* conv_dtype_t of q and out */
  int batch, heads, kv_heads, q_len, head_dim;
  int pages, page_size, table_width;
  float scale;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const unsigned char* scales;
  const int* block_table;
  const int* kv_lengths;
  const int* draft_lengths; /* or NULL */
  const int* parents;       /* or NULL */
  void* out;
  float* lse; /* or NULL */
  long long table_stride, parent_stride;
  long long q_stride[3], out_stride[3];           /* batch, token, head */
  long long k_cache_stride[3], v_cache_stride[3]; /* page, token, head */
} tree_attention_args_t;

/* Workspace bytes of a call on the current device: the status region and
 * partial results of rows whose keys are shared out.  Of `args` only the
 * sizes and the dtype are read. */
size_t tree_attention_workspace_size(const tree_attention_args_t* args);

conv_status_t tree_attention_fwd(const tree_attention_args_t* args, void* workspace,
                                 size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONV_GB300_DECODER_H */
