// Launch parameters shared by the cross-attention entry points and kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "conv_params.h"

namespace convgb300 {

// What every cross-attention kernel knows about the call.  Strides are in
// elements and 0 along dimensions of extent 1.
struct AttnShape {
  int dtype;  // conv_dtype_t: BF16 or F16
  int batch, heads, kv_heads, q_len, kv_len, head_dim, group;  // group = heads / kv_heads
  float scale;
  const void *q, *k, *v, *out, *dout;
  void *out_w, *dq, *dk, *dv;
  float* lse;
  const int* kv_lengths;
  long long qs[3], ks[3], vs[3], os[3], dos[3], dqs[3], dks[3], dvs[3];  // batch, token, head
  // Packed mask: one bit per key, rows of mask_words 32-bit words (a multiple
  // of 4), bits past kv_len clear; null without a mask.  Row of (b, h, i):
  // b * mask_b + h * mask_h + i * mask_q, in rows (0 for broadcast dimensions).
  const uint32_t* mask_bits;
  int mask_words;
  long long mask_b, mask_h, mask_q;
  // Keys that some query of a tile of 128 attends, in rows like mask_bits':
  // row of (b, h, tile): b * any_b + h * any_h + tile * any_q.
  const uint32_t* mask_any;
  long long any_b, any_h, any_q;
};

constexpr int kAttnRows = 128;  // rows of one MMA: TMEM lanes

// Device status bits, as the convolutions' (1 producer, 2 MMA, 4 the rest).
constexpr unsigned int kAttnProducerTimeout = 1u;
constexpr unsigned int kAttnMmaTimeout = 2u;
constexpr unsigned int kAttnSoftmaxTimeout = 4u;

// Forward launch.  A row tile is up to 128 (token, head) rows of one key
// head: 128 tokens of one head, or (packed) tile_tokens tokens of all its
// query heads.
struct AttnFwdParams {  // aligned like CUtensorMap
  CUtensorMap map_q;    // {D, heads, tokens, batch}, box {64, tile_heads, tile_tokens, 1}
  CUtensorMap map_k;    // {D, kv_heads, tokens, batch}, box {64, 1, kv_box, 1}
  CUtensorMap map_v;
  CUtensorMap map_out;  // as map_q
  AttnShape a;
  int q_mul[2], k_mul[2], v_mul[2];  // {head, batch} coordinate factors: 0 for broadcasts
  int tile_heads, tile_tokens;
  int token_tiles;      // tiles along the tokens
  int row_tiles;        // row tiles of one key head
  FastDiv div_pairs, div_kv_heads, div_token_tiles;  // of pairs of row tiles, ...
  int kv_box;           // keys per tile (multiple of 16, <= 128)
  int stages;           // key/value ring
  int q_stages;
  uint32_t off_q, off_kv, off_out, off_bar;  // shared-memory offsets
  float scale_log2;     // scale * log2(e)
  // One item per CTA step: two row tiles (pairs), or ranges of the sequence
  // of (item, key tile) steps, cut evenly between the CTAs (split).
  long long items;
  long long item_rows;  // kv_heads * row_tiles: items of one batch (split)
  float* part_out;      // split: [2 * grid][128][128] unnormalised rows
  float* part_stat;     // split: [2 * grid][128][2]: maximum (log2 units), sum
  unsigned int* status;
  long long timeout_cycles;
  int fault_mode;       // test hook: 1 = every CTA with work leaves its first keys un-armed
};

size_t attn_fwd_bar_bytes();
cudaError_t launch_attn_fwd(const AttnFwdParams& p, bool split, int grid, size_t smem,
                            cudaStream_t stream);

// Backward launches (attn_bwd.cu).  The dq kernel's row tiles are as the
// forward pass's; the dk, dv kernel takes tiles of 128 tokens of one head.
constexpr int kAttnRowUnroll = 4;     // rows in flight per lane of the rows kernel
constexpr int kAttnRowBlocks = 2048;  // most blocks of each part of the rows kernel

struct AttnBwdParams {  // aligned like CUtensorMap
  CUtensorMap map_q, map_do;  // {D, heads, tokens, batch}, box by kernel
  CUtensorMap map_k, map_v;   // {D, kv_heads, tokens, batch}, box {64, 1, kv_box, 1}
  CUtensorMap map_dq;         // short keys: as map_q, boxes of 128 tokens of one head
  AttnShape a;
  int q_mul[2], do_mul[2], k_mul[2], v_mul[2];
  int tile_heads, tile_tokens, token_tiles, row_tiles;
  FastDiv div_token_tiles;
  FastDiv div_heads, div_groups, div_kv_heads, div_key_groups;  // (groups of the rows kernel)
  int kv_box;           // keys per tile (multiple of 16, <= 128)
  int q_box;            // dk, dv: tokens per box
  int q_tiles;          // tiles of 128 tokens
  int item_steps;       // dk, dv: group * q_tiles
  int last_cols;        // queries of the last tile, to a multiple of 16
  long long item_rows;
  int region, bufs;     // short keys: TMEM columns of S (and of dp), buffers; else 0
  int x_stages, y_stages;
  uint32_t off_a, off_x, off_y, off_stat, off_mask, off_bar;
  float scale_log2;
  float p_shift, p_unscale;  // fp16: p is held times 2^p_shift; 2^-p_shift
  float* stats;         // [batch][heads][q_tiles][2, in fp16 3][128]
  // fp16: the largest squares of the norms of neighbouring rows (as many as a warp
  // of the rows kernel takes), of do [batch][heads][q_tiles][...] and of v
  // [batch][kv_heads][key_groups].
  float *row_norms, *value_norms;
  int key_groups;
  int row_blocks, value_blocks;  // blocks of the rows kernel
  int row_slots;                 // its rows side by side in a warp
  bool q_whole, kv_whole;        // no item of the dq, of the dk, dv kernel is cut
  float* part_q;        // [2 * CTAs][128][128]
  float* part_kv;       // [2 * CTAs][2][128][128]
  unsigned int* status;
  long long timeout_cycles;
  int fault_mode;
};

size_t attn_bwd_bar_bytes();
cudaError_t launch_attn_rows(const AttnBwdParams& p, cudaStream_t stream);
cudaError_t launch_attn_dq(const AttnBwdParams& p, int grid, size_t smem, cudaStream_t stream);
cudaError_t launch_attn_dkv(const AttnBwdParams& p, int grid, size_t smem, cudaStream_t stream);
cudaError_t launch_attn_bwd_join(const AttnBwdParams& p, int q_ctas, int kv_ctas,
                                 long long q_blocks, long long kv_blocks, cudaStream_t stream);

// Short keys (attn_short.cu): at most 128, head_dim <= 64, no mask.
size_t attn_one_bar_bytes();
size_t attn_short_bar_bytes();
int attn_short_stages();
cudaError_t launch_attn_one(const AttnFwdParams& p, int ctas, int grid, size_t smem,
                            cudaStream_t stream);
cudaError_t launch_attn_short_bwd(const AttnBwdParams& p, int grid, size_t smem, cudaStream_t stream);

// Without keys: zeros to out (batch, q_len, heads rows) and -inf to lse.
cudaError_t launch_attn_no_keys(const AttnShape& a, cudaStream_t stream);

// Packs the byte mask into AttnShape::mask_bits and mask_any (batches x heads x queries
// rows, extents after broadcasting).
cudaError_t launch_mask_pack(const unsigned char* mask, const long long stride[4], int batches,
                             int heads, int queries, int keys, int words, uint32_t* bits,
                             uint32_t* any, cudaStream_t stream);

}  // namespace convgb300
