// Launch parameters shared by the cross-attention entry points and kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

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
};

// Packs the byte mask into AttnShape::mask_bits (batches x heads x queries
// rows, extents after broadcasting).
cudaError_t launch_mask_pack(const unsigned char* mask, const long long stride[4], int batches,
                             int heads, int queries, int keys, int words, uint32_t* bits,
                             cudaStream_t stream);

}  // namespace convgb300
