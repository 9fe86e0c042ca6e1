// The byte mask of a cross-attention call as bits, one per key: an eighth of
// its bytes for the kernels that read it up to three times, in words that a
// row's thread takes whole; and, for every 128 queries, which keys any of them
// attends, so that the kernels skip key tiles that nobody attends and clear
// keys that must not meet a product.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_internal.h"
#include "attn_params.h"
#include "ptx.cuh"

namespace convgb300 {

namespace {

// One block packs 128 queries x 128 keys: a warp takes four rows, each lane
// four bytes of one, a ballot makes a word.  Bound by the latency of one read
// of the mask, for which all of a block's reads are in flight together.
constexpr int kWarps = 32, kRows = kAttnRows / kWarps;

__global__ void __launch_bounds__(32 * kWarps)
    mask_pack_kernel(const unsigned char* mask, long long sb, long long sh, long long sq,
                     long long sk, int heads, int queries, int keys, int words, int tiles,
                     uint32_t* bits, uint32_t* any) {
  __shared__ uint4 seen[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int across = words >> 2;
  const unsigned row = blockIdx.x / across;  // of `any`
  const int col = static_cast<int>(blockIdx.x - row * across);
  const long long bh = row / tiles;
  const int tile = static_cast<int>(row - bh * tiles);
  const long long b = bh / heads, h = bh - b * heads;
  const int i0 = tile * kAttnRows + warp;
  const int j0 = col * 128 + lane;
  const unsigned char* p = mask + b * sb + h * sh + i0 * sq + j0 * sk;
  grid_dependency_wait();
  grid_launch_dependents();
  bool on[kRows][4];
#pragma unroll
  for (int u = 0; u < kRows; ++u)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      on[u][k] = i0 + u * kWarps < queries && j0 + k * 32 < keys && p[u * kWarps * sq + k * 32 * sk] != 0;
  uint4 all = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int i = i0 + u * kWarps;
    uint4 w;
    w.x = __ballot_sync(0xFFFFFFFFu, on[u][0]);
    w.y = __ballot_sync(0xFFFFFFFFu, on[u][1]);
    w.z = __ballot_sync(0xFFFFFFFFu, on[u][2]);
    w.w = __ballot_sync(0xFFFFFFFFu, on[u][3]);
    if (lane == 0 && i < queries)
      *reinterpret_cast<uint4*>(bits + (bh * queries + i) * words + col * 4) = w;
    all.x |= w.x;
    all.y |= w.y;
    all.z |= w.z;
    all.w |= w.w;
  }
  if (lane == 0) seen[warp] = all;
  __syncthreads();
  if (warp == 0) {
    all = seen[lane];
    all.x = __reduce_or_sync(0xFFFFFFFFu, all.x);
    all.y = __reduce_or_sync(0xFFFFFFFFu, all.y);
    all.z = __reduce_or_sync(0xFFFFFFFFu, all.z);
    all.w = __reduce_or_sync(0xFFFFFFFFu, all.w);
    if (lane == 0) *reinterpret_cast<uint4*>(any + static_cast<long long>(row) * words + col * 4) = all;
  }
}

}  // namespace

cudaError_t launch_mask_pack(const unsigned char* mask, const long long stride[4], int batches,
                             int heads, int queries, int keys, int words, uint32_t* bits,
                             uint32_t* any, cudaStream_t stream) {
  const int tiles = (queries + kAttnRows - 1) / kAttnRows;
  const long long blocks = static_cast<long long>(batches) * heads * tiles * (words / 4);
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;  // 2^45 bytes of mask
  return launch_pdl(mask_pack_kernel, dim3(static_cast<unsigned>(blocks)), dim3(32 * kWarps), 0,
                    stream, mask, stride[0], stride[1], stride[2], stride[3], heads, queries, keys,
                    words, tiles, bits, any);
}

}  // namespace convgb300
