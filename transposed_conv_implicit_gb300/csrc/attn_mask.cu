// The byte mask of a cross-attention call as bits, one per key: an eighth of
// its bytes for the kernels that read it up to three times, and in words that
// a row's thread takes whole.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_internal.h"
#include "attn_params.h"
#include "ptx.cuh"

namespace convgb300 {

namespace {

// One word (32 keys) per warp step: each lane reads one byte and the ballot is
// the word.  Bound by the mask's bytes.
__global__ void __launch_bounds__(256)
    mask_pack_kernel(const unsigned char* mask, long long sb, long long sh, long long sq,
                     long long sk, int heads, int queries, int keys, int words, long long total,
                     uint32_t* bits) {
  const int lane = threadIdx.x & 31;
  const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
  grid_dependency_wait();
  for (long long row = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
       row < total; row += warps) {
    const long long bh = row / queries;
    const long long i = row - bh * queries;
    const long long b = bh / heads, h = bh - b * heads;
    const unsigned char* p = mask + b * sb + h * sh + i * sq;
    for (int w0 = 0; w0 < words; w0 += 4) {
      uint32_t word[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = (w0 + u) * 32 + lane;
        const bool on = j < keys && p[j * sk] != 0;
        word[u] = __ballot_sync(0xFFFFFFFFu, on);
      }
      if (lane == 0)
        *reinterpret_cast<uint4*>(bits + row * words + w0) =
            make_uint4(word[0], word[1], word[2], word[3]);
    }
  }
  grid_launch_dependents();
}

}  // namespace

cudaError_t launch_mask_pack(const unsigned char* mask, const long long stride[4], int batches,
                             int heads, int queries, int keys, int words, uint32_t* bits,
                             cudaStream_t stream) {
  const long long total = static_cast<long long>(batches) * heads * queries;
  const int sms = attn_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int grid = static_cast<int>(std::min<long long>((total + 7) / 8, sms * 8ll));
  if (grid == 0) return cudaSuccess;
  return launch_pdl(mask_pack_kernel, dim3(grid), dim3(256), 0, stream, mask, stride[0], stride[1],
                    stride[2], stride[3], heads, queries, keys, words, total, bits);
}

}  // namespace convgb300
