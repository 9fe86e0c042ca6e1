// Launcher of one implicit-GEMM kernel instance (shared by the kernel
// translation units).
#pragma once

#include <atomic>

#include "conv_internal.h"
#include "conv_kernel.cuh"
#include "smem_limit.h"

namespace convgb300 {

template <int kKind, typename OutT, bool kGather, bool kPair = false, bool kStreamK = false>
cudaError_t launch_instance(const ConvKernelParams& p, int grid, size_t smem_bytes,
                            cudaStream_t stream) {
  static std::atomic<size_t> configured[kMaxDevices];
  cudaError_t err =
      raise_smem(conv_igemm_kernel<kKind, OutT, kGather, kPair, kStreamK>, configured, smem_bytes);
  if (err != cudaSuccess) return err;
  // Programmatic stream serialization: the kernel may be scheduled while the
  // previous kernel of the stream drains; it waits (griddepcontrol.wait)
  // before touching global memory, so stream order is preserved.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (kPair) {  // clusters of two CTAs (grid is even)
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  err = cudaLaunchKernelEx(&cfg, conv_igemm_kernel<kKind, OutT, kGather, kPair, kStreamK>, p);
  if (err != cudaSuccess) return err;
  return cudaGetLastError();
}

template <bool kGather, bool kPair = false, bool kStreamK = false>
cudaError_t launch_family(int kind, bool out_bf16, const ConvKernelParams& p, int grid,
                          size_t smem_bytes, cudaStream_t stream) {
  if (kind == kKindF8)
    return launch_instance<kKindF8, __nv_bfloat16, kGather, kPair, kStreamK>(p, grid, smem_bytes,
                                                                            stream);
  if (out_bf16)
    return launch_instance<kKindF16, __nv_bfloat16, kGather, kPair, kStreamK>(p, grid, smem_bytes,
                                                                             stream);
  return launch_instance<kKindF16, __half, kGather, kPair, kStreamK>(p, grid, smem_bytes, stream);
}

}  // namespace convgb300
