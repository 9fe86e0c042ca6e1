// Declarations shared by the attention entry points and their kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <cstdint>

#include "smem_limit.h"

namespace convgb300 {

// SMs of the current device, or -1.
int attn_sm_count();

// The driver's tiled tensor-map encoder, or null.
PFN_cuTensorMapEncodeTiled_v12000 tiled_map_encoder();

// Limit of every bounded wait, in SM cycles, and the test hook's fault mode.
long long wait_limit_cycles();
int wait_fault_mode();

// Launch with programmatic stream serialization: the kernel may be scheduled
// while the stream's previous kernel drains, and waits (griddepcontrol.wait)
// before it touches global memory.
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, args...);
  return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace convgb300
