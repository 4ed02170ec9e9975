// launch.h -- launches of the kernels that wait (griddepcontrol.wait) for the
// kernel before them, so that their set-up may overlap its end.
#pragma once
#include <cuda_runtime.h>

#include <cstring>

#include "mxgemm.h"

namespace mxg {

// With programmatic stream serialization, and clusters of `cluster` CTAs along
// x where it is above 1.
template <typename... Params, typename... Args>
int launch(void (*kern)(Params...), dim3 grid, int threads, int smem, int cluster, cudaStream_t stream,
           const Args &...args) {
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    cudaGetLastError();
    return MXGEMM_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
    cudaGetLastError();
    return MXGEMM_ERR_CUDA;
  }
  return MXGEMM_OK;
}

}  // namespace mxg
