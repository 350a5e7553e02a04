// Launches of the decoder operators' kernels that take several arguments.
#pragma once

#include "dq_launch.cuh"

namespace dq_host {

// A programmatic dependent launch (launch_programmatic) in clusters of `cluster`
// CTAs along x (1: none, or those that the kernel names itself).
template <typename Kernel, typename... Args>
dq_status launch_dependent(Kernel kernel, dim3 grid, int block, size_t smem, int cluster, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return DQ_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace dq_host
