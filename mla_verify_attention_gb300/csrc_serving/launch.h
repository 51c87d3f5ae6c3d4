// Launches that the cache operators share.
#pragma once
#include <cuda_runtime.h>

#include "mla_verify_attn.h"

namespace mla {

// A programmatic dependent of the grid before it (every kernel here waits for
// that grid before it reads anything): its launch overlaps that grid's end.
template <class P>
int launch_dependent(void (*fn)(P), const P& p, dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                     unsigned cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
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
  if (cudaLaunchKernelEx(&cfg, fn, p) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_LAUNCH;
  }
  return MLA_OK;
}

}  // namespace mla
