// Launch with programmatic stream serialization and an optional cluster.
#pragma once
#include <utility>

#include <cuda_runtime.h>

namespace qe {

// The kernel may be scheduled while the previous kernel on the stream drains: before it touches memory that
// another kernel reads or writes, each of its threads that does waits in grid_dep_wait() for that kernel, and
// with it everything earlier, to have ended. It calls grid_dep_launch() only after that wait, so a kernel
// that begins behind it finds all work before it done.
// Its inputs may still be written while it is resident, so it reads them with ordinary loads behind the wait: no
// non-coherent load (__ldg, or what the compiler makes of a const __restrict__ pointer) is ordered behind anything.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st,
                             Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace qe
