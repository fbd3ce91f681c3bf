// Launches whose set-up overlaps the end of the kernel before them in the stream.
//
// A kernel launched by launch_overlapped may start when every CTA of the one before it in the
// stream has called launch_next() or ended. All of its threads call wait_previous() before
// their first access to global memory, which returns when that kernel has ended and its
// writes are there; so a chain of such launches sees memory as ordinary launches do. What
// another kernel may have written does not stay the same over such a kernel's life, so none
// of its loads takes the read-only path: no __ldg, no const __restrict__ (block scores read the
// means of an earlier call with them).
//
// launch_next() stands where a CTA has little left to do. At its start it lets the next
// kernel's CTAs take up whatever room the last ones leave, and those of a grid of about one
// wave then sit unevenly on the SMs until the end (scores of 8 query blocks: 37 us
// instead of 15).
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <utility>

namespace h3 {

__device__ __forceinline__ void launch_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <class... P, class... A>
cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                              unsigned cluster, cudaStream_t s, A&&... args) {
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// Clusters of `size` CTAs (2 to 8) that run at once on the current device, asked for once
// per device: with one CTA per SM a GPC's SMs need not fill up. 0 where that fails.
template <class Kernel>
int clusters_at_once(std::atomic<int> (&known)[64][9], Kernel kernel, unsigned threads, size_t smem,
                     int size) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64) {
    const int n = known[dev][size].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(size);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(size));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev < 64) known[dev][size].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace h3
