// cluster.cuh -- launching clusters of CTAs, and asking how many the GPU holds.
#pragma once
#include <cuda_runtime.h>

#include <atomic>

namespace ssm {

constexpr int kMaxCluster = 16;      // of sm_103a; past 8 a kernel has to allow it
constexpr int kPortableCluster = 8;

// `units` clusters of `size` CTAs.  It points at itself: keep it where it was made.
struct ClusterLaunch {
  cudaLaunchAttribute attr = {};
  cudaLaunchConfig_t cfg = {};
  ClusterLaunch(int64_t units, int size, int threads, size_t smem, cudaStream_t s) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(units * size));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = size > 1 ? 1 : 0;
  }
  ClusterLaunch(const ClusterLaunch&) = delete;
  ClusterLaunch& operator=(const ClusterLaunch&) = delete;
};

inline cudaError_t allow_large_clusters(const void* kernel) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

// How many clusters of 2^i CTAs of KERNEL the GPU holds at once (0 where it takes none of
// that size), asked for once per kernel.  The kernel has been allowed its shared memory.
template <auto KERNEL>
int resident_clusters(int i, int threads, size_t smem) {
  static std::atomic<int> known[5];  // 0: not asked yet; the number + 1
  int n = known[i].load(std::memory_order_relaxed);
  if (n > 0) return n - 1;
  const int size = 1 << i;
  const ClusterLaunch l(1, size, threads, smem, nullptr);
  if ((size > kPortableCluster &&
       allow_large_clusters(reinterpret_cast<const void*>(KERNEL)) != cudaSuccess) ||
      cudaOccupancyMaxActiveClusters(&n, KERNEL, &l.cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  known[i].store(n + 1, std::memory_order_relaxed);
  return n;
}

}  // namespace ssm
