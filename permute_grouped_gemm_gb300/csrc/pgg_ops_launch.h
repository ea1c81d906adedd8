// What a launch needs of the device, asked or set once per device and kept, as
// device attributes are (the calls cost microseconds): how many clusters of a
// kernel fit, and how much dynamic shared memory it may take. That limit is the
// kernel's, not a launch's: it is set to the most that any call takes, so that
// calls of several threads do not lower it for each other.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

namespace pgg {

struct SmemLimit {
  std::atomic<int> set[64] = {};  // by device
};

// Lets `kern` take up to `most` bytes of dynamic shared memory (one value per kernel).
template <typename Kern>
cudaError_t allow_smem(SmemLimit* limit, Kern kern, int most) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (limit->set[dev].load()) return cudaSuccess;
  err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (err == cudaSuccess) limit->set[dev].store(1);
  return err;
}

struct ClusterLimits {
  std::atomic<int> fit[64][4] = {};  // [device][log2 of the cluster size], 0 = not asked yet
};

template <typename Kern>
cudaError_t clusters_that_fit(ClusterLimits* limits, Kern kern, int threads, int smem,
                              int cluster, int num_sms, int* clusters) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::atomic<int>& kept =
      limits->fit[dev][cluster == 1 ? 0 : cluster == 2 ? 1 : cluster == 4 ? 2 : 3];
  *clusters = kept.load();
  if (*clusters > 0) return cudaSuccess;
  err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms / cluster * cluster), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaOccupancyMaxActiveClusters(clusters, kern, &cfg);
  if (err != cudaSuccess) return err;
  if (*clusters < 1) return cudaErrorInvalidConfiguration;
  kept.store(*clusters);
  return cudaSuccess;
}

}  // namespace pgg
