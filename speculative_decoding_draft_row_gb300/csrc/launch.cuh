// launch.cuh - launches of thread-block clusters with what they need looked up once a device.
#pragma once

#include <atomic>

#include "common.cuh"

namespace tfd_host {

constexpr int kMaxDevices = 64;
constexpr int kSmemLimit = 227 * 1024;  // shared memory a block can have (sm_103a)

// SMs of the current device, looked up once a device (0 when no device answers).
inline int device_sms(int& dev) {
  static std::atomic<int> count[kMaxDevices];
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int n = count[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    n = sm_count();
    count[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Launches Kernel(args) on `clusters` clusters of c blocks. The first launch on a device allows the
// kernel `max_smem` bytes of dynamic shared memory and clusters of up to 16 blocks there.
template <auto Kernel, class Args>
tfd_status launch_clusters(const Args& args, int64_t clusters, int c, int threads, size_t smem,
                           int max_smem, cudaStream_t stream) {
  static std::atomic<bool> ready[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return TFD_ERR_CUDA;
  if (!ready[dev].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem) !=
            cudaSuccess ||
        cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
            cudaSuccess) {
      cudaGetLastError();
      return TFD_ERR_CUDA;
    }
    ready[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * c));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, Kernel, args);
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? TFD_OK : TFD_ERR_CUDA;
}

}  // namespace tfd_host
