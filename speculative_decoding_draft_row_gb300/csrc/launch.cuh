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

// Whether two ranges of memory share a byte; a null one shares none.
inline bool overlap(const void* p, int64_t bytes, const void* q, int64_t qbytes) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return p && q && a < b + (uint64_t)qbytes && b < a + (uint64_t)bytes;
}

// How many clusters of c blocks of a kernel run at once on the current device (asked of the runtime
// once a device and Class of launches, for one with `smem` bytes): clusters do not cross the GPU's
// partitions of SMs, so for large c it is well below (SMs * blocks an SM) / c (c = 16 at two blocks
// an SM: 14, not 19). 0 where none can be placed, which is kept as well; -1 where the runtime did
// not say, which is asked again the next time.
constexpr int kMaxCluster = 16;
constexpr int kPortable = 8;  // clusters up to here run on every device of the architecture
template <auto Kernel, int Class = 0>
int clusters_at_once(int dev, int c, int threads, size_t smem) {
  static std::atomic<int> count[kMaxDevices][kMaxCluster + 1];  // one more than the answer; 0: none yet
  if (dev < 0 || dev >= kMaxDevices) return -1;
  int n = count[dev][c].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = c;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int got = 0;
    if (cudaOccupancyMaxActiveClusters(&got, Kernel, &cfg) != cudaSuccess || got < 0) {
      cudaGetLastError();
      return -1;
    }
    n = got + 1;
    count[dev][c].store(n, std::memory_order_relaxed);
  }
  return n - 1;
}

// The blocks a cluster, 1 to 16, at which `units` clusters cost least: cost(c, rounds) for rounds of
// at_once(c) clusters (clusters_at_once). Sizes that fits(c) turns down or that cannot be placed are
// left out; where the runtime does not say, a portable size counts as one cluster at a time, and a
// larger one is taken only when nothing else is left. 0: no size will do.
template <class AtOnce, class Fits, class Cost>
int cheapest_cluster(int64_t units, AtOnce at_once, Fits fits, Cost cost) {
  int c = 0, unknown = 0;
  int64_t best = 0;
  for (int i = 1; i <= kMaxCluster; ++i) {
    if (!fits(i)) continue;
    int n = at_once(i);
    if (n < 0 && i > kPortable) unknown = i;
    if (n == 0 || (n < 0 && i > kPortable)) continue;
    if (n < 0) n = 1;
    const int64_t x = cost(i, (units + n - 1) / n);
    if (c == 0 || x < best) {
      best = x;
      c = i;
    }
  }
  return c ? c : unknown;
}

// The first use of a kernel on a device: allows it `max_smem` bytes of dynamic shared memory and
// clusters of up to 16 blocks there.
template <auto Kernel>
bool allow_clusters(int dev, int max_smem) {
  static std::atomic<bool> ready[kMaxDevices];
  if (dev < 0 || dev >= kMaxDevices) return false;
  if (ready[dev].load(std::memory_order_relaxed)) return true;
  if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem) !=
          cudaSuccess ||
      cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
          cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  ready[dev].store(true, std::memory_order_relaxed);
  return true;
}

// First in a kernel that launch_clusters starts, whose blocks are placed while the kernel before it in the
// stream ends: waits until that one has, and its results can be read. Calls in a row without a graph
// are 1-2 us shorter for it (1 x 4096 drawn 15.0 to 12.5 us), graph nodes 0.4. Placing the blocks
// earlier still, where the one before has only just begun, cost full launches a third (96 x 163840,
// top-k 50: 35 to 55 us): they go where room is, not where they would spread best.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launches Kernel(args) on `clusters` clusters of c blocks on the current device, `dev`.
template <auto Kernel, class Args>
tfd_status launch_clusters(const Args& args, int dev, int64_t clusters, int c, int threads,
                           size_t smem, int max_smem, cudaStream_t stream) {
  if (!allow_clusters<Kernel>(dev, max_smem)) return TFD_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * c));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, Kernel, args);
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? TFD_OK : TFD_ERR_CUDA;
}

}  // namespace tfd_host
