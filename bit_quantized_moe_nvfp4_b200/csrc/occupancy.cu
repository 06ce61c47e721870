// occupancy.cu -- per-device launch facts shared by the kernel launchers: the SM count and
// how many blocks of a kernel fit on one SM, each looked up once and cached.
#include <atomic>
#include <map>
#include <mutex>
#include <tuple>
#include <utility>

#include "moe.cuh"

namespace nvfp4 {

// SM count of the current device, looked up once per device (devices may differ).
int num_sms() {
  constexpr int kMaxDev = 64;
  static std::atomic<int> cached[kMaxDev];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDev) dev = 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n <= 0) {
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (n <= 0) n = kNumSMs;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

namespace {

// What a launch is asked about: a kernel on a device with this block size, shared memory and
// cluster size (0: no cluster).  Each answer is kept; how many there are is bounded by the kernels
// and the block and memory sizes that they are launched with (the norms: up to 32 widths of block
// and two memory sizes a kernel), not by the calls.
using Key = std::tuple<const void *, int, int, size_t, int>;
std::mutex g_mu;
std::map<Key, int> g_answers;
std::map<std::pair<const void *, int>, size_t> g_limits;

template <typename Query>
int answer(const Key &key, Query query) {   // with g_mu held
  const auto it = g_answers.find(key);
  if (it != g_answers.end()) return it->second;
  int n = 0;
  const cudaError_t e = query(&n);
  if (e != cudaSuccess) {
    set_last_cuda_error(e);
    return -1;
  }
  g_answers[key] = n;
  return n;
}

}  // namespace

// Blocks of kernel k that fit on one SM at once with this block size and shared memory,
// after raising the kernel's dynamic shared-memory limit to at least `smem`.  The limit is a
// per-kernel, per-device attribute that only ever grows here (a call with less memory must
// not lower it under a size another call still launches with).
int resident_blocks_fn(const void *fn, int threads, size_t smem) {
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lock(g_mu);
  const auto lim = g_limits.find({fn, dev});
  if (lim == g_limits.end() || lim->second < smem) {
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) {
      set_last_cuda_error(e);
      return -1;
    }
    g_limits[{fn, dev}] = smem;
  }
  return answer({fn, dev, threads, smem, 0}, [&](int *n) {
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, fn, threads, smem);
  });
}

int resident_clusters_fn(const void *fn, int threads, size_t smem, int size) {
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lock(g_mu);
  return answer({fn, dev, threads, smem, size}, [&](int *n) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, fn, &cfg);
  });
}

}  // namespace nvfp4
