// Launch helpers shared by the library's translation units: grid sizes, the
// per-kernel shared-memory limit, and launches that are counted for
// mpzch_launch_count.  Not part of the public ABI.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>
#include <utility>
#include <vector>

#include "mpzch.h"
#include "mpzch_internal.h"

namespace mpzch_internal {

inline cudaStream_t S(void* s) { return reinterpret_cast<cudaStream_t>(s); }

inline int sm_count() {
  static int n = 0;
  if (n == 0) {
    int dev = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (n <= 0) n = 148;
  }
  return n;
}

// Grid for a grid-stride kernel: enough blocks for `work` threads, at most
// `per_sm` resident blocks on every SM.
inline unsigned grid_for(int64_t work_threads, int block, int per_sm = 8) {
  int64_t g = (work_threads + block - 1) / block;
  const int64_t cap = (int64_t)sm_count() * per_sm;
  if (g > cap) g = cap;
  if (g < 1) g = 1;
  return (unsigned)g;
}

// Blocks of `kern` (with `block` threads, `smem` dynamic bytes) resident on
// one SM, looked up once per kernel and device; at least 1.
inline int resident_blocks(const void* kern, int block, size_t smem) {
  struct Entry {
    const void* kern;
    int device, block;
    size_t smem;
    int blocks;
  };
  static std::mutex mu;
  static std::vector<Entry> done;
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lock(mu);
  for (const Entry& e : done)
    if (e.kern == kern && e.device == dev && e.block == block && e.smem == smem) return e.blocks;
  int b = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, kern, block, smem) != cudaSuccess) {
    cudaGetLastError();
    b = 1;
  }
  if (b < 1) b = 1;
  done.push_back({kern, dev, block, smem, b});
  return b;
}

inline int after_launch() {
  count_launch();
  return cudaGetLastError() == cudaSuccess ? MPZCH_OK : MPZCH_ECUDA;
}

// Raises a kernel's dynamic shared-memory limit to `bytes` on the current
// device, once per (kernel, device) and size: the attribute belongs to the
// kernel function on one device, so kernels sharing a signature (template
// instances) and devices are tracked separately.
inline int allow_dynamic_smem(const void* kern, size_t bytes) {
  struct Entry {
    const void* kern;
    int device;
    size_t bytes;
  };
  static std::mutex mu;
  static std::vector<Entry> done;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MPZCH_ECUDA;
  std::lock_guard<std::mutex> lock(mu);
  for (const Entry& e : done)
    if (e.kern == kern && e.device == dev && e.bytes >= bytes) return MPZCH_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) !=
      cudaSuccess) {
    cudaGetLastError();
    return MPZCH_ECUDA;
  }
  done.push_back({kern, dev, bytes});
  return MPZCH_OK;
}

// Launches a kernel; with `pdl` it may start while the previous kernel of the
// stream drains (programmatic dependent launch: every kernel waits for its
// predecessors with griddepcontrol.wait before touching memory).
template <typename... KArgs, typename... Args>
int launch(void (*kern)(KArgs...), dim3 grid, unsigned block, cudaStream_t st, bool pdl,
           Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
  count_launch();
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MPZCH_ECUDA;
  }
  return MPZCH_OK;
}

template <typename... KArgs, typename... Args>
int launch_smem(void (*kern)(KArgs...), dim3 grid, unsigned block, size_t smem,
                cudaStream_t st, bool pdl, Args&&... args) {
  int rc = allow_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
  if (rc) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
  count_launch();
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MPZCH_ECUDA;
  }
  return MPZCH_OK;
}

}  // namespace mpzch_internal
