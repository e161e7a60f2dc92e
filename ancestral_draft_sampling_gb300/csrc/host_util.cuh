// host_util.cuh -- small host-side helpers shared by the entry points: the
// number of multiprocessors, pointer checks and the tensor-map encoder.
#pragma once

#include <atomic>
#include <cstdint>
#include <cstdlib>
#include <mutex>
#include <utility>

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "../../include/dspark.h"

namespace dspark {

inline bool aligned_to(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// Streaming multiprocessors of the current device (cached per device).
inline int sm_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  int n = cache[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) !=
            cudaSuccess ||
        n <= 0)
      n = 1;
    cache[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// DSPARK_TEST_STALL_WAIT=1 (tests of the failure path only): the tensor-core
// kernels' product issuers wait, with a limit of kStallPolls polls, for a
// barrier phase that nothing completes and that guards no copy (the draft
// block's: the second phase of the barrier of u, once u is ready), so that the
// wait runs out, the kernel records kDevErrTimeout and takes its abort path.
constexpr uint32_t kStallPolls = 1u << 12;
// =2: the second stream's warps of the attention over items with few rows come late to
// every unit's end, by kLateNs.  No wait runs out.
// =3: one of the selection's warps that load queries has given up; the others' waits
// run out.
constexpr int kStallWait = 1, kStallLate = 2, kStallAlone = 3;
constexpr unsigned kLateNs = 50000;
inline int stall_requested() {
  const char* env = std::getenv("DSPARK_TEST_STALL_WAIT");
  return env != nullptr && env[0] >= '1' && env[0] <= '9' ? env[0] - '0' : 0;
}
inline bool stall_first_wait_requested() { return stall_requested() == kStallWait; }

inline dspark_status from_cuda(cudaError_t e) {
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

// Launches a kernel that waits for the kernels before it on the device
// (griddepcontrol.wait before it touches global memory), so that its blocks
// may be set up while the last of those still runs.
template <typename... Params, typename... Args>
inline cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                                 cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// The driver's tensor-map encoder, or null where the driver has none.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

}  // namespace dspark
