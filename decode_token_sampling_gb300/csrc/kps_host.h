// kps_host.h — host-side helpers shared by the library's translation units.
#pragma once

#include "kps.h"

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <atomic>
#include <cstdint>

namespace kps {

// An NVTX range around each public call: it names the call in a profiler's timeline
// (Nsight Systems, ncu's NVTX filters) and costs a pointer check when no tool is attached.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

// What the calling thread's last sampling call launched: the kernel (1 cluster, 2 row), how many
// kernels, and the CTAs per cluster; zeros before the first.
struct LastCall {
  int kernel, launches, cluster;
};
LastCall& last_call();

// The current device's SMs, or 0.
static inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) return n;
  (void)cudaGetLastError();
  return 0;
}

// Lets a kernel take as much dynamic shared memory as a block can have: the same for every call,
// so that calls side by side do not undo each other's; once for each device.
constexpr int kMaxDynamic = 224 * 1024;
constexpr int kMaxDevices = 64;
template <class Kernel>
static inline bool allow_shared(Kernel* kernel, std::atomic<bool>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    (void)cudaGetLastError();
    return false;
  }
  if (done[dev].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamic) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  done[dev].store(true, std::memory_order_release);
  return true;
}

// A gradient buffer of its own for [N, V] logits: rows of at least V elements, sharing no byte with the logits' rows.
static inline kps_status check_grad(const void* logits, int64_t N, int64_t V, int64_t ld, kps_dtype dt, const void* grad, int64_t ld_grad) {
  const uintptr_t size = dt == KPS_BF16 ? 2 : 4;
  const uintptr_t a = reinterpret_cast<uintptr_t>(logits), b = reinterpret_cast<uintptr_t>(grad);
  if (!grad || b % size != 0 || (N > 1 && ld_grad < V)) return KPS_ERR_INVALID_ARG;
  const uintptr_t an = ((N - 1) * ld + V) * size, bn = ((N - 1) * ld_grad + V) * size;
  return a < b + bn && b < a + an ? KPS_ERR_INVALID_ARG : KPS_OK;
}

}  // namespace kps
