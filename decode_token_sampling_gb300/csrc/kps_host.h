// kps_host.h — host-side helpers shared by the library's translation units.
#pragma once

#include <nvtx3/nvToolsExt.h>

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

}  // namespace kps
