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

}  // namespace kps
