// NVTX ranges over the entry points.
#pragma once

#ifndef FLCE_NO_NVTX
#include <nvtx3/nvToolsExt.h>
#endif

namespace flce {

// An NVTX range over one entry point, so that profilers (ncu --nvtx, nsys)
// can select a pass by name. Without an attached tool the calls cost a few
// nanoseconds. Builds with FLCE_NO_NVTX leave them out.
struct NvtxRange {
  explicit NvtxRange(const char* name) {
#ifndef FLCE_NO_NVTX
    nvtxRangePushA(name);
#else
    (void)name;
#endif
  }
  ~NvtxRange() {
#ifndef FLCE_NO_NVTX
    nvtxRangePop();
#endif
  }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

}  // namespace flce
