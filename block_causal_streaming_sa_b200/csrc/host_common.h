// Host-side helpers shared by the translation units of libsa.so.
#pragma once

#include <string>

#include <nvtx3/nvToolsExt.h>

#include "sa_internal.h"

namespace sa {

// Text of the last error of a call without a handle (sa_last_error(NULL)).
extern thread_local std::string g_error;

// Memory type of a tensor pointer, queried on the host before anything is
// launched: device memory (of `device`, or of any device when device < 0) or
// managed memory passes; host memory (pageable or pinned) and unknown
// addresses are refused. NULL passes (presence is checked by the callers).
bool device_memory(const void* p, int device, const char* what, std::string* why);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// NVTX range over one entry point (visible in Nsight timelines; a no-op
// without a tool attached).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

}  // namespace sa
