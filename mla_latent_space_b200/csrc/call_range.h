// What every launching entry point of the C ABI begins with.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

namespace mla {

// Around an entry point's host work (argument checks, tensor-map encoding,
// launches): an NVTX range, so a profiler's timeline names each call (a few
// nanoseconds when no tool is attached), and a clean slate, so that an error
// which an earlier call has returned is not taken for this one's (the launch
// checks read the last error, which stays until it is read).
struct CallRange {
  explicit CallRange(const char* name) {
    nvtxRangePushA(name);
    (void)cudaGetLastError();
  }
  ~CallRange() { nvtxRangePop(); }
  CallRange(const CallRange&) = delete;
  CallRange& operator=(const CallRange&) = delete;
};

}  // namespace mla
