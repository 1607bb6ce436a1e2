// rc_nvtx.h -- what the entry points share on the host: the NVTX range around
// a call, and the injected launch failure of the failure-path tests.
#pragma once
#include <cstdlib>
#include <cstring>

#include <nvtx3/nvToolsExt.h>

namespace rc {

// A named NVTX range around each entry point that enqueues work, so that a
// timeline tool (Nsight Systems, or ncu --nvtx --nvtx-include) shows which
// call launched which kernels; with no tool attached the calls do nothing.
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

// RC_FAULT_INJECT=launch: every entry point that launches kernels fails after
// its argument checks and before it changes anything.
inline bool launch_fault() {
    const char* e = std::getenv("RC_FAULT_INJECT");
    return e != nullptr && std::strcmp(e, "launch") == 0;
}

}  // namespace rc
