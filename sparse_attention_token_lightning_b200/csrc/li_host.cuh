// Host helpers of the entry points: error messages, alignment, profiler ranges.
#pragma once

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include <nvtx3/nvToolsExt.h>

#include "li_internal.cuh"

namespace li {
namespace host {

// Records the message li_last_error_string() returns and passes the status on.
inline li_status fail(li_status st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return st;
}
inline li_status ok() {
    set_last_error("");
    return LI_OK;
}
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// NVTX range around each entry point and each stage it enqueues, for timeline tools; without a tool
// attached a push/pop pair costs a few nanoseconds. Building with -DNVTX_DISABLE compiles them out.
struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

}  // namespace host

// A 16- or 32-bit floating type's bytes (0 for other types).
inline int dtype_bytes(int32_t dtype) {
    return dtype == LI_DTYPE_BF16 || dtype == LI_DTYPE_FP16 ? 2 : dtype == LI_DTYPE_FP32 ? 4 : 0;
}

}  // namespace li
