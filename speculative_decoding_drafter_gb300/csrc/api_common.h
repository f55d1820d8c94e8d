// api_common.h -- what the C-ABI files share: status macros, alignment checks, NVTX ranges.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include <nvtx3/nvToolsExt.h>

#include "dflash2.h"

namespace df2 {

// NVTX range around an entry point: the calls show up by name in a profiler's timeline, and
// `ncu --nvtx --nvtx-include "dflash2_select/"` captures the kernels of one call.  Without a
// profiler attached the push and pop return at once (header-only NVTX, no library linked).
struct TraceRange {
    explicit TraceRange(const char *name) { nvtxRangePushA(name); }
    ~TraceRange() { nvtxRangePop(); }
    TraceRange(const TraceRange &) = delete;
    TraceRange &operator=(const TraceRange &) = delete;
};

constexpr size_t kAlign = 256;

inline size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline df2_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DF2_OK : DF2_ERR_CUDA; }

}  // namespace df2

#define DF2_TRY(expr)                        \
    do {                                     \
        const df2_status _s = (expr);        \
        if (_s != DF2_OK)                    \
            return _s;                       \
    } while (0)

#define DF2_CUDA(expr) DF2_TRY(from_cuda(expr))
