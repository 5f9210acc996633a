// Host-side helpers shared by the C-ABI translation units (internal to the library).
#pragma once

#include <nvtx3/nvToolsExt.h>

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dsrows.h"

namespace dsrows {

// Record the message that ds_rows_last_error() returns on this thread, and return `code`.
int fail(int code, const char* fmt, ...);
int cuda_fail(cudaError_t err, const char* what);

// An NVTX range over the host-side enqueue of one stage ("dsrows.<stage>"), so
// a profiler can attribute each launch to its stage; free without a tool.
struct StageRange {
    explicit StageRange(const char* name) { nvtxRangePushA(name); }
    ~StageRange() { nvtxRangePop(); }
    StageRange(const StageRange&) = delete;
    StageRange& operator=(const StageRange&) = delete;
};

// Multiprocessors of the current device; 0 without one.
int num_sms();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// A paged cache's fields, checked for `dim`-wide rows (and, for `rows` > 0, that
// it has that many entries).
int check_cache(const ds_paged_cache_t* cache, uint32_t dim, int rows);
uint32_t page_row_bytes(uint32_t dim, int format);

}  // namespace dsrows
