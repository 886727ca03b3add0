// paged.h -- what the paged-cache sources share (host side).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "inkling_paged_attn.h"

namespace ira {

cudaError_t note_cuda_error(cudaError_t e);  // host.cu: keeps the error for inkling_rel_attn_last_cuda_error

// A cache descriptor after its checks: strides of extents of 1 are 0.
struct CacheLayout {
    int64_t page_stride = 0, token_stride = 0, head_stride = 0;
    bool e4m3 = false;
};
inkling_status check_cache(const inkling_kv_cache_desc* c, CacheLayout* out);

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A named NVTX range over an entry point (a no-op when no profiler is attached).
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

}  // namespace ira
