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

// j / size for 0 <= j < 2^31 by a multiplication (Granlund and Montgomery): with 2^s >= size
// and m = floor(2^(31+s) / size) + 1, m size - 2^(31+s) <= 2^s, so j m >> (31 + s) is exact.
struct PageDivisor {
    int size = 1;
    uint32_t mul = 0, shift = 0;
    PageDivisor() = default;
    explicit PageDivisor(int64_t page_size) : size(int(page_size)) {
        uint32_t s = 0;
        while ((int64_t(1) << s) < page_size) ++s;
        mul = uint32_t((uint64_t(1) << (31 + s)) / uint64_t(page_size) + 1);
        shift = 31 + s;
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int index(int j) const { return int((uint64_t(uint32_t(j)) * mul) >> shift); }
#endif
};

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

#ifdef __CUDACC__
// Kernels of a serving step follow each other within microseconds, so each is launched while
// its predecessor runs (launch_early) and waits for that one's results before it reads or
// writes anything (wait_for_predecessor, which every block runs first); most let their own
// successor be launched in the same way (release_successor). One short decode call 3.35 ->
// 2.90 us, an append of 64 rows 1.63 -> 1.47 us of GPU time. As what they read may be written
// while they run, they use no non-coherent loads (__ldg).
__device__ __forceinline__ void wait_for_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void release_successor() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... A, class... B>
cudaError_t launch_early(void (*kernel)(A...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, B... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) (void)cudaGetLastError();  // returned here: leave nothing behind for later checks
    return e;
}
#endif

// A named NVTX range over an entry point (a no-op when no profiler is attached).
struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

}  // namespace ira
