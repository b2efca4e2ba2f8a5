// cache.cuh -- the paged 8-bit key/value cache as the kernels see it (cache.cu, cache_attn.cu).
#pragma once
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include "../../include/entmax_cache.h"

namespace entmax {

constexpr int PAGE = ENTMAX_PAGE_TOKENS;
constexpr int BLOCK_BYTES = PAGE * 64;   // one page's e4m3 numbers of one layer and head
constexpr int STATUS_ARG = ENTMAX_ERR_ARG;

struct CacheArgs {
    uint8_t* K;
    uint8_t* V;
    float* ks;
    float* vs;
    int* refs;
    int* table;
    int* lens;
    int n_layers, n_pages, Hkv, n_seqs, max_pages;
    int* status;
    // index of block (layer, page, head): its numbers start at BLOCK_BYTES times it, its scale is at it
    __device__ __forceinline__ size_t block(int layer, int page, int head) const {
        return ((size_t)layer * n_pages + page) * Hkv + head;
    }
};

// Host side, cache.cu: checks a cache and fills the kernels' view of it (ENTMAX_OK or an error).
int cache_args(const entmax_cache* c, CacheArgs* out);

__device__ __forceinline__ void cache_error(const CacheArgs& c) { atomicExch(c.status, STATUS_ARG); }
__host__ __device__ __forceinline__ int pages_of(int tokens) { return (int)(((unsigned)tokens + PAGE - 1) / PAGE); }

// Two kernels of one call: the first lets the second's CTAs start early (no more than their launch is early: they
// wait for its end before they read anything), which hides the second launch.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <class... P, class... A>
cudaError_t launch_next(void (*f)(P...), unsigned grid, unsigned threads, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, f, static_cast<P>(args)...);
}

// Two e4m3 numbers (low byte first) as two fp16 numbers: exact, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}

// Two fp32 values to e4m3, nearest even, x in the low byte; |x| above 448 gives 448, NaN gives NaN.
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float x, float y) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
    return r;
}

}  // namespace entmax
