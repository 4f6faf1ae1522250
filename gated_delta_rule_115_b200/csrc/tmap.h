// tmap.h -- tensor maps of the attention layer's kernels (host side).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace muir {

// Token-major 16-bit tensor [tokens][heads][d] whose tokens lie `ld` elements apart:
// boxes of 64 channels x 1 head x `box_tokens` tokens, 128-byte swizzle.  Coordinates
// (channel, head, token); what lies past the last token reads as zero.
cudaError_t make_tmap_tokens(CUtensorMap* m, const void* base, int d, int heads, long long ld,
                             uint64_t tokens, int box_tokens);

// Cache pages of 8-bit codes [blocks][page][d]: boxes of one block's `box_rows` rows of d
// codes, swizzled over the row's d bytes (64 or 128).  Coordinates (channel, row, block).
cudaError_t make_tmap_u8(CUtensorMap* m, const void* base, int d, int page, uint64_t blocks,
                         int box_rows);

// Allows kernel `f` `bytes` of dynamic shared memory on the current device, once for each
// device (`done`: the caller's static, one bit a device; devices past 63 are set every time).
template <class F>
cudaError_t allow_smem(F* f, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    err = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

// Launches `f`, with `early` so that its blocks may start while the kernel before it in the
// stream (one of this library's own, launched in the same call) still runs: what they do
// before grid_wait() must not touch what that kernel writes.
template <class F, class... A>
cudaError_t launch_early(F* f, bool early, dim3 grid, int threads, int smem, cudaStream_t st, const A&... args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, f, args...);
}

#ifdef __CUDACC__
// The kernel before (of launch_early) has finished and its writes are visible.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Blocks of the kernel after may start.
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

}  // namespace muir
