// checks.h -- argument checks shared by the extern "C" entry points.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/muir.h"

namespace {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
#ifdef MUIR_DEBUG
// Debug builds (build.py --debug) also ask the CUDA runtime where each
// pointer lives and refuse host memory the device cannot address.
inline bool device_addressable(const void* p) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged ||
           (a.type == cudaMemoryTypeHost && a.devicePointer != nullptr);
}
inline bool ok_ptr(const void* p) { return p != nullptr && aligned16(p) && device_addressable(p); }
inline bool ok_opt(const void* p) { return p == nullptr || (aligned16(p) && device_addressable(p)); }
#else
inline bool ok_ptr(const void* p) { return p != nullptr && aligned16(p); }
inline bool ok_opt(const void* p) { return p == nullptr || aligned16(p); }
#endif
inline bool ok_dtype(muir_dtype d) { return d == MUIR_BF16 || d == MUIR_FP32; }

// The kernels use sm_100a instructions: require compute capability 10.x.
inline muir_status check_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MUIR_ERR_CUDA;
    int major = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
        return MUIR_ERR_CUDA;
    return major == 10 ? MUIR_OK : MUIR_ERR_UNSUPPORTED;
}

inline muir_status from_cuda(cudaError_t err) {
    if (err == cudaSuccess) return MUIR_OK;
    if (err == cudaErrorNotSupported) return MUIR_ERR_UNSUPPORTED;
    return MUIR_ERR_CUDA;
}

}  // namespace
