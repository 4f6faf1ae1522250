// tmap.cu -- tensor maps of the attention layer's kernels (host side).
#include "tmap.h"

namespace muir {
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &qr) != cudaSuccess ||
            qr != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

cudaError_t encode3(CUtensorMap* m, CUtensorMapDataType type, const void* base, const cuuint64_t (&dims)[3],
                    const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle) {
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const cuuint32_t es[3] = {1, 1, 1};
    auto encode = [&] {
        return enc(m, type, 3, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    if (encode() == CUDA_SUCCESS) return cudaSuccess;
    // A driver call needs a current context, which a thread that has made no runtime call
    // yet (an autograd worker's first) does not have: selecting its device makes it current.
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaSetDevice(dev);
    if (err != cudaSuccess) return err;
    return encode() == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t make_tmap_tokens(CUtensorMap* m, const void* base, int d, int heads, long long ld,
                             uint64_t tokens, int box_tokens) {
    return encode3(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base,
                   {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens},
                   {(cuuint64_t)d * 2, (cuuint64_t)ld * 2}, {64, 1, (cuuint32_t)box_tokens},
                   CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaError_t make_tmap_u8(CUtensorMap* m, const void* base, int d, int page, uint64_t blocks, int box_rows) {
    return encode3(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base,
                   {(cuuint64_t)d, (cuuint64_t)page, (cuuint64_t)blocks},
                   {(cuuint64_t)d, (cuuint64_t)page * d}, {(cuuint32_t)d, (cuuint32_t)box_rows, 1},
                   d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace muir
