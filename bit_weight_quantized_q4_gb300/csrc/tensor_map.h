// tensor_map.h -- host: tensor maps of 16-bit matrices for TMA copies in the
// 128-byte swizzle, and the launch configuration of a programmatic dependent.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

namespace q4 {

// cuTensorMapEncodeTiled, resolved once (the library links the runtime only)
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeTiled encode_tiled() {
    static std::atomic<void *> cached{nullptr};
    void *f = cached.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult res;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &res) !=
                cudaSuccess ||
            res != cudaDriverEntryPointSuccess)
            return nullptr;
        cached.store(f, std::memory_order_release);
    }
    return (EncodeTiled)f;
}

// A row-major map of 16-bit values with boxes of 64 values (128 bytes) by
// box[1 ..] rows, 128-byte swizzled; dims innermost first, rank at most 5.
inline bool make_map(CUtensorMap *m, bool bf16, const void *base, int rank, const cuuint64_t *dims,
                     const cuuint32_t *box) {
    EncodeTiled enc = encode_tiled();
    if (!enc) return false;
    cuuint64_t strides[5];
    cuuint64_t s = 2;
    for (int i = 0; i + 1 < rank; ++i) {
        s *= dims[i];
        strides[i] = s;
    }
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank,
               const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline cudaLaunchConfig_t pdl_config(unsigned grid, unsigned block, size_t smem, cudaStream_t stream,
                                     cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

}  // namespace q4
