// Tensor maps of row-major matrices for the TMA loads of the kernels in translation units of their own.
#pragma once

#include <cuda.h>

#include "bts_internal.cuh"

namespace bts {

// A [rows, cols] matrix of `es`-byte elements (1: bytes, 2: bf16) seen in box_rows x box_cols boxes, 128-byte swizzled;
// elements outside read as zeros.  False: the address or the row length does not suit a tensor map (16-byte
// multiples), or the driver refused it.
inline bool matrix_map(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int es, int box_cols,
                       int box_rows)
{
    typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<EncodeFn>(p) : nullptr;
    }();
    if (!fn || rows < 1 || (reinterpret_cast<uintptr_t>(base) & 15) || (cols * es) % 16) return false;
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(cols) * es};
    const cuuint32_t bx[2] = {cuuint32_t(box_cols), cuuint32_t(box_rows)};
    const cuuint32_t one[2] = {1, 1};
    return fn(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
              const_cast<void *>(base), dims, strides, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Number of SMs of the current device, looked up once per device; 0 if the runtime refused.
inline int device_sms(int *dev_out)
{
    static std::atomic<int> sms[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    *dev_out = dev;
    int n = sms[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        sms[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace bts
