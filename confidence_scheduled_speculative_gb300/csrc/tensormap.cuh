// tensormap.cuh -- host side: tensor maps of the tiled copies (tensor.cuh).
#pragma once

#include <cuda.h>

#include <atomic>

#include "dspark_common.cuh"

namespace dspark {

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once.
inline EncodeFn encoder() {
    static std::atomic<EncodeFn> kept{nullptr};
    EncodeFn f = kept.load(std::memory_order_acquire);
    if (f) return f;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
        return nullptr;
    f = reinterpret_cast<EncodeFn>(p);
    kept.store(f, std::memory_order_release);
    return f;
}

inline int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// A 4-D tensor map of bfloat16 or bytes; boxes of `width` elements a row, with the
// swizzle of that many bytes or none.  (L2 promotion: a head's codes are 128 bytes beside
// the next head's, which 256 bytes fetch as well.  Two long contexts' trees then read 956
// MB, with 128 bytes 618, in the same 264 us: HBM does not bound them.)
inline bool encode(CUtensorMap *map, const void *p, int elem_bytes, int width, bool swizzle, const int64_t (&dims)[4],
            const int64_t (&strides)[3], int box1, int box3) {
    const EncodeFn f = encoder();
    if (!f) return false;
    cuuint64_t d[4], s[3];
    for (int i = 0; i < 4; ++i) d[i] = (cuuint64_t)dims[i];
    for (int i = 0; i < 3; ++i) s[i] = (cuuint64_t)(strides[i] * elem_bytes);
    const cuuint32_t box[4] = {(cuuint32_t)width, (cuuint32_t)box1, 1, (cuuint32_t)box3};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    const bool codes = elem_bytes == 1;
    return f(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void *>(p), d, s, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE
             : width * elem_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace dspark
