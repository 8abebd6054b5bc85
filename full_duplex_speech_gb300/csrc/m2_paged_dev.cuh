// Device helpers shared by the attention kernels over the paged e4m3 cache.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>

#include "m2_common.cuh"
#include "m2_paged.h"
#include "m2_tc.cuh"
#include "m2_tile_dev.cuh"

namespace m2 {

// two e4m3 codes (the low byte first) as fp16, exactly
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}
// ... and two e5m2 codes
__device__ __forceinline__ uint32_t e5m2x2_to_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
// The power of two that takes a row's largest magnitude to [2^to, 2^(to + 1))
// (1 for a row of zeros; the power is kept at 2^126 at most).
__device__ __forceinline__ float row_power(float amax, int to) {
    const int ex = (int)(__float_as_uint(amax) >> 23) - 127;
    return amax == 0.f ? 1.f : __uint_as_float((uint32_t)(min(to - ex, 126) + 127) << 23);
}

// Pages as rows of 128 bytes, 128-byte swizzled; a box is a page, or box_rows
// rows of a longer one.
inline cudaError_t make_page_map(const uint8_t* pages, const KvCache& c, int box_rows, CUtensorMap* map) {
    tc::EncodeTiledFn enc = tc::encode_tiled();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)kKvD, (cuuint64_t)c.n_pages * c.Hkv * c.ps};
    const cuuint64_t strides[1] = {(cuuint64_t)kKvD};
    const cuuint32_t box[2] = {(cuuint32_t)kKvD, (cuuint32_t)(c.ps < box_rows ? c.ps : box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(pages), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace m2
