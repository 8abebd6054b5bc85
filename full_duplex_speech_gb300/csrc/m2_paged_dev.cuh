// Device helpers shared by the attention kernels over the paged e4m3 cache.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>

#include "m2_common.cuh"
#include "m2_paged.h"
#include "m2_tc.cuh"

namespace m2 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -FLT_MAX;  // a running maximum before any position: below every finite score

__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float lg2_approx(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
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
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
// 16 bytes global -> shared
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
// 4 bytes global -> shared, completion counted by cp_async_arrive
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc::smem_u32(dst)), "l"(src) : "memory");
}
// One of the barrier's expected arrivals, made when this thread's earlier
// cp.async copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}

// 16 bytes into a cluster's shared window
__device__ __forceinline__ void st_cluster_f32x4(uint32_t caddr, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(caddr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// ... and out of it
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t caddr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(caddr)
                 : "memory");
    return v;
}

// The descriptor of the copies to come, fetched ahead of the first.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

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
