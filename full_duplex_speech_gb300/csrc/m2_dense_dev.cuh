// Device helpers shared by the kernels over packed prompts and dense caches.
#pragma once

#include <limits.h>

#include <atomic>

#include "m2_common.cuh"
#include "m2_dense.h"
#include "m2_launch.h"
#include "m2_tile_dev.cuh"

namespace m2 {

// The tile `x` of all the sessions' tiles of `per` rows each, found by the
// whole block: session and tile of it, the last tile of a session first (it
// sees the most positions). `scratch`: blockDim / 32 + 3 ints of shared memory.
// False past the last tile. A session whose rows do not lie within the call's, or
// begin before an entry ahead of them, has no tiles. (The append records it.)
__device__ __forceinline__ bool find_tile(const PromptArgs& a, int per, int x, int* scratch, int* session, int* tile) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = (int)blockDim.x >> 5;
    int* found = scratch + warps;  // session, tile, one more than the last tile so far
    if (tid == 0) found[0] = -1;
    int base = 0;
    bool fell = false;  // an entry so far is below the one ahead of it;
    int top = 0;        // then, the largest entry ahead of these
    for (int s0 = 0; s0 < a.S; s0 += (int)blockDim.x) {
        const int s = s0 + tid, b = s < a.S ? a.start[s] : 0, e = s < a.S ? a.start[s + 1] : 0;
        // (the barrier: the scratch of the block before is read)
        const bool falls = __syncthreads_or(e < b);
        bool behind = true;  // this session begins behind the entries ahead
        if (fell || falls) {
            if (!fell) top = a.start[s0];
            fell = true;
            int largest = s < a.S ? b : INT_MIN;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int below = __shfl_up_sync(0xffffffffu, largest, off);
                if (lane >= off) largest = max(largest, below);
            }
            if (lane == 31) scratch[warp] = largest;
            const int below = __shfl_up_sync(0xffffffffu, largest, 1);
            __syncthreads();
            int ahead = lane > 0 ? max(top, below) : top;
            for (int w = 0; w < warps; ++w) {
                if (w < warp) ahead = max(ahead, scratch[w]);
                top = max(top, scratch[w]);
            }
            behind = s >= a.S || b >= ahead;
            __syncthreads();  // (the scratch is read)
        }
        const int mine = b < 0 || e < b || e > a.rows || !behind ? 0 : (e - b + per - 1) / per;
        int upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int below = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += below;
        }
        if (lane == 31) scratch[warp] = upto;
        __syncthreads();
        int ahead = base, all = base;
        for (int w = 0; w < warps; ++w) {
            const int t = scratch[w];
            if (w < warp) ahead += t;
            all += t;
        }
        const int first = ahead + upto - mine;
        if (x >= first && x < first + mine) {
            found[0] = s;
            found[1] = mine - 1 - (x - first);
        }
        base = all;
        if (x < base) break;  // the same in the whole block
    }
    __syncthreads();
    *session = found[0];
    *tile = found[1];
    return found[0] >= 0;
}

// Tiles of `per` rows that the sessions have at most, from what the host knows.
inline long most_tiles(int S, int rows, int per) {
    const long n = (long)rows / per + S;
    return n < rows ? n : rows;
}

// Lets a kernel have `bytes` of dynamic shared memory, once per device. (A key of
// its own for each kernel: the function's type is not one.)
template <int kKernel>
inline cudaError_t allow_shared(const void* kernel, int bytes) {
    static std::atomic<uint64_t> done{0};  // a bit a device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

// bf16 rows of 128 dims as [outer][middle][128]; a box is 64 dims x box_mid x
// box_out, 128-byte swizzled.
inline cudaError_t make_rows_map(const void* p, unsigned long long mid, unsigned long long out, unsigned long long mid_bytes,
                                 unsigned long long out_bytes, int box_mid, int box_out, CUtensorMap* map) {
    tc::EncodeTiledFn enc = tc::encode_tiled();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)kAttnD, mid, out};
    const cuuint64_t strides[2] = {mid_bytes, out_bytes};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_mid, (cuuint32_t)box_out};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

constexpr float kLn2 = 0.6931471805599453f;
// The tensor cores cut their sums off toward zero as they add, so that a sum of 128 products comes out too small:
// on average by 2^-23 of it where it is large (measured: 1e-7 of sums of 20 to 80, a third of that where
// they are small and terms of both signs cancel). Scores are multiplied by as much more.
constexpr float kCutOff = 1.f + 0x1p-23f;

}  // namespace m2
