// The dense key/value caches of the attention layers kept bounded over a long
// session: attention of packed whole prompts with their append, the weight
// that cached positions receive, and eviction, as the launchers see them
// (m2_attn_prompt.cu, m2_attn_weights.cu, m2_kv_evict.cu; called by the C ABI
// layer after it has validated every argument). The cached decode that adds up
// weights is m2_attn.cu's.
#pragma once

#include <cuda_runtime.h>
#include <limits.h>
#include <stddef.h>
#include <stdint.h>

namespace m2 {

// Packed rows of S sessions and their caches [S, Hkv, Tmax, 128].
struct PromptArgs {
    int S, rows, Hq, Hkv, Tmax;
    bool bf16;
    const int* start;           // [S + 1] session s has rows start[s] .. start[s + 1] - 1 (device)
    const int* lens;            // [S] positions cached before (NULL: none)
    const void *q, *k_new, *v_new;
    long q_stride, kv_stride;   // elements from one row to the next
    void *k_cache, *v_cache;
    float scale;
    void* out;
    long out_stride;
    float* lse;                 // [rows, Hq] (NULL: not wanted)
    unsigned int* err;          // device error word
};
// (the append into the caches, then the attention over them)
cudaError_t launch_attn_prompt(const PromptArgs& a, cudaStream_t st);
// the attention in bf16, behind the append (m2_attn_prompt_tile.cu)
cudaError_t launch_attn_prompt_tiles(const PromptArgs& a, cudaStream_t st);

// Weights that cached positions receive from the last `window` rows of each
// session: PromptArgs' q, lse (read) and k_cache, and
struct PromptSums {
    int window;
    const float* acc;           // [S, Hkv, Tmax]
    float* acc_out;             // ... (may be acc)
};
cudaError_t launch_attn_prompt_weights(const PromptArgs& a, const PromptSums& w, cudaStream_t st);
// ... in bf16 (m2_attn_weights_tile.cu)
cudaError_t launch_attn_weights_tiles(const PromptArgs& a, const PromptSums& w, cudaStream_t st);

struct EvictArgs {
    int S, Hkv, Tmax, out_max;
    int row_bytes;              // of a key or value
    const int* lens;
    const void *k, *v;          // [S, Hkv, Tmax, 128]
    const float* acc;           // [S, Hkv, Tmax]
    int keep, recent;
    void *k_out, *v_out;        // [S, Hkv, out_max, 128] (may be k, v)
    float* acc_out;             // [S, Hkv, out_max] (may be acc)
    int* kept;                  // [S, Hkv, keep] (NULL: not wanted)
    unsigned int* err;
};
cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t st);

#ifdef __CUDACC__
struct Session {
    int row0, n, before;  // its first packed row, its rows, the positions cached before them
    bool ok;              // its positions fit the cache
};
// Session s of the call; false where its rows do not lie within the call's. A session
// also has to begin at or behind every entry of row_start ahead of its first (they all
// do where no entry is below the one ahead of it): only such sessions have rows of their
// own, one behind the other. That is the caller's to see.
__device__ __forceinline__ bool session_of(const PromptArgs& a, int s, Session* x) {
    const int b = a.start[s], e = a.start[s + 1];
    x->row0 = b;
    x->n = e - b;
    x->before = a.lens ? a.lens[s] : 0;
    x->ok = x->before >= 0 && (long)x->before + x->n <= a.Tmax;
    return b >= 0 && e >= b && e <= a.rows;
}
// Whether session s begins behind the entries ahead, found by the whole block. `ahead`:
// what load_ahead gave, so that it is on its way with the caller's other loads.
__device__ __forceinline__ int load_ahead(const PromptArgs& a, int s) {
    return (int)threadIdx.x < s ? a.start[threadIdx.x] : INT_MIN;
}
__device__ __forceinline__ bool block_begins_behind(const PromptArgs& a, int s, int ahead) {
    constexpr int kFlight = 8;  // of a thread's on their way together
    for (int i0 = threadIdx.x + blockDim.x; i0 < s; i0 += kFlight * blockDim.x) {
        int e[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) e[f] = i0 + f * (int)blockDim.x < s ? a.start[i0 + f * blockDim.x] : INT_MIN;
#pragma unroll
        for (int f = 0; f < kFlight; ++f) ahead = max(ahead, e[f]);
    }
    return __syncthreads_and(ahead <= a.start[s]);
}
#endif

}  // namespace m2
