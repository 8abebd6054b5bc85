// The paged 8-bit key/value cache of one attention layer, as its kernels see
// it, and their launchers (m2_kv_append.cu, m2_attn_paged.cu; called by the
// C ABI layer after it has validated every argument).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace m2 {

constexpr int kKvBlock = 16;     // positions that share a scale
constexpr int kKvD = 128;        // head_dim
constexpr float kE4m3Max = 448.f;
// The least block maximum a scale is made of: its reciprocal times 448, and
// the scale itself, are normal fp32 numbers.
constexpr float kKvTiny = 7.888609052210118e-31f;  // 2^-100

struct KvCache {
    int S, Hkv, ps, ps_shift, n_pages, max_pages;  // ps = 1 << ps_shift positions a page
    const int* table;                              // [S, max_pages]
    uint8_t *kp, *vp;                              // [n_pages, Hkv, ps, 128] e4m3
    float *ks, *vs;                                // [n_pages, Hkv, ps / 16]
    const float *kt, *vt;                          // [S, Hkv, 16, 128] the open block in fp32, read
    float *kto, *vto;                              // ... and written
    unsigned int* err;                             // device error word
    __host__ __device__ long capacity() const { return (long)max_pages << ps_shift; }
};

struct KvAppendArgs {
    KvCache c;
    bool bf16;
    int T, Hq;            // new positions a session, query heads (0: none to rotate)
    const int *lens, *n_new;
    const void *k, *v, *q;
    void* q_out;
    long kv_stride, q_stride, qo_stride;  // elements from one position's row to the next
    int rot, interleaved, n_pos;          // rotated dims (0: none)
    const float *cos, *sin;               // [n_pos, rot / 2]
};
cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t st);

struct PagedAttnArgs {
    KvCache c;
    bool bf16, causal;
    int T, Hq;
    const int *lens, *n_new;
    const void* q;
    void* out;
    long q_stride, out_stride;
    float scale;
};
cudaError_t launch_attn_paged(const PagedAttnArgs& a, cudaStream_t st);
// How a call is run: the CTAs that share a set of rows' positions, and a guess
// of a form's time in microseconds, from the sizes that the host knows.
struct PagedAttnPlan {
    int W;
    float us;
    bool tiles;  // the form for many rows
};
cudaError_t plan_attn_paged(const PagedAttnArgs& a, PagedAttnPlan* plan);
// the form for many rows, bf16 (m2_attn_paged_tile.cu)
cudaError_t plan_attn_paged_tiles(const PagedAttnArgs& a, PagedAttnPlan* plan);
cudaError_t launch_attn_paged_tiles(const PagedAttnArgs& a, int W, cudaStream_t st);

#ifdef __CUDACC__
// A session's positions before the call and its new ones (n_new clamped to
// [0, T]); false where they do not fit the session's row of the page table
// or the rotation's table.
__device__ __forceinline__ bool kv_extent(const KvCache& c, int s, int T, const int* lens, const int* n_new, long limit,
                                          int* before, int* fresh) {
    const int L = lens[s];
    const int n = n_new ? min(max(n_new[s], 0), T) : T;
    *before = L;
    *fresh = n;
    return L >= 0 && (long)L + n <= limit;
}
#endif

}  // namespace m2
