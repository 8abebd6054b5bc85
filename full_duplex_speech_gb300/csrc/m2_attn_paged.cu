// Grouped-query attention over the paged e4m3 cache (m2_kv_append.cu writes
// it): for session s with total = lengths[s] + n_new[s] positions cached,
// query t of the call (position lengths[s] + t) and head h (kv head g = h / R)
//     a_p = scale q . (ks_p k_p),   out = sum_p softmax(a)_p vs_p v_p
// over the positions p <= lengths[s] + t (causal), or over p < lengths[s]
// (cross attention: a cache of other states, the same for every query). ks
// and vs are the scales of the position's block of 16.
//
// One warp per (session, query, head), 32 positions at a time: each lane a
// position's score, then each lane 4 dims of the weighted values, with the
// running maximum and sum of an online softmax; fp32 throughout.
#include <cuda_fp8.h>

#include "m2_common.cuh"
#include "m2_paged.h"

namespace m2 {

namespace {

constexpr int kPaWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float e4m3_to_float(uint32_t b) {
    __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3);
    return __half2float(__half(h));
}

template <typename TA>
__global__ void __launch_bounds__(32 * kPaWarps) attn_paged_simple_kernel(PagedAttnArgs a) {
    __shared__ float sq[kPaWarps][kKvD];
    const KvCache& c = a.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, s = blockIdx.y;
    const long r = (long)blockIdx.x * kPaWarps + warp;
    const int t = (int)(r / a.Hq), h = (int)(r % a.Hq), g = h / (a.Hq / c.Hkv);
    pdl_wait();
    pdl_trigger();
    int L, n;
    const bool ok = kv_extent(c, s, a.T, a.lens, a.n_new, c.capacity(), &L, &n);
    if (!ok) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(c.err, ERR_ATTN_LENGTH);
        L = 0;
    }
    if (t >= n) return;
    const int seen = !ok ? 0 : a.causal ? L + t + 1 : L;
    const size_t qo = ((size_t)s * a.T + t) * a.q_stride + (size_t)h * kKvD + 4 * lane;
#pragma unroll
    for (int j = 0; j < 4; ++j) sq[warp][4 * lane + j] = load_act<TA>(a.q, qo + j);
    __syncwarp();
    const float sl2 = a.scale * kLog2e;
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    bool bad_page = false;
    for (int p0 = 0; p0 < seen; p0 += 32) {
        const int p = p0 + lane;
        float v = -INFINITY, vs = 0.f;
        size_t at = 0;
        if (p < seen) {
            const int page = c.table[(size_t)s * c.max_pages + (p >> c.ps_shift)];
            if (page < 0 || page >= c.n_pages) {
                bad_page = true;
            } else {
                at = ((size_t)page * c.Hkv + g) * c.ps + (p & (c.ps - 1));
                float d = 0.f;
                for (int i = 0; i < kKvD / 16; ++i) {
                    const uint4 w = *reinterpret_cast<const uint4*>(c.kp + at * kKvD + 16 * i);
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 16; ++e) d = fmaf(sq[warp][16 * i + e], e4m3_to_float((u[e / 4] >> (8 * (e % 4))) & 0xFFu), d);
                }
                v = d * (c.ks[at / kKvBlock] * sl2);
                vs = c.vs[at / kKvBlock];
            }
        }
        if (__any_sync(0xffffffffu, bad_page)) {
            bad_page = true;
            break;
        }
        float mx = v;
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m, mx), corr = ex2_approx(m - mn);
        m = mn;
        const float pr = ex2_approx(v - mn);
        l = fmaf(l, corr, pr);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] *= corr;
        for (int i = 0; i < min(32, seen - p0); ++i) {
            const float w = __shfl_sync(0xffffffffu, pr * vs, i);
            const size_t ai = __shfl_sync(0xffffffffu, at, i);
            const uint32_t u = *reinterpret_cast<const uint32_t*>(c.vp + ai * kKvD + 4 * lane);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = fmaf(w, e4m3_to_float((u >> (8 * j)) & 0xFFu), acc[j]);
        }
    }
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    if (bad_page) {
        if (lane == 0) atomicOr(c.err, ERR_KV_PAGE);
        l = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = 0.f;
    }
    const size_t o = ((size_t)s * a.T + t) * a.out_stride + (size_t)h * kKvD + 4 * lane;
#pragma unroll
    for (int j = 0; j < 4; ++j) store_act<TA>(a.out, o + j, l == 0.f ? 0.f : acc[j] / l);
}

}  // namespace

size_t attn_paged_workspace_bytes(const KvCache& c, int T, int Hq, bool bf16) {
    (void)c, (void)T, (void)Hq, (void)bf16;
    return 0;
}

cudaError_t launch_attn_paged(const PagedAttnArgs& a, cudaStream_t st) {
    const long rows = (long)a.T * a.Hq;
    const dim3 grid((unsigned)((rows + kPaWarps - 1) / kPaWarps), (unsigned)a.c.S);
    return a.bf16 ? launch_pdl(attn_paged_simple_kernel<bf16_t>, grid, dim3(32 * kPaWarps), 0, st, a)
                  : launch_pdl(attn_paged_simple_kernel<float>, grid, dim3(32 * kPaWarps), 0, st, a);
}

}  // namespace m2
