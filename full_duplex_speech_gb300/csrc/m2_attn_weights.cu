// The weight that cached positions receive from the last `window` rows of each
// session of a packed prompt (m2_attn_prompt.cu), given the rows' lse:
//     acc_out[g][p] = acc[g][p] (p < before, else 0)
//                     + sum over rows t of the window with p <= before + t, and
//                       heads h of kv head g, of e^(scale q_t,h . k_p - lse_t,h)
// Every position of a kv head belongs to one CTA, which sums its weights in a
// fixed order: no atomics, and the same sums from call to call.
#include <math.h>

#include "m2_dense_dev.cuh"
#include "m2_tc.cuh"

namespace m2 {

namespace {

// ------------------------------------------------- fp32 products of fp32 units
// A CTA takes 64 positions of one (session, kv head) and walks the window's
// rows that see any of them, whole packed rows of R heads, up to 64 at a time.
// Bound by what shared memory returns: a warp's 16-byte read of keys is 512 bytes
// for 16 products a lane (four sessions of 600 rows behind 1,000 positions, 40 / 8
// heads, fp32, all rows: 1,226 us; 32 rows a step and three CTAs an SM were no faster).
constexpr int kWfThreads = 256, kWfRows = 64, kWfPos = 64;
constexpr int kWfPitch = kAttnD + 4;
struct WfSmem {
    static constexpr int kQ = 0, kK = kQ + kWfRows * kWfPitch, kL = kK + kWfPos * kWfPitch, kSum = kL + kWfRows,
                         kFloats = kSum + 16 * kWfPos;
};

template <typename TA> __device__ __forceinline__ float4 load4(const void* p, size_t elem) {
    if constexpr (sizeof(TA) == 2) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + elem);
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                           __uint_as_float(w.y & 0xFFFF0000u));
    } else {
        return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + elem);
    }
}

// grid (position tiles x W, Hkv, S); W > 1: a cluster takes a tile, a CTA a run of its rows.
template <typename TA>
__global__ void __launch_bounds__(kWfThreads) weights_fp32_kernel(PromptArgs a, PromptSums w, int W) {
    extern __shared__ __align__(16) float wf[];
    float *sQ = wf + WfSmem::kQ, *sK = wf + WfSmem::kK, *sL = wf + WfSmem::kL, *sSum = wf + WfSmem::kSum;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int R = a.Hq / a.Hkv, per = kWfRows / R;
    const int g = blockIdx.y, s = blockIdx.z, wk = blockIdx.x % W, p0 = blockIdx.x / W * kWfPos;
    pdl_wait();
    pdl_trigger();
    Session x;
    if (!block_begins_behind(a, s, load_ahead(a, s)) || !session_of(a, s, &x)) {
        if (tid == 0) record_error(a.err, ERR_ROW_START);
        return;
    }
    if (!x.ok) {
        if (tid == 0) record_error(a.err, ERR_ATTN_LENGTH);
        return;
    }
    const int total = x.before + x.n;
    if (p0 >= total) return;
    const size_t head = ((size_t)s * a.Hkv + g) * a.Tmax;
    int first = max(max(0, x.n - w.window), p0 - x.before);  // the first row of the window that sees a position here
    // this CTA's run of the rows, in whole steps
    const int run = ((max(x.n - first, 0) + per - 1) / per + W - 1) / W * per;
    first += wk * run;
    const int end = min(first + run, x.n);
    if (first < end)
        for (int i = tid; i < kWfPos * kAttnD / 4; i += kWfThreads) {
            const int p = i / (kAttnD / 4), d = i % (kAttnD / 4) * 4;
            float4 k = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p0 + p < total) k = load4<TA>(a.k_cache, (head + p0 + p) * kAttnD + d);
            *reinterpret_cast<float4*>(sK + p * kWfPitch + d) = k;
        }
    const float sl2 = a.scale * kLog2e;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t0 = first; t0 < end; t0 += per) {
        const int rows = min(per, x.n - t0) * R;
        __syncthreads();
        for (int i = tid; i < kWfRows * kAttnD / 4; i += kWfThreads) {
            const int row = i / (kAttnD / 4), d = i % (kAttnD / 4) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < rows)
                v = load4<TA>(a.q, (size_t)(x.row0 + t0 + row / R) * a.q_stride + (size_t)(g * R + row % R) * kAttnD + d);
            *reinterpret_cast<float4*>(sQ + row * kWfPitch + d) = v;
        }
        if (tid < rows) sL[tid] = a.lse[(size_t)(x.row0 + t0 + tid / R) * a.Hq + g * R + tid % R] * kLog2e;
        __syncthreads();
        float d4[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) d4[i][j] = 0.f;
#pragma unroll 4
        for (int d = 0; d < kAttnD; d += 4) {
            float4 qv[4], kv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(sQ + (4 * ty + i) * kWfPitch + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(sK + (tx + 16 * j) * kWfPitch + d);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    d4[i][j] = fmaf(qv[i].x, kv[j].x, d4[i][j]);
                    d4[i][j] = fmaf(qv[i].y, kv[j].y, d4[i][j]);
                    d4[i][j] = fmaf(qv[i].z, kv[j].z, d4[i][j]);
                    d4[i][j] = fmaf(qv[i].w, kv[j].w, d4[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 4 * ty + i, see = row < rows ? x.before + t0 + row / R - p0 : -1;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (tx + 16 * j <= see) sum[j] += ex2_approx(fmaf(d4[i][j], sl2, -sL[row]));
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) sSum[ty * kWfPos + tx + 16 * j] = sum[j];
    __syncthreads();
    if (tid < kWfPos && p0 + tid < total) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += sSum[i * kWfPos + tid];
        if (W > 1)
            sL[tid] = t;
        else
            w.acc_out[head + p0 + tid] = (p0 + tid < x.before ? w.acc[head + p0 + tid] : 0.f) + t;
    }
    if (W == 1) return;
    tc::cluster_arrive();  // every CTA's sums are in its shared memory ...
    tc::cluster_wait();
    // ... and each adds up its share of the positions', in order
    const int p = wk * (kWfPos / W) + tid;
    if (tid < kWfPos / W && p0 + p < total) {
        float t = 0.f;
        for (int c = 0; c < W; ++c) t += ld_cluster_f32(tc::cluster_map(tc::smem_u32(sL + p), c));
        w.acc_out[head + p0 + p] = (p0 + p < x.before ? w.acc[head + p0 + p] : 0.f) + t;
    }
    tc::cluster_arrive();  // nobody leaves while its memory is read
    tc::cluster_wait();
}

template <typename TA>
cudaError_t launch_fp32(const PromptArgs& a, const PromptSums& w, cudaStream_t st) {
    constexpr int bytes = WfSmem::kFloats * 4;
    cudaError_t e = allow_shared<sizeof(TA)>((const void*)weights_fp32_kernel<TA>, bytes);
    if (e != cudaSuccess) return e;
    const long reach = a.lens ? a.Tmax : a.rows < a.Tmax ? a.rows : a.Tmax, tiles = reach > 0 ? (reach + kWfPos - 1) / kWfPos : 1;
    // CTAs that share a tile's rows, while the tiles leave SMs idle (three an SM; one session of 300, all rows, 12 / 2
    // heads: 31 us with eight, 57, 103 and 200 with four, two and one; 40 / 8 heads 51 with eight, 67 where two an SM
    // were the limit, 167 with one)
    const long window = w.window < a.rows ? w.window : a.rows, steps = window * (a.Hq / a.Hkv) / kWfRows;
    int W = 1;
    while (W < 8 && 2 * W <= steps && tiles * a.Hkv * a.S * 2 * W <= 3 * 152) W *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(W * tiles), a.Hkv, a.S);
    cfg.blockDim = dim3(kWfThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = W;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = W > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, weights_fp32_kernel<TA>, a, w, W);
}

}  // namespace

cudaError_t launch_attn_prompt_weights(const PromptArgs& a, const PromptSums& w, cudaStream_t st) {
    if (!a.bf16) return launch_fp32<float>(a, w, st);
    // (the tiles divide by the scale: lse / scale stays a normal number for every lse in earnest)
    const float size = fabsf(a.scale);
    return size >= 0x1p-40f && size <= 0x1p40f ? launch_attn_weights_tiles(a, w, st) : launch_fp32<bf16_t>(a, w, st);
}

}  // namespace m2
