// Eviction from the dense caches by accumulated attention weight. For each
// session with L > keep positions and each kv head, the last `recent`
// positions stay, and of the older ones the keep - recent that received the
// most weight (ties: the lowest position); what stays moves together, in
// order, in place or into another cache:
//     k_out[j] = k[kept_j],  v_out[j] = v[kept_j],  acc_out[j] = acc[kept_j].
// Bound by HBM: the kept rows are read and written once.
//
// A (session, kv head) is a cluster of W CTAs, and CTA w moves 1 / W of every
// row's bytes, of keys and values alike. So each CTA moves its columns in
// order by itself: a batch of rows is read before any of it is written, and
// a row never moves up, so that in place nothing is written that a later batch
// still reads, with no word between the CTAs. (Rows dealt to CTAs would have
// to wait for one another.) Each CTA finds the least weight that stays by
// itself: a radix selection, three passes over the weights.
#include <math.h>

#include "m2_dense_dev.cuh"
#include "m2_tc.cuh"

namespace m2 {

namespace {

constexpr int kEvThreads = 512, kEvWarps = kEvThreads / 32;
constexpr int kEvBlock = 1024;        // positions that are looked through at a time
constexpr int kEvBins = 2048;         // 11 bits of a key
constexpr int kEvMaxW = 8;
constexpr int kEvFlight = 8;          // 16-byte pieces a thread has in flight

// Weights in order as whole numbers: NaN above all, +0 and -0 alike.
__device__ __forceinline__ uint32_t weight_key(float f) {
    if (f != f) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(f + 0.f);
    return u >> 31 ? ~u : u | 0x80000000u;
}

struct EvSmem {
    int bins[kEvBins];
    int list[kEvBlock];               // positions of the block that stay
    int warp[kEvWarps + 1];
    int pick[2];
};

// Exclusive sum of v over the block, and its total.
__device__ __forceinline__ int block_sum(int v, int* warp, int* total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int upto = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int below = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += below;
    }
    __syncthreads();
    if (lane == 31) warp[w] = upto;
    __syncthreads();
    int ahead = 0, all = 0;
#pragma unroll
    for (int i = 0; i < kEvWarps; ++i) {
        const int t = warp[i];
        if (i < w) ahead += t;
        all += t;
    }
    *total = all;
    return ahead + upto - v;
}

// grid (W, Hkv, S), a cluster of W
__global__ void __launch_bounds__(kEvThreads) kv_evict_kernel(EvictArgs a, int W) {
    __shared__ EvSmem sm;
    const int tid = threadIdx.x, w = blockIdx.x, g = blockIdx.y, s = blockIdx.z;
    pdl_wait();
    pdl_trigger();
    const int L = a.lens[s];
    if (L < 0 || L > a.Tmax) {  // the whole cluster
        if (tid == 0 && w == 0) record_error(a.err, ERR_ATTN_LENGTH);
        return;
    }
    const bool in_place = a.k == a.k_out;
    const size_t from = ((size_t)s * a.Hkv + g) * a.Tmax, to = ((size_t)s * a.Hkv + g) * a.out_max;
    const float* acc = a.acc + from;
    const bool cut = L > a.keep;
    if (!cut && in_place && a.kept == nullptr && a.acc == a.acc_out) return;
    const int old = cut ? L - a.recent : L;        // positions below it are weighed
    const int want = cut ? a.keep - a.recent : 0;  // of which so many stay
    // the key of the last that stays, and how many of that key do
    uint32_t least = 0;
    int ties = 0;
    if (cut && want > 0) {
        int left = want;
        uint32_t prefix = 0;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            const uint32_t above = pass == 0 ? 0u : ~0u << (pass == 1 ? 21 : 10);
            for (int i = tid; i < kEvBins; i += kEvThreads) sm.bins[i] = 0;
            __syncthreads();
            for (int p = tid; p < old; p += kEvThreads) {
                const uint32_t k = weight_key(acc[p]);
                if ((k & above) == prefix) atomicAdd(sm.bins + ((k >> shift) & ((1u << bits) - 1u)), 1);
            }
            __syncthreads();
            // the bin that holds the left-th largest: thread i has bins from the top, 4 i .. 4 i + 3
            int c[4], mine = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) mine += c[j] = sm.bins[kEvBins - 1 - (4 * tid + j)];
            int all;
            int ahead = block_sum(mine, sm.warp, &all);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (ahead < left && left <= ahead + c[j]) sm.pick[0] = kEvBins - 1 - (4 * tid + j), sm.pick[1] = left - ahead;
                ahead += c[j];
            }
            __syncthreads();
            prefix |= (uint32_t)sm.pick[0] << shift;
            left = sm.pick[1];
            __syncthreads();
        }
        least = prefix;
        ties = left;
    }
    // Which positions of a block stay: ascending, into sm.list; returns how many.
    // `seen` ties came before.
    auto block_list = [&](int p0, int* seen) -> int {
        int n = 0;
#pragma unroll
        for (int h = 0; h < kEvBlock / kEvThreads; ++h) {
            const int p = p0 + h * kEvThreads + tid;
            bool keep = false, tie = false;
            if (p < L) {
                if (!cut || p >= old)
                    keep = true;
                else if (want > 0) {
                    const uint32_t k = weight_key(acc[p]);
                    keep = k > least;
                    tie = k == least;
                }
            }
            int all;
            const int rank = block_sum(tie ? 1 : 0, sm.warp, &all) + *seen;
            *seen += all;
            keep = keep || (tie && rank < ties);
            const int at = block_sum(keep ? 1 : 0, sm.warp, &all);
            if (keep) sm.list[n + at] = p;
            n += all;
        }
        __syncthreads();
        return n;
    };
    const bool rows_move = cut || !in_place;
    if (rows_move) {
        // 16-byte pieces of this CTA: `per` of a row's keys, then as many of its values
        const int per = a.row_bytes / 16 / W, both = 2 * per, at_once = kEvThreads / both;
        const int lane_row = tid / both, piece = tid % both;
        const bool value = piece >= per;
        const size_t column = (size_t)(w * per + piece % per) * 16;
        const uint8_t* src = static_cast<const uint8_t*>(value ? a.v : a.k) + from * a.row_bytes + column;
        uint8_t* dst = static_cast<uint8_t*>(value ? a.v_out : a.k_out) + to * a.row_bytes + column;
        int seen = 0, done = 0;
        for (int p0 = 0; p0 < L; p0 += kEvBlock) {
            const int n = block_list(p0, &seen);
            if (!(in_place && done == p0 && n == min(kEvBlock, L - p0))) {  // (nothing left before: already there)
                for (int i0 = 0; i0 < n; i0 += kEvFlight * at_once) {
                    uint4 v[kEvFlight];
#pragma unroll
                    for (int f = 0; f < kEvFlight; ++f) {
                        const int i = i0 + f * at_once + lane_row;
                        if (i < n) v[f] = *reinterpret_cast<const uint4*>(src + (size_t)sm.list[i] * a.row_bytes);
                    }
                    if (in_place) __syncthreads();  // the batch is read before any of it is written
#pragma unroll
                    for (int f = 0; f < kEvFlight; ++f) {
                        const int i = i0 + f * at_once + lane_row;
                        if (i < n) *reinterpret_cast<uint4*>(dst + (size_t)(done + i) * a.row_bytes) = v[f];
                    }
                }
            }
            done += n;
            __syncthreads();  // the list is read
        }
    }
    // The weights and the list, by the first CTA, when no other reads the weights any more.
    if (W > 1) {
        tc::cluster_arrive();
        tc::cluster_wait();
    }
    if (w != 0) return;
    int seen = 0, done = 0;
    float* acc_out = a.acc_out + to;
    int* kept = a.kept ? a.kept + ((size_t)s * a.Hkv + g) * a.keep : nullptr;
    for (int p0 = 0; p0 < L; p0 += kEvBlock) {
        const int n = block_list(p0, &seen);
        float v[kEvBlock / kEvThreads];
#pragma unroll
        for (int h = 0; h < kEvBlock / kEvThreads; ++h)
            if (tid + h * kEvThreads < n) v[h] = acc[sm.list[tid + h * kEvThreads]];
        __syncthreads();
#pragma unroll
        for (int h = 0; h < kEvBlock / kEvThreads; ++h) {
            const int j = tid + h * kEvThreads;
            if (j >= n) continue;
            acc_out[done + j] = v[h];
            if (kept) kept[done + j] = sm.list[j];
        }
        done += n;
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t st) {
    // CTAs a (session, kv head): while the GPU's 152 SMs hold them at once, four of 512 threads an SM
    int W = 1;
    while (W < kEvMaxW && (long)a.S * a.Hkv * 2 * W <= 2 * 152) W *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(W, a.Hkv, a.S);
    cfg.blockDim = dim3(kEvThreads);
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
    return cudaLaunchKernelEx(&cfg, kv_evict_kernel, a, W);
}

}  // namespace m2
