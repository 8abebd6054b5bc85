// Eviction from the dense caches by accumulated attention weight. For each
// session with L > keep positions and each kv head, the last `recent`
// positions stay, and of the older ones the keep - recent that received the
// most weight (ties: the lowest position); what stays moves together, in
// order, in place or into another cache:
//     k_out[j] = k[kept_j],  v_out[j] = v[kept_j],  acc_out[j] = acc[kept_j].
// Bound by HBM: the kept rows are read and written once.
//
// W CTAs share a (session, kv head). Each finds by itself the least weight that
// stays: a radix selection, three passes over the weights, which it keeps in shared
// memory as whole numbers in the weights' order.
//   Out of place a CTA then moves the rows of a run of positions.
//   In place the W are a cluster, and each moves 1 / W of every row's bytes, of keys
// and values alike. So it moves its columns in order by itself: a batch of rows
// is read before any of it is written, and a row never moves up, so that nothing
// is written that a later batch still reads, with no word between the CTAs. (Rows
// dealt to CTAs would have to wait for one another.) The weights move last, when
// no CTA reads them any more.
#include <math.h>

#include "m2_dense_dev.cuh"
#include "m2_tc.cuh"

namespace m2 {

namespace {

constexpr int kEvThreads = 512, kEvWarps = kEvThreads / 32;  // a position a thread is looked at at a time: a block
constexpr int kEvBins = 2048;         // 11 bits of a key
constexpr int kEvMaxW = 8;            // in place
constexpr int kEvRun = 128;           // positions a CTA is worth having for, out of place
constexpr int kEvFlight = 8;          // 16-byte pieces, or keys, a thread has in flight
constexpr int kEvStaged = 24576;      // positions whose keys fit in shared memory; longer caches read the weights again

// Weights in order as whole numbers: NaN above all, +0 and -0 alike.
__device__ __forceinline__ uint32_t weight_key(float f) {
    if (f != f) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(f + 0.f);
    return u >> 31 ? ~u : u | 0x80000000u;
}

struct EvSmem {
    int bins[kEvBins];
    int list[kEvThreads];             // positions of the block that stay
    int warp[2][kEvWarps];
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

// grid (W, Hkv, S); in place a cluster of W
__global__ void __launch_bounds__(kEvThreads) kv_evict_kernel(EvictArgs a, int W, bool in_place) {
    __shared__ EvSmem sm;
    extern __shared__ uint32_t keys[];  // of the older positions, where they fit
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, w = blockIdx.x, g = blockIdx.y, s = blockIdx.z;
    pdl_wait();
    pdl_trigger();
    const int L = a.lens[s];
    if (L < 0 || L > a.Tmax) {  // every CTA of them
        if (tid == 0 && w == 0) record_error(a.err, ERR_ATTN_LENGTH);
        return;
    }
    const bool rows_stay = a.k == a.k_out;
    const size_t from = ((size_t)s * a.Hkv + g) * a.Tmax, to = ((size_t)s * a.Hkv + g) * a.out_max;
    const float* acc = a.acc + from;
    const bool cut = L > a.keep;
    if (!cut && rows_stay && a.kept == nullptr && a.acc == a.acc_out) return;
    const int old = cut ? L - a.recent : L;        // positions below it are weighed
    const int want = cut ? a.keep - a.recent : 0;  // of which so many stay
    const bool weigh = cut && want > 0, staged = old <= kEvStaged;
    for (int i = tid; i < kEvBins; i += kEvThreads) sm.bins[i] = 0;
    __syncthreads();
    // the key of the last that stays, and how many of that key do
    uint32_t least = 0;
    int ties = 0;
    if (weigh) {
        int left = want;
        uint32_t prefix = 0;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            const uint32_t above = pass == 0 ? 0u : ~0u << (pass == 1 ? 21 : 10);
            for (int p0 = tid; p0 < old; p0 += kEvFlight * kEvThreads) {
                uint32_t k[kEvFlight];
                if (pass > 0 && staged) {
#pragma unroll
                    for (int f = 0; f < kEvFlight; ++f)
                        if (p0 + f * kEvThreads < old) k[f] = keys[p0 + f * kEvThreads];
                } else {
                    float x[kEvFlight];
#pragma unroll
                    for (int f = 0; f < kEvFlight; ++f)
                        if (p0 + f * kEvThreads < old) x[f] = acc[p0 + f * kEvThreads];
#pragma unroll
                    for (int f = 0; f < kEvFlight; ++f)
                        if (p0 + f * kEvThreads < old) {
                            k[f] = weight_key(x[f]);
                            if (staged) keys[p0 + f * kEvThreads] = k[f];
                        }
                }
#pragma unroll
                for (int f = 0; f < kEvFlight; ++f)
                    if (p0 + f * kEvThreads < old && (k[f] & above) == prefix)
                        atomicAdd(sm.bins + ((k[f] >> shift) & ((1u << bits) - 1u)), 1);
            }
            __syncthreads();
            // the bin that holds the left-th largest: thread i has bins from the top, 4 i .. 4 i + 3
            int c[4], mine = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                int* bin = sm.bins + kEvBins - 1 - (4 * tid + j);
                mine += c[j] = *bin;
                *bin = 0;  // for the next pass
            }
            int all;
            int ahead = block_sum(mine, sm.warp[0], &all);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (ahead < left && left <= ahead + c[j]) sm.pick[0] = kEvBins - 1 - (4 * tid + j), sm.pick[1] = left - ahead;
                ahead += c[j];
            }
            __syncthreads();
            prefix |= (uint32_t)sm.pick[0] << shift;
            left = sm.pick[1];
        }
        least = prefix;
        ties = left;
    }
    auto key_at = [&](int p) { return staged ? keys[p] : weight_key(acc[p]); };
    // Which positions of the block p0 .. end - 1 stay: ascending, into sm.list; returns how many.
    // `seen` ties came before.
    auto block_list = [&](int p0, int end, int* seen) -> int {
        const int p = p0 + tid;
        bool keep = false, tie = false;
        if (p < end) {
            if (!cut || p >= old) {
                keep = true;
            } else if (weigh) {
                const uint32_t k = key_at(p);
                keep = k > least;
                tie = k == least;
            }
        }
        // both counts of a warp's ahead of its own, in one round
        const unsigned below = (1u << lane) - 1u, kb = __ballot_sync(0xffffffffu, keep), tb = __ballot_sync(0xffffffffu, tie);
        __syncthreads();
        if (lane == 0) sm.warp[0][warp] = __popc(kb), sm.warp[1][warp] = __popc(tb);
        __syncthreads();
        int n = 0, ties_here = *seen, at = 0;
#pragma unroll
        for (int i = 0; i < kEvWarps; ++i) {
            const int t = sm.warp[1][i], first = min(max(ties - ties_here, 0), t), stay = sm.warp[0][i] + first;
            if (i == warp) {
                // this warp's first `first` ties stay
                const bool mine = keep || (tie && __popc(tb & below) < first);
                const unsigned all = __ballot_sync(0xffffffffu, mine);
                keep = mine;
                at = n + __popc(all & below);
            }
            n += stay;
            ties_here += t;
        }
        if (keep) sm.list[at] = p;
        *seen = ties_here;
        __syncthreads();
        return n;
    };
    // the run of positions whose rows this CTA moves, and what stays of those ahead of it
    const int q0 = in_place ? 0 : (int)((long)L * w / W), q1 = in_place ? L : (int)((long)L * (w + 1) / W);
    int seen = 0, done = 0;
    if (q0 > 0) {
        int n = 0, t = 0;
        for (int p = tid; p < q0; p += kEvThreads) {
            if (!cut || p >= old) {
                ++n;
            } else if (weigh) {
                const uint32_t k = key_at(p);
                n += k > least;
                t += k == least;
            }
        }
        block_sum(n, sm.warp[0], &done);
        block_sum(t, sm.warp[1], &seen);
        done += min(seen, ties);
    }
    float* acc_out = a.acc_out + to;
    int* kept = a.kept ? a.kept + ((size_t)s * a.Hkv + g) * a.keep : nullptr;
    if (cut || !rows_stay) {
        // 16-byte pieces of this CTA: `per` of a row's keys, then as many of its values
        const int share = in_place ? W : 1, per = a.row_bytes / 16 / share, both = 2 * per, at_once = kEvThreads / both;
        const int lane_row = tid / both, piece = tid % both;
        const bool value = piece >= per;
        const size_t column = (size_t)((in_place ? w : 0) * per + piece % per) * 16;
        const uint8_t* src = static_cast<const uint8_t*>(value ? a.v : a.k) + from * a.row_bytes + column;
        uint8_t* dst = static_cast<uint8_t*>(value ? a.v_out : a.k_out) + to * a.row_bytes + column;
        for (int p0 = q0; p0 < q1; p0 += kEvThreads) {
            const int n = block_list(p0, q1, &seen);
            float weight = 0.f;
            if (!in_place && tid < n) weight = acc[sm.list[tid]];
            if (!(rows_stay && done == p0 && n == min(kEvThreads, L - p0))) {  // (nothing left before: already there)
                for (int i0 = 0; i0 < n; i0 += kEvFlight * at_once) {
                    uint4 v[kEvFlight];
#pragma unroll
                    for (int f = 0; f < kEvFlight; ++f) {
                        const int i = i0 + f * at_once + lane_row;
                        if (i < n) v[f] = *reinterpret_cast<const uint4*>(src + (size_t)sm.list[i] * a.row_bytes);
                    }
                    if (rows_stay) __syncthreads();  // the batch is read before any of it is written
#pragma unroll
                    for (int f = 0; f < kEvFlight; ++f) {
                        const int i = i0 + f * at_once + lane_row;
                        if (i < n) *reinterpret_cast<uint4*>(dst + (size_t)(done + i) * a.row_bytes) = v[f];
                    }
                }
            }
            if (!in_place && tid < n) {
                acc_out[done + tid] = weight;
                if (kept) kept[done + tid] = sm.list[tid];
            }
            done += n;
            __syncthreads();  // the list is read
        }
    }
    if (!in_place) return;
    // The weights and the list, by the first CTA, when no other reads the weights any more.
    if (W > 1) {
        tc::cluster_arrive();
        tc::cluster_wait();
    }
    if (w != 0) return;
    seen = done = 0;
    for (int p0 = 0; p0 < L; p0 += kEvThreads) {
        const int n = block_list(p0, L, &seen);
        float v = 0.f;
        if (tid < n) v = acc[sm.list[tid]];
        __syncthreads();
        if (tid < n) {
            acc_out[done + tid] = v;
            if (kept) kept[done + tid] = sm.list[tid];
        }
        done += n;
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_kv_evict(const EvictArgs& a, cudaStream_t st) {
    const bool in_place = a.k == a.k_out || a.acc == a.acc_out;
    const int staged = a.Tmax < kEvStaged ? a.Tmax : kEvStaged;
    const cudaError_t e = allow_shared<3>((const void*)kv_evict_kernel, kEvStaged * 4);
    if (e != cudaSuccess) return e;
    // CTAs a (session, kv head): in place while the 152 SMs hold them at once, two an SM (eight heads, one
    // session of 7,500 to 4096: 46.9 us; 64 of up to 7,500 to 2048, a CTA a head: 152). Out of place one an SM
    // for a single session, since each CTA chooses by itself, which takes as long as moving 400 rows (7,500 to
    // 4096: 16.8 us with 19 a head, 20.3 with 12, 18.4 with 38). For several no more than are held at once, two
    // an SM, as long as that is four a head or more; more sessions differ more in what they have to move, which
    // more CTAs even out, up to two a head where there are many. Eight heads, to 2048, the mean of eight draws of
    // lengths up to 7,500, and in brackets all of 7,500: two sessions 18.6 (20.4) with 19, 23.4 (27.6) with 25;
    // four 24.7 (26.3) with 9, 28.1 (34.9) with 12; eight 34.4 (37.4) with 4, 36.3 (45.4) with 6; ten 38.8 (49.6)
    // with 5, 39.7 (42.6) with 3; 16 51.8 (69.2) with 3, 52.7 (58.2) with 2, to 4096 74.3 and 80.1; 64 156 (202)
    // with 2, 168 (191) with one, 158 (200) with 3.
    int W = 1;
    const long pairs = (long)a.S * a.Hkv;
    if (in_place) {
        while (W < kEvMaxW && pairs * 2 * W <= 2 * 152) W *= 2;
    } else {
        const long runs = (a.Tmax + kEvRun - 1) / kEvRun;
        long most = (a.S == 1 ? 152 : 304) / pairs;
        if (a.S > 1 && most < 4) most = 400 / pairs;
        W = (int)(most < 2 ? 2 : most);
        W = (int)(W < runs ? W : runs);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(W, a.Hkv, a.S);
    cfg.blockDim = dim3(kEvThreads);
    cfg.dynamicSmemBytes = (size_t)staged * 4;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = W;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = in_place && W > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kv_evict_kernel, a, W, in_place);
}

}  // namespace m2
