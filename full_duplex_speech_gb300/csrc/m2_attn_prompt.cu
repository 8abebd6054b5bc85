// Attention of packed whole prompts over the dense caches: the rows of several
// sessions, of different lengths, one behind the other, appended to their
// caches and each attending over its session's positions up to its own.
//     a_p = scale q_t,h . k_p  (p <= before + t),  out_t,h = sum_p softmax(a)_p v_p,
//     lse_t,h = ln sum_p e^(a_p)
// with kv head g = h / R, R = Hq / Hkv. A kv head's rows are its (row, head)
// pairs, t R + r.
#include <limits.h>
#include <math.h>

#include "m2_dense_dev.cuh"
#include "m2_tc.cuh"

namespace m2 {

namespace {

// ---------------------------------------------------------------- the append
// A warp a row: its keys and values, 16 bytes a lane at a time, to position
// before + t of its session's caches. The session is the one that ends at the first
// entry of row_start past the row: those ahead of that are at or before the row, and
// sessions behind it begin before it. It is left out where an entry ahead of its first
// is larger. (Every entry up to it is looked at: a search would take fewer looks, and
// see nothing of that. 64 sessions: 25 us with the tiles either way; 65,535 of one row:
// 2.7 ms, 1.8 with a search.)
constexpr int kApThreads = 256;
__device__ __forceinline__ void append_row(const PromptArgs& a, int row_bytes, int row, int lane) {
    const int pieces = a.Hkv * row_bytes / 16, per = row_bytes / 16;  // of keys, of a head
    const size_t from = (size_t)row * a.kv_stride * (row_bytes / kAttnD);
    const uint4* ks = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.k_new) + from);
    const uint4* vs = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.v_new) + from);
    // (the first of them are under way while the session is looked up)
    constexpr int kFlight = 4;
    uint4 k[kFlight], v[kFlight];
    auto load = [&](int i0) {
#pragma unroll
        for (int f = 0; f < kFlight; ++f)
            if (i0 + 32 * f + lane < pieces) k[f] = __ldg(ks + i0 + 32 * f + lane), v[f] = __ldg(vs + i0 + 32 * f + lane);
    };
    load(0);
    int lo = -1, top = INT_MIN;  // the session; this lane's largest of the entries ahead of its last
    int row0 = 0, end = 0, before = 0;
    {  // the first 32 with all there is of them, so that nothing follows where there are no more
        const int b = lane < a.S ? a.start[lane] : INT_MIN, e = lane < a.S ? a.start[lane + 1] : INT_MIN;
        const int len = lane < a.S && a.lens ? a.lens[lane] : 0;
        const unsigned past = __ballot_sync(0xffffffffu, e > row);
        const int at = past ? __ffs(past) - 1 : 32;
        if (lane <= at) top = b;
        if (lane < at) top = max(top, e);
        if (past) {
            lo = at, row0 = __shfl_sync(0xffffffffu, b, at), end = __shfl_sync(0xffffffffu, e, at);
            before = __shfl_sync(0xffffffffu, len, at);
        }
    }
    constexpr int kEach = 8;  // then their last entries alone
    for (int s0 = 32; lo < 0 && s0 < a.S; s0 += 32 * kEach) {
        int e[kEach], largest = INT_MIN;
#pragma unroll
        for (int f = 0; f < kEach; ++f) {
            const int s = s0 + 32 * f + lane;
            e[f] = s < a.S ? a.start[s + 1] : INT_MIN;
            largest = max(largest, e[f]);
        }
        if (!__any_sync(0xffffffffu, largest > row)) {
            top = max(top, largest);
            continue;
        }
#pragma unroll
        for (int f = 0; f < kEach; ++f) {
            if (lo >= 0) continue;  // (the same in the whole warp)
            const unsigned past = __ballot_sync(0xffffffffu, e[f] > row);
            const int at = past ? __ffs(past) - 1 : 32;
            if (lane < at) top = max(top, e[f]);
            if (past) lo = s0 + 32 * f + at;
        }
        row0 = a.start[lo], end = a.start[lo + 1], before = a.lens ? a.lens[lo] : 0;
    }
    // (rows ahead of the first session's or behind the last's are nobody's)
    if (lo < 0 || row < row0 || row0 < 0 || end > a.rows || row0 < __reduce_max_sync(0xffffffffu, top)) return;
    if (before < 0 || (long)before + (end - row0) > a.Tmax) return;
    const size_t to = ((size_t)lo * a.Hkv * a.Tmax + before + (row - row0)) * row_bytes;
    for (int i0 = 0; i0 < pieces; i0 += 32 * kFlight) {
        if (i0 > 0) load(i0);
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int i = i0 + 32 * f + lane;
            if (i >= pieces) continue;
            const size_t at = to + (size_t)(i / per) * a.Tmax * row_bytes + (size_t)(i % per) * 16;
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.k_cache) + at) = k[f];
            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.v_cache) + at) = v[f];
        }
    }
}

__global__ void __launch_bounds__(kApThreads) prompt_append_kernel(PromptArgs a, int row_bytes) {
    pdl_wait();
    pdl_trigger();
    const long thread = blockIdx.x * (long)kApThreads + threadIdx.x;
    const int row = (int)(thread >> 5);
    if (row < a.rows) append_row(a, row_bytes, row, threadIdx.x & 31);
    // What is wrong with any session is recorded here, also where it has no rows or lies behind
    // the last one that has. (A session that begins before an entry ahead of it lies behind one
    // whose own entries decrease.)
    for (long s = thread; s < a.S; s += (long)gridDim.x * kApThreads) {
        Session x;
        if (!session_of(a, (int)s, &x))
            record_error(a.err, ERR_ROW_START);
        else if (!x.ok)
            record_error(a.err, ERR_ATTN_LENGTH);
    }
}

cudaError_t launch_append(const PromptArgs& a, cudaStream_t st) {
    const unsigned blocks = a.rows > 0 ? (unsigned)(((long)a.rows * 32 + kApThreads - 1) / kApThreads) : 1u;
    return launch_pdl(prompt_append_kernel, dim3(blocks), dim3(kApThreads), 0, st, a, kAttnD * (a.bf16 ? 2 : 4));
}

// ------------------------------------------------------ fp32, on the CUDA cores
// A CTA takes up to 32 rows of one (session, kv head), whole packed rows of R
// heads, and walks the positions 64 at a time with an online softmax: a thread 4
// rows x 4 positions of the scores, then 4 rows x 8 dims of the output, in paired
// fp32 arithmetic. Bound by those products and their reads of shared memory; the
// copies of a chunk's values run under its scores, those of the next keys under
// its values. Two CTAs an SM, so that one's products cover the other's barriers
// (five prompts of up to 301, 12 / 2 heads: 55 us; with 64 rows, 256 threads, one
// CTA an SM and no copies ahead 70). As mma.sync products of split operands, 64 rows
// a CTA (tf32 in two terms, three products, or bf16 in three, six: the same time), four
// prompts of 600 behind 1,000 took 1,223 us where this takes 1,696, but these 66.
constexpr int kPfThreads = 128, kPfRows = 32, kPfPos = 64;
constexpr int kPfPitch = kAttnD + 4;  // floats: a column of 16-byte pieces meets all banks
struct PfSmem {
    static constexpr int kQ = 0, kK = kQ + kPfRows * kPfPitch, kV = kK + kPfPos * kPfPitch, kP = kV + kPfPos * kAttnD,
                         kBad = kP + kPfRows * (kPfPos + 4), kFind = kBad + 4, kFloats = kFind + kPfThreads / 32 + 4;
    static_assert(2 * (kFloats * 4 + 1024) <= 228 * 1024, "two CTAs an SM");
    // W > 1, after the walk: the rows' sums over the keys, their (m, l) over the weights
    static constexpr int kO = kK, kMl = kP;
};

// grid W x Hkv x tiles; W > 1: a cluster's CTAs share a tile's positions and merge through
// distributed shared memory.
__global__ void __launch_bounds__(kPfThreads, 2) prompt_f32_kernel(PromptArgs a, int W) {
    extern __shared__ __align__(16) float pf[];
    float *sQ = pf + PfSmem::kQ, *sK = pf + PfSmem::kK, *sV = pf + PfSmem::kV, *sP = pf + PfSmem::kP;
    // values that are not finite, a bit a position; for the chunks in turn (one's are still read when the next begins)
    unsigned* sBads = reinterpret_cast<unsigned*>(pf + PfSmem::kBad);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int R = a.Hq / a.Hkv, per = kPfRows / R;
    const int wk = blockIdx.x % W, block = blockIdx.x / W, g = block % a.Hkv;
    const float* q = static_cast<const float*>(a.q);
    float* out = static_cast<float*>(a.out);
    pdl_wait();
    pdl_trigger();
    int s, tile;
    if (!find_tile(a, per, block / a.Hkv, reinterpret_cast<int*>(pf + PfSmem::kFind), &s, &tile)) return;
    Session x;
    session_of(a, s, &x);
    const int t0 = tile * per, rows = min(per, x.n - t0) * R;
    auto packed = [&](int row) { return (size_t)(x.row0 + t0 + row / R); };
    auto column = [&](int row) { return (size_t)(g * R + row % R) * kAttnD; };
    if (!x.ok) {  // the whole cluster
        if (wk > 0) return;
        for (int i = tid; i < rows * kAttnD; i += kPfThreads)
            out[packed(i / kAttnD) * a.out_stride + column(i / kAttnD) + i % kAttnD] = 0.f;
        if (a.lse)
            for (int row = tid; row < rows; row += kPfThreads) a.lse[packed(row) * a.Hq + g * R + row % R] = -INFINITY;
        return;
    }
    const int all = x.before + t0 + 1;           // positions that every row sees
    const int total = x.before + t0 + rows / R;  // ... and that the last one does
    // this CTA's run of positions
    const int run = ((total + kPfPos - 1) / kPfPos + W - 1) / W * kPfPos, begin = wk * run, end = min(begin + run, total);
    const size_t cache0 = ((size_t)s * a.Hkv + g) * a.Tmax * kAttnD;
    // a warp copies four positions at a time, a lane 16 bytes of each
    auto copy = [&](const void* cache, int p0, float* to, int pitch) {
        const float* from = static_cast<const float*>(cache) + cache0 + (size_t)p0 * kAttnD + (tid & 31) * 4;
        for (int p = tid >> 5; p < kPfPos && p0 + p < total; p += kPfThreads / 32)
            cp_async16(to + p * pitch + (tid & 31) * 4, from + (size_t)p * kAttnD);
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = tid; i < kPfRows * kAttnD / 4; i += kPfThreads) {
        const int row = i / (kAttnD / 4), d = i % (kAttnD / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < rows) v = *reinterpret_cast<const float4*>(q + packed(row) * a.q_stride + column(row) + d);
        *reinterpret_cast<float4*>(sQ + row * kPfPitch + d) = v;
    }
    if (begin < end) copy(a.k_cache, begin, sK, kPfPitch);
    const float sl2 = a.scale * kLog2e;
    int lim[4];  // the last position that this thread's rows see
    float m[4], l[4];
    float2 o[4][4];
    bool bad[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 4 * ty + i;
        lim[i] = row < rows ? x.before + t0 + row / R : -1;
        m[i] = kNone, l[i] = 0.f, bad[i] = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = make_float2(0.f, 0.f);
    }
    for (int p0 = begin; p0 < end; p0 += kPfPos) {
        const bool cut = p0 + kPfPos > all;
        unsigned* sBad = sBads + 2 * (p0 / kPfPos & 1);
        asm volatile("cp.async.wait_all;" ::: "memory");  // the keys
        if (tid < 2) sBad[tid] = 0u;
        __syncthreads();  // (and the values before are read)
        copy(a.v_cache, p0, sV, kAttnD);
        float2 z[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) z[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int d = 0; d < kAttnD; d += 4) {
            float4 qv[4], kv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(sQ + (4 * ty + i) * kPfPitch + d);
#pragma unroll
            for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4*>(sK + (tx + 16 * j) * kPfPitch + d);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    z[i][j] = fma2(make_float2(qv[i].x, qv[i].y), make_float2(kv[j].x, kv[j].y), z[i][j]);
                    z[i][j] = fma2(make_float2(qv[i].z, qv[i].w), make_float2(kv[j].z, kv[j].w), z[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int see = lim[i] - p0;
            float w[4], top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // (keys behind the last are whatever was there)
                w[j] = tx + 16 * j <= see ? (z[i][j].x + z[i][j].y) * sl2 : -INFINITY;
                top = fmaxf(top, w[j]);
            }
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float now = fmaxf(m[i], top), f = ex2_approx(m[i] - now);
            m[i] = now;
            l[i] *= f;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = mul2(o[i][e], make_float2(f, f));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = ex2_approx(w[j] - now);
                l[i] += p;
                sP[(4 * ty + i) * (kPfPos + 4) + tx + 16 * j] = p;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");  // the values
        if (cut) {
            // A value that is not finite must not reach the rows that do not see it: it counts as 0 here, and
            // the rows that see it read NaN. Positions behind the last count as 0 too. (Each thread looks
            // at what it copied.)
            for (int p = tid >> 5; p < kPfPos; p += kPfThreads / 32) {
                float4* at = reinterpret_cast<float4*>(sV + p * kAttnD + (tid & 31) * 4);
                const float4 v = *at;
                const bool there = p0 + p < total;
                const bool off = !(fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY && fabsf(v.z) < INFINITY && fabsf(v.w) < INFINITY);
                if (there && off) atomicOr(sBad + (p >> 5), 1u << (p & 31));
                if (!there || off) *at = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        __syncthreads();  // the values, the weights; the keys are read
        if (p0 + kPfPos < end) copy(a.k_cache, p0 + kPfPos, sK, kPfPitch);
        if (cut && (sBad[0] | sBad[1])) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int see = lim[i] - p0;
                if (see >= 0)
                    bad[i] |= (sBad[0] & (see >= 31 ? ~0u : (2u << see) - 1u)) != 0u ||
                              (see >= 32 && (sBad[1] & (see >= 63 ? ~0u : (2u << (see - 32)) - 1u)) != 0u);
            }
        }
#pragma unroll 2
        for (int p = 0; p < kPfPos; p += 4) {
            float4 pr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) pr[i] = *reinterpret_cast<const float4*>(sP + (4 * ty + i) * (kPfPos + 4) + p);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 va = *reinterpret_cast<const float4*>(sV + (p + e) * kAttnD + 4 * tx);
                const float4 vb = *reinterpret_cast<const float4*>(sV + (p + e) * kAttnD + 64 + 4 * tx);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float c = (&pr[i].x)[e];
                    const float2 c2 = make_float2(c, c);
                    o[i][0] = fma2(c2, make_float2(va.x, va.y), o[i][0]);
                    o[i][1] = fma2(c2, make_float2(va.z, va.w), o[i][1]);
                    o[i][2] = fma2(c2, make_float2(vb.x, vb.y), o[i][2]);
                    o[i][3] = fma2(c2, make_float2(vb.z, vb.w), o[i][3]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
        const int row = 4 * ty + i;
        if (row >= rows || W > 1) continue;
        float* to = out + packed(row) * a.out_stride + column(row) + 4 * tx;
        const float inv = bad[i] ? NAN : 1.f / l[i];
        *reinterpret_cast<float4*>(to) = make_float4(o[i][0].x * inv, o[i][0].y * inv, o[i][1].x * inv, o[i][1].y * inv);
        *reinterpret_cast<float4*>(to + 64) = make_float4(o[i][2].x * inv, o[i][2].y * inv, o[i][3].x * inv, o[i][3].y * inv);
        if (a.lse && tx == 0) a.lse[packed(row) * a.Hq + g * R + row % R] = fmaf(m[i], kLn2, logf(l[i]));
    }
    if (W == 1) return;
    __syncthreads();  // the keys and the weights are read
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 4 * ty + i;
        const float poison = bad[i] ? NAN : 0.f;
        float* to = pf + PfSmem::kO + row * kAttnD + 4 * tx;
        *reinterpret_cast<float4*>(to) = make_float4(o[i][0].x + poison, o[i][0].y + poison, o[i][1].x + poison, o[i][1].y + poison);
        *reinterpret_cast<float4*>(to + 64) =
            make_float4(o[i][2].x + poison, o[i][2].y + poison, o[i][3].x + poison, o[i][3].y + poison);
        if (tx == 0) *reinterpret_cast<float2*>(pf + PfSmem::kMl + 2 * row) = make_float2(m[i], l[i]);
    }
    tc::cluster_arrive();  // every CTA's rows are in its shared memory ...
    tc::cluster_wait();
    // ... and each merges a share of them, a warp a row, four dims a lane
    const int share = kPfRows / W, lane = tid & 31;
    const uint32_t base = tc::smem_u32(pf);
    for (int row = wk * share + (tid >> 5); row < min((wk + 1) * share, rows); row += kPfThreads / 32) {
        float M = kNone, L = 0.f;
        for (int w = 0; w < W; ++w)
            M = fmaxf(M, ld_cluster_f32x2(tc::cluster_map(base + (PfSmem::kMl + 2 * row) * 4, w)).x);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < W; ++w) {
            const float2 ml = ld_cluster_f32x2(tc::cluster_map(base + (PfSmem::kMl + 2 * row) * 4, w));
            const float4 v = ld_cluster_f32x4(tc::cluster_map(base + (PfSmem::kO + row * kAttnD + 4 * lane) * 4, w));
            const float f = ex2_approx(ml.x - M);
            L = fmaf(f, ml.y, L);
            sum.x = fmaf(f, v.x, sum.x), sum.y = fmaf(f, v.y, sum.y), sum.z = fmaf(f, v.z, sum.z), sum.w = fmaf(f, v.w, sum.w);
        }
        const float inv = 1.f / L;
        *reinterpret_cast<float4*>(out + packed(row) * a.out_stride + column(row) + 4 * lane) =
            make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
        if (a.lse && lane == 0) a.lse[packed(row) * a.Hq + g * R + row % R] = fmaf(M, kLn2, logf(L));
    }
    tc::cluster_arrive();  // nobody leaves while its memory is read
    tc::cluster_wait();
}

cudaError_t launch_f32(const PromptArgs& a, cudaStream_t st) {
    constexpr int bytes = PfSmem::kFloats * 4;
    cudaError_t e = allow_shared<0>((const void*)prompt_f32_kernel, bytes);
    if (e != cudaSuccess) return e;
    const long blocks = most_tiles(a.S, a.rows, kPfRows / (a.Hq / a.Hkv)) * a.Hkv;
    // CTAs that share a tile's positions, while they leave SMs idle (two an SM; 12 / 2 heads, 75 rows behind 7,400
    // positions: 123 us with eight, 149, 285 and 553 with four, two and one; one row behind 600: 16, 21, 31 and 52)
    const long reach = a.lens || a.rows > a.Tmax ? a.Tmax : a.rows, chunks = (reach + kPfPos - 1) / kPfPos;
    int W = 1;
    while (W < 8 && 2 * W <= chunks && blocks * 2 * W <= 2 * 152) W *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(W * blocks));
    cfg.blockDim = dim3(kPfThreads);
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
    return cudaLaunchKernelEx(&cfg, prompt_f32_kernel, a, W);
}

}  // namespace

cudaError_t launch_attn_prompt(const PromptArgs& a, cudaStream_t st) {
    cudaError_t e = launch_append(a, st);
    if (e != cudaSuccess || a.rows == 0) return e;
    return a.bf16 ? launch_attn_prompt_tiles(a, st) : launch_f32(a, st);
}

}  // namespace m2
