// Grouped-query attention over the paged e4m3 cache (m2_kv_append.cu writes
// it): for session s with total = lengths[s] + n_new[s] positions cached,
// query t of the call (position lengths[s] + t) and head h (kv head g = h / R)
//     a_p = scale q . (ks_p k_p),   out = sum_p softmax(a)_p vs_p v_p
// over the positions p <= lengths[s] + t (causal), or over p < lengths[s]
// (cross attention: a cache of other states, the same for every query). ks
// and vs are the scales of the position's block of 16.
//
// attn_paged_rows_kernel: few rows (single frames). A kv head's rows are its
// (query, head) pairs, row = t R + r, taken 8 or 16 at a time. Bound by HBM:
// every cached key and value is read once for 8 or 16 rows, 256 bytes and
// 32 scale-bits a position and kv head. One CTA ("walker") takes every W-th
// 64-position chunk of one (session, kv head, row group): a producer warp
// keeps a ring of TMA copies in flight (a page, or the part of one that lies
// in the chunk, is one box of 128-byte rows; the scales come by 4-byte
// asynchronous copies on the same barrier), and each of four warps takes 16
// positions of every chunk, which is one block of the cache, so that both
// scales are constants of the warp. The walkers of one (session, kv head, row
// group) form a thread-block cluster and merge through distributed shared
// memory, so that one launch does it all.
//   Measured, 40 query and 8 kv heads, bf16: 64 sessions of 40 to 7,500
// positions 86 us (5.9 TB/s of cache, 89% of a copy's rate); one session over
// 7,500 positions 9.1 us, over 300 4.3 us, where latency counts: a launch, two
// rounds of loads, the merge.
//
// Codes become fp16 exactly (cvt from e4m3), so the products run on fp16
// matrix instructions with fp32 sums:
//   q      scaled by a power of two for each row (its largest element to
//          [2^14, 2^15)): a bf16 row is exact, an fp32 row goes in as two
//          terms, hi + lo, 22 bits;
//   weight p = 2^(x - m) goes in times its value's scale, relative to the
//          running maximum of that product: w = p vs 2^(m - mv + 15), at most
//          2^15, one fp16 term (2^-11) for bf16 activations, two for fp32.
//          Blocks whose values are of very different size thus lose nothing
//          to fp16's range; sums of p (l) stay fp32 and apart.
//     out = 2^(mv - m - 15) acc / l.
#include <math.h>

#include <mutex>

#include "m2_paged_dev.cuh"

namespace m2 {

namespace {

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// d += A B, m16n8k16, fp16 in, fp32 accumulate
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The warp's 8 x 8 matrix of 16-bit elements, transposed, in the same layout.
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
constexpr int kRwWarps = 4;                              // warps that compute
constexpr int kRwThreads = 32 * kRwWarps + 32;           // ... and the producer
constexpr int kRwTc = 16 * kRwWarps;                     // positions per chunk
constexpr uint32_t kRwTile = kRwTc * kKvD;               // a chunk's keys (or values)
constexpr int kRwMaxW = 16;                              // walkers per cluster
constexpr uint32_t kRwSlotF = kKvD + 4;                  // floats of a merge slot: acc, m, l, mv

// Shared memory of rows groups of 8 NT rows: the ring (keys, then values of
// each stage), the stages' scales, the slots that an owner receives, barriers.
template <int NT>
struct RwSmem {
    static constexpr int kRows = 8 * NT;
    static constexpr int kStages = NT == 1 ? 6 : 5;
    static constexpr int kSlots = kRows + kRwMaxW - 1;  // ceil(rows / W) W, at most
    static constexpr uint32_t kScales = kStages * 2 * kRwTile;               // float [stage][8]
    static constexpr uint32_t kRecv = kScales + kStages * 2 * kRwWarps * 4;
    static constexpr uint32_t kBar = kRecv + kSlots * kRwSlotF * 4;          // full, empty [kStages]
    static constexpr uint32_t kFlag = kBar + 2 * kStages * 8;
    static constexpr uint32_t kKeys = kFlag + 16;                            // int [kRwThreads + 1]: the sessions' ranking
    static constexpr uint32_t kBytes = kKeys + (kRwThreads + 1) * 4 + 1024;  // + slack to align to 1024
    // the warps' merge, over the ring: acc [warp][row][128], then (m, l, mv)
    static constexpr uint32_t kMl = kRwWarps * kRows * kKvD * 4;
    static_assert(kMl + kRwWarps * kRows * 4 * 4 <= kScales, "the merge fits in the ring");
    static_assert(2 * (kBytes + 1024) <= 228 * 1024, "two CTAs an SM");
};

struct RwMaps {
    CUtensorMap kv[2];  // the keys' pages, the values'
};

// A lane's 32 dims of a query row: 4t .. 4t + 3 of each 16, as loaded.
template <typename TA>
struct QueryRow {
    using Four = typename std::conditional<sizeof(TA) == 2, uint2, float4>::type;
    Four w[8];
    __device__ __forceinline__ void load(const PagedAttnArgs& a, int s, int g, int R, int row, int t) {
        const size_t at = ((size_t)s * a.T + row / R) * a.q_stride + (size_t)(g * R + row % R) * kKvD + 4 * t;
        const char* p = reinterpret_cast<const char*>(a.q) + at * sizeof(TA);
#pragma unroll
        for (int u = 0; u < 8; ++u) w[u] = __ldg(reinterpret_cast<const Four*>(p + 16 * u * sizeof(TA)));
    }
    __device__ __forceinline__ void get(int u, float (&x)[4]) const {
        if constexpr (sizeof(TA) == 2) {
            x[0] = __uint_as_float(w[u].x << 16);
            x[1] = __uint_as_float(w[u].x & 0xFFFF0000u);
            x[2] = __uint_as_float(w[u].y << 16);
            x[3] = __uint_as_float(w[u].y & 0xFFFF0000u);
        } else {
            x[0] = w[u].x, x[1] = w[u].y, x[2] = w[u].z, x[3] = w[u].w;
        }
    }
};

// grid (W x Hkv x row groups, S), a cluster of W walkers when W > 1.
// TERMS: fp16 terms of a query and of a weight (2 for fp32 activations).
template <typename TA, int NT, int TERMS>
__global__ void __launch_bounds__(kRwThreads, 2)
    attn_paged_rows_kernel(PagedAttnArgs a, const __grid_constant__ RwMaps maps, int W, bool ranked) {
    using L = RwSmem<NT>;
    constexpr int ST = L::kStages;
    extern __shared__ uint8_t rw_raw[];
    uint8_t* sm = rw_raw + ((1024u - (tc::smem_u32(rw_raw) & 1023u)) & 1023u);
    float* scales = reinterpret_cast<float*>(sm + L::kScales);
    float* recv = reinterpret_cast<float*>(sm + L::kRecv);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint64_t* empty = full + ST;
    volatile uint32_t* flag = reinterpret_cast<uint32_t*>(sm + L::kFlag);
    const KvCache& c = a.c;
    const int wk = (int)blockIdx.x % W, pair = (int)blockIdx.x / W;
    int s = blockIdx.y;
    const int g = pair % c.Hkv, row0 = pair / c.Hkv * L::kRows;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int R = a.Hq / c.Hkv;

    if (tid == 0) {
        for (int i = 0; i < ST; ++i) {
            tc::mbar_init(full + i, 1 + 32);
            tc::mbar_init(empty + i, kRwWarps);
        }
        tc::fence_mbar_init();
        *flag = 0;
    }
    if (tid == 32) prefetch_map(maps.kv), prefetch_map(maps.kv + 1);
    if (W > 1) tc::cluster_arrive_relaxed();  // waited on before the first remote store: every walker has started
    pdl_wait();  // the queries and the cache may come from the previous kernel
    pdl_trigger();
    if (ranked) {
        // More CTAs than the GPU holds at once, in the order of blockIdx: the
        // sessions by their lengths, the longest first, so that none of them is
        // still at work alone at the end. (At most a session a thread.)
        int* key = reinterpret_cast<int*>(sm + L::kKeys);
        const int mine = tid >= c.S ? 0 : a.n_new && a.n_new[tid] <= 0 ? -1 : a.lens[tid];
        key[tid] = mine;
        __syncthreads();
        if (tid < c.S) {
            int rank = 0;
#pragma unroll 8
            for (int u = 0; u < c.S; ++u) rank += key[u] > mine || (key[u] == mine && u < tid);
            if (rank == (int)blockIdx.y) key[kRwThreads] = tid;
        }
        __syncthreads();
        s = key[kRwThreads];
    }
    // what does not need the session's length is on its way beside it: the
    // page numbers of the first chunks (a lane an entry, ppc a chunk) ...
    const int ppc = c.ps < kRwTc ? kRwTc >> c.ps_shift : 1;
    auto entry = [&](int k) -> int {
        const long i = ((long)(wk + (k + lane / ppc) * W) * kRwTc >> c.ps_shift) + lane % ppc;
        return i < c.max_pages ? c.table[(size_t)s * c.max_pages + i] : 0;
    };
    int page_ids = warp == kRwWarps ? entry(0) : 0;
    // ... and the queries (rows past the session's new ones are read, not used)
    QueryRow<TA> q[NT];
    if (warp < kRwWarps) {
#pragma unroll
        for (int f = 0; f < NT; ++f) q[f].load(a, s, g, R, min(row0 + 8 * f + (lane >> 2), a.T * R - 1), lane & 3);
    }
    int before, n;
    const bool ok = kv_extent(c, s, a.T, a.lens, a.n_new, a.causal ? c.capacity() : c.capacity() + a.T, &before, &n) &&
                    before <= c.capacity();
    if (!ok && blockIdx.x == 0 && tid == 0) record_error(c.err, ERR_ATTN_LENGTH);
    const int rows = min(n * R - row0, (int)L::kRows);
    if (rows <= 0) return;  // the whole cluster
    // positions that this group's last row sees, and this walker's chunks of
    // them: wk, wk + W, ...
    const int total = !ok ? 0 : a.causal ? before + (row0 + rows - 1) / R + 1 : before;
    const int nch = (total + kRwTc - 1) / kRwTc, nc = nch > wk ? (nch - wk + W - 1) / W : 0;
    __syncthreads();  // the barriers are initialised

    if (warp == kRwWarps) {
        // ---------------------------------------------------------- producer
        const int box = min(c.ps, kRwTc), pieces = kRwTc / box;  // rows a copy, copies a chunk
        int held = 0;  // the first chunk whose pages the lanes hold
        bool good = true;
        for (int k = 0; k < nc && good; ++k) {
            const int st = k % ST;
            const uint32_t round = (uint32_t)(k / ST);
            if (round > 0 && !tc::mbar_wait(empty + st, (round - 1) & 1)) {
                if (lane == 0) record_error(c.err, ERR_MBAR_TIMEOUT_LOAD);
                *flag = 1;
                good = false;
            }
            good = __all_sync(0xffffffffu, good);
            if (!good) break;
            const int p0 = (wk + k * W) * kRwTc, left = min(kRwTc, total - p0);  // positions to load
            if (k - held == 32 / ppc) {
                held = k;
                page_ids = entry(k);
            }
            const int at0 = (k - held) * ppc;  // lane of the chunk's first page
            if (lane >= at0 && lane < at0 + ppc && p0 + ((lane - at0) << c.ps_shift) < total &&
                (page_ids < 0 || page_ids >= c.n_pages)) {
                record_error(c.err, ERR_KV_PAGE);
                page_ids = 0;  // some page of the pool: what is read is undefined
            }
            __syncwarp();
            uint8_t* dst = sm + st * 2 * kRwTile;
            const int live = (left + box - 1) / box;
            if (lane == 0) tc::mbar_arrive_expect_tx(full + st, (uint32_t)(live * box * kKvD * 2));
            __syncwarp();
            {
                // lane i: keys of page i of the chunk, lane 16 + i its values (one lane for all
                // of them took 1 us more with pages of 16). In one instruction, 64 sessions'
                // frames take 86 us against 89 in two; with 16 rows, two save the registers
                // that it spills (187 us against 189 for 40 rows of 64 sessions).
                const int i = lane & 15;
                const int page = __shfl_sync(0xffffffffu, page_ids, at0 + min(i, pieces - 1));
                if (i < live) {
                    const int y = (page * c.Hkv + g) * c.ps + (p0 & (c.ps - 1));  // (0 for pages of at most a chunk)
                    if constexpr (NT == 1)
                        tc::tma_load_2d(dst + (lane >> 4) * kRwTile + i * box * kKvD, maps.kv + (lane >> 4), 0, y, full + st);
                    else if (lane < 16)
                        tc::tma_load_2d(dst + i * box * kKvD, maps.kv, 0, y, full + st);
                    else
                        tc::tma_load_2d(dst + kRwTile + i * box * kKvD, maps.kv + 1, 0, y, full + st);
                }
            }
            // the chunk's scales: lanes 0 .. 3 the keys' four blocks, 4 .. 7 the values'
            {
                const int b = lane & (kRwWarps - 1), p = p0 + b * kKvBlock;
                const int page = __shfl_sync(0xffffffffu, page_ids, at0 + (b * kKvBlock >> c.ps_shift));
                if (lane < 2 * kRwWarps && p < total) {
                    const size_t at = (((size_t)page * c.Hkv + g) << (c.ps_shift - 4)) + ((p & (c.ps - 1)) >> 4);
                    cp_async4(scales + st * 2 * kRwWarps + lane, (lane < kRwWarps ? c.ks : c.vs) + at);
                }
                cp_async_arrive(full + st);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    const int gq = lane >> 2, t = lane & 3;  // fragment row and lane in its quad
    // per fragment of 8 rows: scores' factor, and the last position seen, of
    // rows 2t and 2t + 1; running maximum, this lane's part of the sum,
    // reference of the weights; acc^T: dims 16 u + 2 gq (+ 1) of rows 2t, 2t + 1
    float m[NT][2], l[NT][2], mv[NT][2], acc[NT][8][4];
#pragma unroll
    for (int f = 0; f < NT; ++f) {
#pragma unroll
        for (int e = 0; e < 2; ++e) m[f][e] = mv[f][e] = kNone, l[f][e] = 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[f][u][e] = 0.f;
    }
    if (warp < kRwWarps) {
        // Q^T as the B operand (k = dims, n = row gq): the 16 dims of a K-step
        // are taken in the order of the keys' bytes, lane t its dims 4t .. 4t + 3
        uint32_t qb[NT][8][TERMS][2];
        float cs[NT][2];
        int lim[NT][2];
#pragma unroll
        for (int f = 0; f < NT; ++f) {
            float x[8][4], top = 0.f;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                q[f].get(u, x[u]);
#pragma unroll
                for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(x[u][e]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // (a row that holds an infinity reads NaN)
            const float pw = top < INFINITY ? row_power(top, 14) : NAN, sg = a.scale < 0.f ? -pw : pw;
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float y0 = x[u][2 * h] * sg, y1 = x[u][2 * h + 1] * sg;
                    qb[f][u][0][h] = pack_f16x2(y0, y1);
                    if constexpr (TERMS == 2) {
                        const float2 hi = unpack_f16x2(qb[f][u][0][h]);
                        qb[f][u][1][h] = pack_f16x2(y0 - hi.x, y1 - hi.y);
                    }
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float p2 = __shfl_sync(0xffffffffu, pw, 4 * (2 * t + e));
                cs[f][e] = fabsf(a.scale) * kLog2e / p2;
                const int r = 8 * f + 2 * t + e;
                lim[f][e] = r >= rows ? -1 : a.causal ? before + (row0 + r) / R : total - 1;
            }
        }
        bool good = true;
        for (int k = 0; k < nc; ++k) {
            const int st = k % ST;
            if (!tc::mbar_wait(full + st, (uint32_t)(k / ST) & 1)) {
                record_error(c.err, ERR_MBAR_TIMEOUT_LOAD);
                *flag = 1;
                good = false;
            }
            good = __all_sync(0xffffffffu, good);
            if (!good) break;
            const int p0 = (wk + k * W) * kRwTc + 16 * warp;  // this warp's block
            if (p0 < total) {
                uint8_t* sV = sm + st * 2 * kRwTile + kRwTile + warp * 16 * kKvD;
                const uint32_t kb = tc::smem_u32(sV - kRwTile), vb = tc::smem_u32(sV);
                const float ks = scales[st * 2 * kRwWarps + warp], vs = scales[st * 2 * kRwWarps + kRwWarps + warp];
                // whatever lies behind the last position counts as zero values, and so do
                // those of a block with a scale that is not finite: the rows that see it get
                // their NaN by the weights, and the others none
                const int from = fabsf(vs) < INFINITY ? min(total - p0, 16) : 0;
                if (from < 16) {
                    for (int e = lane; e < (16 - from) * 8; e += 32)
                        *reinterpret_cast<uint4*>(sV + from * kKvD + e * 16) = make_uint4(0u, 0u, 0u, 0u);
                    tc::fence_proxy_async_smem();  // ahead of the next copy into the stage
                    __syncwarp();
                }
                // S^T (16 positions x 8 rows): lanes 8j .. 8j + 7 address the
                // 8 x 16-byte piece j: positions + 8 (j & 1), 16-byte unit + (j >> 1)
                const int fr = (lane & 7) + 8 * ((lane >> 3) & 1), fu = lane >> 4;
                float sc[NT][4];
#pragma unroll
                for (int f = 0; f < NT; ++f)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[f][e] = 0.f;
#pragma unroll
                for (int u = 0; u < 8; u += 2) {
                    uint32_t w[4];
                    ldsm_x4(kb + fr * kKvD + (((u + fu) ^ (fr & 7)) << 4), w);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t a0 = e4m3x2_to_f16x2(w[2 * h] & 0xFFFFu), a2 = e4m3x2_to_f16x2(w[2 * h] >> 16);
                        const uint32_t a1 = e4m3x2_to_f16x2(w[2 * h + 1] & 0xFFFFu), a3 = e4m3x2_to_f16x2(w[2 * h + 1] >> 16);
#pragma unroll
                        for (int f = 0; f < NT; ++f)
#pragma unroll
                            for (int k = 0; k < TERMS; ++k)
                                mma_f16(sc[f], a0, a1, a2, a3, qb[f][u + h][k][0], qb[f][u + h][k][1]);
                    }
                }
                const float lvs = lg2_approx(vs);
                uint32_t pb[NT][TERMS][2];
#pragma unroll
                for (int f = 0; f < NT; ++f) {
                    float x[4], w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[e] = p0 + gq + 8 * (e >> 1) <= lim[f][e & 1] ? sc[f][e] * (cs[f][e & 1] * ks) : -INFINITY;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(x[e], x[e + 2]);
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                        const float mn = fmaxf(m[f][e], mx), vn = fmaxf(mv[f][e], mx + lvs);
                        const float cl = ex2_approx(m[f][e] - mn), cv = ex2_approx(mv[f][e] - vn);
                        m[f][e] = mn;
                        mv[f][e] = vn;
                        const float pa = ex2_approx(x[e] - mn), pc = ex2_approx(x[e + 2] - mn);  // 0 for -inf
                        l[f][e] = fmaf(l[f][e], cl, pa + pc);
                        const float to = vs == 0.f || p0 > lim[f][e] ? 0.f : vs * ex2_approx(mn - vn + 15.f);
                        w[e] = pa * to;
                        w[e + 2] = pc * to;
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            acc[f][u][e] *= cv;
                            acc[f][u][e + 2] *= cv;
                        }
                    }
                    // P^T as the B operand (k = positions, n = row gq)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t hi = pack_f16x2(w[2 * h], w[2 * h + 1]);
                        pb[f][0][h] = movmatrix_t(hi);
                        if constexpr (TERMS == 2) {
                            const float2 back = unpack_f16x2(hi);
                            pb[f][1][h] = movmatrix_t(pack_f16x2(w[2 * h] - back.x, w[2 * h + 1] - back.y));
                        }
                    }
                }
                // acc^T += V^T P^T. A transposed 8 x 8 piece gives a lane the
                // dims (2 gq, 2 gq + 1) of positions 2t, 2t + 1: dim 2 gq goes to
                // the product's row gq, 2 gq + 1 to row gq + 8
#pragma unroll
                for (int u = 0; u < 8; u += 2) {
                    uint32_t w[4];
                    ldsm_x4_trans(vb + fr * kKvD + (((u + fu) ^ (fr & 7)) << 4), w);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t lo = __byte_perm(w[2 * h], 0, 0x3120), hi = __byte_perm(w[2 * h + 1], 0, 0x3120);
                        const uint32_t a0 = e4m3x2_to_f16x2(lo & 0xFFFFu), a1 = e4m3x2_to_f16x2(lo >> 16);
                        const uint32_t a2 = e4m3x2_to_f16x2(hi & 0xFFFFu), a3 = e4m3x2_to_f16x2(hi >> 16);
#pragma unroll
                        for (int f = 0; f < NT; ++f)
#pragma unroll
                            for (int k = 0; k < TERMS; ++k) mma_f16(acc[f][u + h], a0, a1, a2, a3, pb[f][k][0], pb[f][k][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(empty + st);
        }
    }
    __syncthreads();  // the ring is free for the merge
    if (*flag) {
        // a wait gave up: let the copies still in flight land (bounded) and
        // contribute nothing (the error word is set)
        if (tid == 0)
            for (int i = 0; i < ST; ++i)
                tc::mbar_wait(full + i, 0, 100000000ull), tc::mbar_wait(full + i, 1, 100000000ull);
        __syncthreads();
#pragma unroll
        for (int f = 0; f < NT; ++f) {
#pragma unroll
            for (int e = 0; e < 2; ++e) m[f][e] = mv[f][e] = kNone, l[f][e] = 0.f;
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[f][u][e] = 0.f;
        }
    }
    // the warps' results through shared memory
    float* sacc = reinterpret_cast<float*>(sm);
    float4* sml = reinterpret_cast<float4*>(sm + L::kMl);
    if (warp < kRwWarps) {
#pragma unroll
        for (int f = 0; f < NT; ++f)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) l[f][e] += __shfl_xor_sync(0xffffffffu, l[f][e], off);
                const int r = warp * L::kRows + 8 * f + 2 * t + e;
                if (gq == 0) sml[r] = make_float4(m[f][e], l[f][e], mv[f][e], 0.f);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    *reinterpret_cast<float2*>(sacc + r * kKvD + 16 * u + 2 * gq) = make_float2(acc[f][u][e], acc[f][u][e + 2]);
            }
    }
    __syncthreads();
    if (W > 1) tc::cluster_wait();  // every walker of the cluster has started: its shared memory is there
    // A warp takes a row and a lane four of its dims. This walker's (acc, m, l,
    // mv) of row r, each relative to the walker's own references, go to the
    // row's owner: slot (r / W) W + wk of walker r % W.
    auto write = [&](int r, const float (&o)[4], float sum, float from) {
        const int row = row0 + r;
        const size_t at = ((size_t)s * a.T + row / R) * a.out_stride + (size_t)(g * R + row % R) * kKvD + 4 * lane;
        const float f = sum == 0.f ? 0.f : 1.f / sum;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = sum == 0.f ? 0.f : o[e] * f * from;  // a row that sees nothing: zeros
        if constexpr (sizeof(TA) == 2) {
            *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at) =
                make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
        } else {
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
        }
    };
    for (int r = warp; r < rows; r += kRwThreads / 32) {
        float4 x[kRwWarps], y[kRwWarps];
        float M = kNone, V = kNone, sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kRwWarps; ++w) {
            x[w] = sml[w * L::kRows + r];
            y[w] = *reinterpret_cast<const float4*>(sacc + (w * L::kRows + r) * kKvD + 4 * lane);
            M = fmaxf(M, x[w].x);
            V = fmaxf(V, x[w].z);
        }
#pragma unroll
        for (int w = 0; w < kRwWarps; ++w) {
            const float f = ex2_approx(x[w].z - V);
            o[0] = fmaf(f, y[w].x, o[0]), o[1] = fmaf(f, y[w].y, o[1]);
            o[2] = fmaf(f, y[w].z, o[2]), o[3] = fmaf(f, y[w].w, o[3]);
            sum = fmaf(ex2_approx(x[w].x - M), x[w].y, sum);
        }
        if (W == 1) {
            write(r, o, sum, ex2_approx(V - M - 15.f));
        } else {
            const uint32_t slot = tc::cluster_map(tc::smem_u32(recv + ((r / W) * W + wk) * kRwSlotF), (uint32_t)(r % W));
            st_cluster_f32x4(slot + 16u * lane, make_float4(o[0], o[1], o[2], o[3]));
            if (lane == 0) st_cluster_f32x4(slot + 4u * kKvD, make_float4(M, sum, V, 0.f));
        }
    }
    if (W == 1) return;
    tc::cluster_arrive();  // the stores into the owners' slots are visible ...
    tc::cluster_wait();    // ... once every walker has made them
    for (int r = wk + W * warp; r < rows; r += W * (kRwThreads / 32)) {
        const float* sl = recv + (r / W) * W * kRwSlotF;
        // lane w: walker w's references and sum
        const float4 x = lane < W ? *reinterpret_cast<const float4*>(sl + lane * kRwSlotF + kKvD) : make_float4(kNone, 0.f, kNone, 0.f);
        float M = x.x, V = x.z;
#pragma unroll
        for (int off = 1; off < kRwMaxW; off <<= 1) {
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
            V = fmaxf(V, __shfl_xor_sync(0xffffffffu, V, off));
        }
        M = __shfl_sync(0xffffffffu, M, 0), V = __shfl_sync(0xffffffffu, V, 0);
        float sum = ex2_approx(x.x - M) * x.y;
#pragma unroll
        for (int off = 1; off < kRwMaxW; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        sum = __shfl_sync(0xffffffffu, sum, 0);
        const float fw = ex2_approx(x.z - V);
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int w = 0; w < W; ++w) {
            const float f = __shfl_sync(0xffffffffu, fw, w);
            const float4 y = *reinterpret_cast<const float4*>(sl + w * kRwSlotF + 4 * lane);
            o[0] = fmaf(f, y.x, o[0]), o[1] = fmaf(f, y.y, o[1]), o[2] = fmaf(f, y.z, o[2]), o[3] = fmaf(f, y.w, o[3]);
        }
        write(r, o, sum, ex2_approx(V - M - 15.f));
    }
}

// Per device, once: the kernel's shared-memory and cluster attributes, and
// how many clusters of 2, 4, 8 and 16 walkers the device holds at once.
struct RwSetup {
    bool done;
    int clusters[5];
};

template <typename TA, int NT, int TERMS>
cudaError_t rows_setup(const RwSetup** out) {
    static std::mutex mutex;
    static RwSetup per_device[64];
    auto* kernel = attn_paged_rows_kernel<TA, NT, TERMS>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mutex);
    RwSetup& u = per_device[dev & 63];
    if (!u.done) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)RwSmem<NT>::kBytes);
        if (e != cudaSuccess) return e;
        const bool wide = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
        u.clusters[0] = 2 * 152;
        for (int k = 1; k < 5; ++k) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(1u << k);
            cfg.blockDim = dim3(kRwThreads);
            cfg.dynamicSmemBytes = RwSmem<NT>::kBytes;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1u << k;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int held = 0;
            if ((k == 4 && !wide) || cudaOccupancyMaxActiveClusters(&held, kernel, &cfg) != cudaSuccess) held = 0;
            u.clusters[k] = held;
        }
        (void)cudaGetLastError();  // a refused query leaves no sticky error
        u.done = true;
    }
    *out = &u;
    return cudaSuccess;
}

template <typename TA, int NT, int TERMS>
cudaError_t plan_rows(const PagedAttnArgs& a, PagedAttnPlan* plan) {
    const RwSetup* setup = nullptr;
    cudaError_t e = rows_setup<TA, NT, TERMS>(&setup);
    if (e != cudaSuccess) return e;
    const int groups = (a.T * (a.Hq / a.c.Hkv) + 8 * NT - 1) / (8 * NT);
    // Walkers: the least time in chunks (of about half a microsecond), with 10
    // for a CTA's start and end and 2 (4 where many merge) for the merge. The
    // lengths are on the device; the table's reach stands for them. One
    // session's walkers are all alike: rounds x a walker's time. Several
    // sessions are mostly shorter than the reach, say by half: the longest
    // walker's time, or all of them over the CTAs held at once. (40
    // query and 8 kv heads, sessions of up to 7,500 positions: 4 sessions 14 us
    // with 8 walkers, 21 with 4; 12: 25 with 4, 31 with 8, 43 with 2; 24: 42
    // with 4, 45 with 2; 40: 53 with 2, 66 with 4, 82 with 1; 64: 89 with 1, 93
    // with 2. One session over 300: 4.4 us with 8, 4.9 with 4.)
    const long pairs = (long)a.c.S * a.c.Hkv * groups, chunks = (a.c.capacity() + kRwTc - 1) / kRwTc;
    plan->tiles = false;
    float least = 0.f;
    for (int k = 0, w = 1; k < 5 && (w == 1 || w < 2 * chunks) && setup->clusters[k] > 0; ++k, w *= 2) {
        const float part = (float)pairs / (float)setup->clusters[k], walk = (float)((chunks + w - 1) / w);
        const float cost = a.c.S == 1 ? ceilf(part) * (walk + (w > 1 ? 12.f : 10.f))
                                      : fmaxf(walk + (w > 1 ? 14.f : 10.f),
                                              part * ((float)chunks / (float)(2 * w) + (w > 1 ? 14.f : 10.f)));
        if (w > 1 && cost >= least) continue;
        least = cost;
        plan->W = w;
        // (fitted to 16 rows a walker, bf16)
        const float start = w > 1 ? 5.5f : 4.5f;
        plan->us = a.c.S == 1 ? ceilf(part) * (start + 0.7f * walk) : fmaxf(start + 0.6f * walk, part * (start + 0.46f * walk));
    }
    return cudaSuccess;
}

template <typename TA, int NT, int TERMS>
cudaError_t launch_rows(const PagedAttnArgs& a, int W, cudaStream_t st) {
    RwMaps maps;
    cudaError_t e = make_page_map(a.c.kp, a.c, kRwTc, &maps.kv[0]);
    if (e == cudaSuccess) e = make_page_map(a.c.vp, a.c, kRwTc, &maps.kv[1]);
    if (e != cudaSuccess) return e;
    const int groups = (a.T * (a.Hq / a.c.Hkv) + 8 * NT - 1) / (8 * NT);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(W * groups * a.c.Hkv, a.c.S);
    cfg.blockDim = dim3(kRwThreads);
    cfg.dynamicSmemBytes = RwSmem<NT>::kBytes;
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
    const bool ranked = a.c.S > 1 && a.c.S <= kRwThreads && (long)a.c.S * a.c.Hkv * groups * W > 2 * 152;
    return cudaLaunchKernelEx(&cfg, attn_paged_rows_kernel<TA, NT, TERMS>, a, maps, W, ranked);
}

// bf16 rows that go 8 at a time
bool few_rows(const PagedAttnArgs& a) { return (long)a.T * (a.Hq / a.c.Hkv) <= 8; }

}  // namespace

cudaError_t plan_attn_paged(const PagedAttnArgs& a, PagedAttnPlan* plan) {
    // fp32 takes 8 rows at a time: 16 hold 255 registers and one CTA an SM (six
    // sessions catching up 111 us against 109, 20 rows of 64 sessions 240 against
    // 207).
    if (!a.bf16) return plan_rows<float, 1, 2>(a, plan);
    if (few_rows(a)) return plan_rows<bf16_t, 1, 1>(a, plan);
    // Sixteen rows at a time, each time reading the cache again, against tiles
    // that compute 256 and take 8 us to start and end: by a guess of both times,
    // whose constants are fitted to 150 calls (40 query and 8 kv heads; one session,
    // several alike or ragged, 10 to 2,000 rows over 12 to 7,500 positions, tables
    // that end with the longest session; the tiles' with a margin, since where the
    // two are near, long lengths cost the rows more).
    // One session, 8 kv heads: 60 rows over 12 positions 5.2 us (tiles: 8.4), over
    // 2,000 9.7 (14.5), over 6,000 16.8 (21.0); 240 rows over 148 6.5 (10.6), over
    // 2,048 21 (17), over 6,048 48 (25). 64 sessions of up to 7,500: 20 rows 148
    // (210), 80 rows 278 (189).
    PagedAttnPlan few, many;
    cudaError_t e = plan_rows<bf16_t, 2, 1>(a, &few);
    if (e == cudaSuccess) e = plan_attn_paged_tiles(a, &many);
    if (e != cudaSuccess) return e;
    *plan = few.us < 0.85f * many.us ? few : many;
    return cudaSuccess;
}

cudaError_t launch_attn_paged(const PagedAttnArgs& a, cudaStream_t st) {
    PagedAttnPlan plan;
    const cudaError_t e = plan_attn_paged(a, &plan);
    if (e != cudaSuccess) return e;
    if (plan.tiles) return launch_attn_paged_tiles(a, plan.W, st);
    if (!a.bf16) return launch_rows<float, 1, 2>(a, plan.W, st);
    return few_rows(a) ? launch_rows<bf16_t, 1, 1>(a, plan.W, st) : launch_rows<bf16_t, 2, 1>(a, plan.W, st);
}

}  // namespace m2
