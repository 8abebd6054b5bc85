// Attention of packed whole prompts over the dense bf16 caches, on the tcgen05
// tensor cores (the operator and its formulas are those of m2_attn_prompt.cu).
//
// One CTA takes two tiles of rows of one (session, kv head) and walks the
// positions they see, 128 at a time. A tile is floor(128 / R) packed rows of R
// heads (all 128 rows of a product for 1, 2, 4 and 8 heads a kv head, 125 for
// the model's 5), so that its queries are one box of a tensor map. Per chunk and
// tile:
//   S = q K^T       kind::f16, both from shared memory (128-byte swizzle);
//   softmax         one thread a row, S read out of tensor memory in fp32 with
//                   its maxima (tcgen05.ld.red): x = S scale log2(e),
//                   p = 2^(x - m), l += p, and p to bf16 over S. bf16 because
//                   both operands of a product have one type and the values are
//                   bf16: a weight is off by 2^-8 of itself at most;
//   O += p V        p from tensor memory, V as the copies left it (MN-major).
// m moves only when a chunk exceeds it by more than 2^8, which fp32 sums and
// bf16 weights allow at no loss; only then is O rescaled in tensor memory.
//     out = O / l,  lse = m ln 2 + ln l.
//
// Warps: 0 copies (rings of K and V by TMA), 1 issues the products, 2 waits for
// their operands, 3 mends the values of chunks that some rows see only partly:
// positions behind the last count as zeros, and so do values that are not
// finite, which must not reach the rows that do not see them (the others read
// NaN); 4-7 and 8-11 the softmax of the tiles. The products of one tile run
// under the other's softmax. Where few CTAs would leave SMs idle, W CTAs of a
// cluster share the positions of one pair of tiles and merge through distributed
// shared memory.
#include <math.h>

#include <mutex>

#include "m2_dense_dev.cuh"
#include "m2_tc.cuh"
#include "m2_tile_meet.h"

namespace m2 {

namespace {

constexpr int kPtThreads = 384;
constexpr int kPtRows = 128;                       // rows of a tile
constexpr int kPtPos = 128;                        // positions a chunk
constexpr uint32_t kPtPanel = 128 * 128;           // 128 rows x 64 dims of bf16
constexpr uint32_t kPtTile = 2 * kPtPanel;
constexpr int kPtStages = 5;                       // of a chunk's K or V, in turn
constexpr float kPtSlack = 8.f;                    // log2 by which a chunk may exceed m
constexpr int kPtCut = 3;                          // chunks that the tiles' at most 256 packed rows see partly, at most
constexpr uint32_t kColO = 0, kColS = 256;         // tensor memory: O of the two tiles, then S (and p over it)

struct PtSmem {
    static constexpr uint32_t kQ = 0;                                // [tile][panel] K-major
    static constexpr uint32_t kRing = kQ + 2 * kPtTile;              // K: K-major, V: MN-major; two panels each
    static constexpr uint32_t kBar = kRing + kPtStages * kPtTile;
    // full[stages], empty[stages], q, cutfull[cut], mended[cut], s[2], o[2], end
    static constexpr int kBars = 2 * kPtStages + 2 * kPtCut + 6;
    static constexpr uint32_t kBad = kBar + kBars * 8;               // values that are not finite: a bit a position
    static constexpr uint32_t kTmem = kBad + kPtCut * 16;
    static constexpr uint32_t kFlag = kTmem + 4;
    static constexpr uint32_t kWork = kFlag + 4;                     // session, its first packed row, rows, positions before, pair
    static constexpr uint32_t kBytes = kWork + 5 * 4 + 1024;         // + slack to align to 1024
    // after the walk, over the ring: 256 rows x 128 floats, then their (m, l)
    static constexpr uint32_t kMl = kRing + 2 * kPtRows * kAttnD * 4;
    static_assert(kMl + 2 * kPtRows * 8 <= kBar, "the merge fits in the ring");
    static_assert(kBytes <= 227 * 1024, "one CTA an SM");
};

constexpr int kRegsLaunch = 168, kRegsFew = 72, kRegsMany = 216;
static_assert(128 * kRegsFew + 256 * kRegsMany <= kPtThreads * kRegsLaunch, "the split is covered by the launch's registers");
// the threads of a tile's softmax; of both tiles'
__device__ __forceinline__ void tile_sync(int i) { asm volatile("barrier.sync %0, 128;" ::"r"(4 + i) : "memory"); }
__device__ __forceinline__ void tiles_sync() { asm volatile("barrier.sync 6, 256;" ::: "memory"); }

// A box of shared memory out to a tensor map's coordinates.
__device__ __forceinline__ void tma_store_3d(const void* tmap, int x, int y, int z, const void* src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(tmap), "r"(x),
                 "r"(y), "r"(z), "r"(tc::smem_u32(src))
                 : "memory");
}

// The pair of tiles `at` of all the sessions' pairs of `per` packed rows each,
// found by a warp, eight sessions a lane at a time (a session's last pair first:
// it sees the most positions). A session whose rows do not lie within the call's
// has none, and is recorded.
__device__ __forceinline__ bool find_pair(const PromptArgs& a, int per, int at, Session* x, int* session, int* pair) {
    constexpr int kEach = 8;
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int s0 = 0; s0 < a.S; s0 += 32 * kEach) {
        int b[kEach + 1], before[kEach], n[kEach], mine = 0;
        const int first = s0 + lane * kEach;
#pragma unroll
        for (int i = 0; i <= kEach; ++i) b[i] = first + i <= a.S ? a.start[first + i] : 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) before[i] = a.lens && first + i < a.S ? a.lens[first + i] : 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            n[i] = 0;
            if (first + i < a.S) {
                if (b[i] < 0 || b[i + 1] < b[i] || b[i + 1] > a.rows)
                    record_error(a.err, ERR_ROW_START);
                else
                    n[i] = (b[i + 1] - b[i] + per - 1) / per;
            }
            mine += n[i];
        }
        int upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int below = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += below;
        }
        int ahead = base + upto - mine;
        int v[5] = {-1, 0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (at >= ahead && at < ahead + n[i])
                v[0] = first + i, v[1] = b[i], v[2] = b[i + 1] - b[i], v[3] = before[i], v[4] = n[i] - 1 - (at - ahead);
            ahead += n[i];
        }
        const unsigned who = __ballot_sync(0xffffffffu, v[0] >= 0);
        if (who) {
            const int from = __ffs(who) - 1;
            *session = __shfl_sync(0xffffffffu, v[0], from);
            x->row0 = __shfl_sync(0xffffffffu, v[1], from);
            x->n = __shfl_sync(0xffffffffu, v[2], from);
            x->before = __shfl_sync(0xffffffffu, v[3], from);
            *pair = __shfl_sync(0xffffffffu, v[4], from);
            return true;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}

// The merge of a cluster's W parts of the rows that CTA wk owns, a warp a row,
// four dims a lane:
//     out = sum_w 2^(m_w - M) O_w / sum_w 2^(m_w - M) l_w
__device__ __forceinline__ void merge_rows(const PromptArgs& a, uint8_t* sm, int W, int wk, int row_end, const Session& x, int t0,
                                           int per, int g) {
    const int lane = threadIdx.x & 31, R = a.Hq / a.Hkv, share = 2 * kPtRows / W;
    const uint32_t here = tc::smem_u32(sm);
    for (int i = (int)(threadIdx.x >> 5); i < share; i += kPtThreads / 32) {
        const int row = wk * share + i, tile = row >> 7, r = row & 127, t = t0 + tile * per + r / R;
        if (r >= per * R || t >= row_end) continue;  // (the same in the whole warp)
        float m = kNone, l = 0.f;
        if (lane < W) {
            const float2 ml = ld_cluster_f32x2(tc::cluster_map(here, (uint32_t)lane) + PtSmem::kMl + row * 8);
            m = ml.x, l = ml.y;
        }
        float M = m;
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        M = __shfl_sync(0xffffffffu, M, 0);
        const float f = lane < W ? ex2_approx(m - M) : 0.f;
        float L = f * l;
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
        L = __shfl_sync(0xffffffffu, L, 0);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < W; ++w) {
            const float fw = __shfl_sync(0xffffffffu, f, w);
            const float4 v = ld_cluster_f32x4(tc::cluster_map(here, (uint32_t)w) + PtSmem::kRing + row * kAttnD * 4 +
                                              (((lane + row) & 31) << 4));
            o.x = fmaf(fw, v.x, o.x), o.y = fmaf(fw, v.y, o.y), o.z = fmaf(fw, v.z, o.z), o.w = fmaf(fw, v.w, o.w);
        }
        const float inv = 1.f / L;
        const size_t packed = (size_t)x.row0 + t;
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + packed * a.out_stride + (size_t)(g * R + r % R) * kAttnD +
                                  4 * lane) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (a.lse && lane == 0) a.lse[packed * a.Hq + g * R + r % R] = fmaf(M, kLn2, logf(L));
    }
}

// grid (W x Hkv x pairs of tiles), a cluster of W CTAs when W > 1
__global__ void __launch_bounds__(kPtThreads, 1)
    attn_prompt_tile_kernel(PromptArgs a, const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                            const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmo, int W) {
    using L = PtSmem;
    extern __shared__ uint8_t pt_raw[];
    uint8_t* sm = pt_raw + ((1024u - (tc::smem_u32(pt_raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint64_t *empty = full + kPtStages, *qbar = empty + kPtStages, *cutfull = qbar + 1, *mended = cutfull + kPtCut,
             *sfull = mended + kPtCut, *ofull = sfull + 2, *endbar = ofull + 2;
    uint32_t* sBad = reinterpret_cast<uint32_t*>(sm + L::kBad);
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + L::kTmem);
    volatile uint32_t* flag = reinterpret_cast<uint32_t*>(sm + L::kFlag);
    int* work = reinterpret_cast<int*>(sm + L::kWork);
    const int wk = (int)blockIdx.x % W, g = (int)blockIdx.x / W % a.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int R = a.Hq / a.Hkv, per = kPtRows / R;  // packed rows a tile

    if (W > 1) tc::cluster_arrive_relaxed();  // waited on before the first remote access: every CTA has started
    // Which rows: warp 0, which then sets the first copies going, while warp 1 takes the tensor
    // memory. (The kernel before this one is this call's append, which has waited for what
    // came before: only the caches are its own.)
    if (warp == 0) {
        if (lane == 0) {
            prefetch_map(&tmq), prefetch_map(&tmk), prefetch_map(&tmv);
            for (int i = 0; i < kPtStages; ++i) tc::mbar_init(full + i, 1), tc::mbar_init(empty + i, 1);
            tc::mbar_init(qbar, 1);
            for (int i = 0; i < kPtCut; ++i) tc::mbar_init(cutfull + i, 1), tc::mbar_init(mended + i, 1);
            for (int i = 0; i < 2; ++i) tc::mbar_init(sfull + i, 1), tc::mbar_init(ofull + i, 1);
            tc::mbar_init(endbar, 1);
            tc::fence_mbar_init();
            *flag = 0;
        }
        Session y;
        int s = -1, pair = 0;
        if (!find_pair(a, 2 * per, (int)blockIdx.x / W / a.Hkv, &y, &s, &pair)) s = -1;
        if (lane == 0) work[0] = s, work[1] = y.row0, work[2] = y.n, work[3] = y.before, work[4] = pair;
    } else if (warp == 1) {
        tc::tmem_alloc(sTmem, 512);
        tc::tmem_relinquish();
    } else if (tid - 64 < kPtCut * 4) {
        sBad[tid - 64] = 0u;
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = *sTmem;
    const int s = work[0];
    Session x;
    x.row0 = work[1], x.n = work[2], x.before = work[3];
    x.ok = s >= 0 && x.before >= 0 && (long)x.before + x.n <= a.Tmax;
    const int t0 = work[4] * 2 * per, row_end = min(t0 + 2 * per, x.n);  // the pair's packed rows of the session
    pdl_wait();     // the append, and with it what it waited for
    pdl_trigger();  // not before the tensor memory is held: the next kernel may take some before it waits for this one
    if (!x.ok) {  // the whole cluster
        if (warp == 1) tc::tmem_dealloc(tm, 512);
        if (s < 0 || wk) return;  // (past the last pair: nothing to do)
        if (tid == 0) record_error(a.err, ERR_ATTN_LENGTH);
        const int rows = (row_end - t0) * R;
        for (int i = tid; i < rows * (kAttnD / 8); i += kPtThreads) {
            const int row = i / (kAttnD / 8);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (size_t)(x.row0 + t0 + row / R) * a.out_stride +
                                      (size_t)(g * R + row % R) * kAttnD + i % (kAttnD / 8) * 8) = make_uint4(0u, 0u, 0u, 0u);
        }
        if (a.lse)
            for (int row = tid; row < rows; row += kPtThreads)
                a.lse[(size_t)(x.row0 + t0 + row / R) * a.Hq + g * R + row % R] = -INFINITY;
        return;
    }
    const int all = x.before + t0 + 1;          // positions that every row sees
    const int total = x.before + row_end;       // ... and that the last one does
    const int total0 = x.before + min(t0 + per, row_end);  // ... of tile 0
    // this CTA's run of chunks cb .. cb + nc - 1, of which tile 0 takes nc0 and tile 1 nc1
    const int nch = (total + kPtPos - 1) / kPtPos, cpw = (nch + W - 1) / W;
    const int cb = min(wk * cpw, nch), nc = min(cpw, nch - cb);
    const int nc0 = min(max((total0 + kPtPos - 1) / kPtPos - cb, 0), nc);
    const int nc1 = row_end > t0 + per ? nc : 0;
    const int cut = max(all / kPtPos, cb);      // the first of the run's chunks that is not whole for every row

    // A bounded wait; the first that runs out stops the CTA's work.
    auto wait_ok = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (tc::mbar_try_wait(bar, parity)) return true;
        if (*flag) return false;
        if (tc::mbar_wait(bar, parity)) return true;
        record_error(a.err, ERR_MBAR_TIMEOUT_MMA);
        *flag = 1;
        return false;
    };
    // the same for a converged warp
    auto warp_ok = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait_ok(bar, parity)); };
    // K of the run's chunk j is the ring's piece 2 j, V 2 j + 1
    auto stage = [](int piece) { return piece % kPtStages; };
    auto phase = [](int piece) { return (uint32_t)(piece / kPtStages) & 1u; };

    float m = kNone, l = 0.f;  // of a softmax thread's row
    if (warp < 4) {
        regs_down<kRegsFew>();
        if (warp == 0) {
            // ------------------------------------------------------------ copies
            if (nc > 0) {
                if (tc::elect_one()) {
                    const int boxes = nc1 > 0 ? 2 : 1;
                    tc::mbar_arrive_expect_tx(qbar, (uint32_t)(boxes * 2 * per * R * 128));
                    for (int i = 0; i < boxes; ++i)
                        for (int h = 0; h < 2; ++h)
                            tc::tma_load_3d(sm + L::kQ + i * kPtTile + h * kPtPanel, &tmq, 64 * h, g * R, x.row0 + t0 + i * per, qbar);
                }
                __syncwarp();
                for (int piece = 0; piece < 2 * nc; ++piece) {
                    if (piece >= kPtStages && !warp_ok(empty + stage(piece), phase(piece - kPtStages))) break;
                    if (tc::elect_one()) {
                        uint8_t* to = sm + L::kRing + stage(piece) * kPtTile;
                        const int c = cb + (piece >> 1);
                        // The values that warp 3 mends are announced to it alone. (They are among the last five
                        // pieces, so that no later one waits for the barrier of their stage.)
                        uint64_t* landed = (piece & 1) && c >= cut ? cutfull + (c - cut) : full + stage(piece);
                        tc::mbar_arrive_expect_tx(landed, kPtTile);
                        for (int h = 0; h < 2; ++h)
                            tc::tma_load_3d(to + h * kPtPanel, piece & 1 ? &tmv : &tmk, 64 * h, c * kPtPos, s * a.Hkv + g, landed);
                    }
                    __syncwarp();
                }
            }
        } else if (warp == 1) {
            // ---------------------------------------------------------- products
            const bool leader = tc::elect_one();
            const uint32_t sbase = tc::smem_u32(sm);
            tile_turns_meet(TileBarriers(), nc, nc0, nc1, [](int) {}, [&](int i, int j) {
                const int nci = i ? nc1 : nc0;
                const bool last = i == 1 || nc1 == 0;  // of the tiles that read this chunk (tile 1 takes every one, where there is one)
                tc::tc_fence_after();
                if (leader) {
                    if (j > 0) {  // O += p V of chunk j - 1
                        const int at = stage(2 * j - 1);
                        const uint64_t bd = tc::sdesc(sbase + L::kRing + at * kPtTile, kPtPanel, 1024, 2);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            tc::mma_bf16_tmem_a(tm + kColO + 128 * i, tm + kColS + 128 * i + 8 * k, bd + (uint64_t)(k * 2048 >> 4),
                                                tc::idesc_bf16(kPtRows, kAttnD, 0, 1), (j > 1 || k > 0) ? 1u : 0u);
                        if (last) tc::mma_commit(empty + at);
                    }
                    if (j < nci) {  // S = q K^T of chunk j, over the weights
                        const int at = stage(2 * j);
                        const uint64_t ad = tc::sdesc(sbase + L::kQ + i * kPtTile, 0, 1024, 2);
                        const uint64_t bd = tc::sdesc(sbase + L::kRing + at * kPtTile, 0, 1024, 2);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint64_t off = (uint64_t)(((k >> 2) * kPtPanel + (k & 3) * 32) >> 4);
                            tc::mma_bf16(tm + kColS + 128 * i, ad + off, bd + off, tc::idesc_bf16(kPtRows, kPtPos, 0, 0),
                                         k > 0 ? 1u : 0u);
                        }
                        tc::mma_commit(sfull + i);
                        if (last) tc::mma_commit(empty + at);
                    } else {
                        tc::mma_commit(ofull + i);
                    }
                }
                __syncwarp();
            });
        } else if (warp == 2) {
            // ------- waits for the operands from memory on behalf of the products
            // (after one that gave up, what the products read is there, if not what it should be,
            // and the CTA's results are dropped)
            bool good = true;
            tile_turns_meet(TileBarriers(), nc, nc0, nc1, [&](int j) {
                if (j == 0) good = good && warp_ok(qbar, 0);
                if (j < nc) good = good && warp_ok(full + stage(2 * j), phase(2 * j));
                if (j > 0) {
                    const int c = j - 1;
                    if (cb + c >= cut)
                        good = good && warp_ok(mended + (cb + c - cut), 0);
                    else
                        good = good && warp_ok(full + stage(2 * c + 1), phase(2 * c + 1));
                }
            }, [](int, int) {});
        } else {
            // ------------------------------------ values of the chunks cut .. the last
            for (int j = cut - cb; j < nc; ++j) {
                const int piece = 2 * j + 1;
                if (!warp_ok(cutfull + (cb + j - cut), 0)) break;
                uint8_t* v = sm + L::kRing + stage(piece) * kPtTile;
                // positions of the chunk from `from` on are not seen by every row, and there is nothing from
                // `left` on; lanes 0 .. 15 have the 16 pieces of a position, 16 .. 31 of the next
                const int from = max(all - (cb + j) * kPtPos, 0), left = min(total - (cb + j) * kPtPos, kPtPos);
                uint32_t* bad = sBad + 4 * (cb + j - cut);
                uint8_t* mine = v + (lane & 7) * 16 + ((lane >> 3) & 1) * kPtPanel;
                for (int p0 = from + (lane >> 4); p0 < left; p0 += 16) {
                    uint4 w[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (p0 + 2 * k < left) w[k] = *reinterpret_cast<const uint4*>(mine + (p0 + 2 * k) * 128);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (p0 + 2 * k >= left) break;
                        const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
                        bool off = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e) off |= (u[e] & 0x7F80u) == 0x7F80u || (u[e] & 0x7F800000u) == 0x7F800000u;
                        if (off) {
                            *reinterpret_cast<uint4*>(mine + (p0 + 2 * k) * 128) = make_uint4(0u, 0u, 0u, 0u);
                            atomicOr(bad + ((p0 + 2 * k) >> 5), 1u << ((p0 + 2 * k) & 31));
                        }
                    }
                }
                for (int p = left + (lane >> 4); p < kPtPos; p += 2)
                    *reinterpret_cast<uint4*>(mine + p * 128) = make_uint4(0u, 0u, 0u, 0u);
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(mended + (cb + j - cut));
            }
        }
    } else {
        // ------------------------------------------ softmax, one row a thread
        regs_up<kRegsMany>();
        const int i = (warp - 4) >> 2, r = tid - 128 - 128 * i;  // tile, row of it
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tm + lanes + kColS + 128 * i, tO = tm + lanes + kColO + 128 * i;
        const int t = t0 + i * per + r / R;
        // The last position seen. (A row behind the tile's last goes with what the last one sees:
        // hiding all from it took its warp 700 cycles more a chunk, and 80 us of the size below.)
        const int lim = min(x.before + t, total - 1);
        const int nci = i ? nc1 : nc0;
        const float cs = fmaxf(fabsf(a.scale) * kLog2e, FLT_MIN);  // not 0: hidden scores are -inf
        bool good = true;
        if (a.scale < 0.f && nci > 0) {  // the sign goes into the queries: the maxima are those of S
            good = warp_ok(qbar, 0);
#pragma unroll 1
            for (int e = 0; e < 16; ++e) {
                uint4* q = reinterpret_cast<uint4*>(sm + L::kQ + i * kPtTile + (e >> 3) * kPtPanel + r * 128) + (e & 7);
                uint4 w = *q;
                w.x ^= 0x80008000u, w.y ^= 0x80008000u, w.z ^= 0x80008000u, w.w ^= 0x80008000u;
                *q = w;
            }
            tc::fence_proxy_async_smem();
        }
        float2 l0 = make_float2(0.f, 0.f), l1 = l0;  // the row's sum, in four parts
        // the weights of the run's chunk j from its scores
        auto softmax_chunk = [&](int j) -> bool {
            if (!warp_ok(sfull + i, (uint32_t)j & 1)) return false;
            tc::tc_fence_after();
            const int see = lim - (cb + j) * kPtPos;  // columns 0 .. see are seen
            const bool part = __any_sync(0xffffffffu, see < kPtPos - 1);
            float v[kPtPos], tops[8];  // the scores, and their maxima
#pragma unroll
            for (int b = 0; b < 8; ++b) tmem_ld16_max(tS + 16 * b, v + 16 * b, tops[b]);
            tc::tmem_wait_ld();
            if (part) {
#pragma unroll
                for (int k = 0; k < kPtPos; ++k) v[k] = k <= see ? v[k] : -INFINITY;
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const float* w = v + 16 * b;
                    tops[b] = max3(max3(max3(w[0], w[1], w[2]), max3(w[3], w[4], w[5]), max3(w[6], w[7], w[8])),
                                   max3(w[9], w[10], w[11]), max3(fmaxf(w[12], w[13]), w[14], w[15]));
                }
            }
            const float mx = max3(max3(tops[0], tops[1], tops[2]), max3(tops[3], tops[4], tops[5]), fmaxf(tops[6], tops[7])) * cs;
            const bool grow = mx > m + kPtSlack;
            const float f = grow ? ex2_approx(m - mx) : 1.f;
            if (grow) {
                l0.x *= f, l0.y *= f, l1.x *= f, l1.y *= f;
                m = mx;
            }
            if (j > 0 && __any_sync(0xffffffffu, grow)) {  // O is idle: its products came before S
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    float o[2][16];
                    tc::tmem_ld16(tO + 32 * q, o[0]);
                    tc::tmem_ld16(tO + 32 * q + 16, o[1]);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t y[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(o[h][k] * f);
                        tmem_st16(tO + 32 * q + 16 * h, y);
                    }
                }
            }
            const float2 nm = make_float2(-m, -m), c2 = make_float2(cs, cs);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t y[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float2 e = fma2(make_float2(v[32 * q + 2 * k], v[32 * q + 2 * k + 1]), c2, nm);
                    const float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
                    if (k & 1)
                        l1 = add2(l1, p);
                    else
                        l0 = add2(l0, p);
                    y[k] = pack_bf16x2(p.x, p.y);
                }
                tmem_st16(tS + 16 * q, y);  // over S, which is read
            }
            tc::tmem_wait_st();
            return true;
        };
        tc::tc_fence_before();
        tile_rows_meet(TileBarriers(), i, nci, [&](int j) {
            good = good && softmax_chunk(j);
            tc::tc_fence_before();
        });
        l = (l0.x + l0.y) + (l1.x + l1.y);
        good = good && (nci == 0 || warp_ok(ofull + i, 0));
        tc::tc_fence_after();
        // ------------------------------------------------------------ O out
        const bool some = good && nci > 0;  // (the same in the whole warp)
        const bool live = r < per * R && t < row_end;
        if (!some) m = kNone, l = 0.f;
        float poison = 0.f;  // NaN where the row sees a value that was not finite
        for (int c = cut; c < cb + nc; ++c)
            for (int w = 0; w < 4; ++w) {
                const int see = lim - c * kPtPos - 32 * w;
                const uint32_t off = sBad[4 * (c - cut) + w];
                if (off && see >= 0 && (off & (see >= 31 ? ~0u : (2u << see) - 1u))) poison = NAN;
            }
        const size_t packed = (size_t)x.row0 + t;
        if (W == 1) {
            // in bf16 over the tile's queries, laid out as they were; a whole tile leaves by two copies
            // of a thread, the last of a session two rows at a time (16 lanes a row)
            const float f = 1.f / l + poison;
            uint8_t* own = sm + L::kQ + i * kPtTile + r * 128;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[32];
                tmem_ld32(tO + 32 * q, v);
                tc::tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(v[k + 2 * e] * f, v[k + 2 * e + 1] * f);
                    *reinterpret_cast<uint4*>(own + (q >> 1) * kPtPanel + (((4 * (q & 1) + k / 8) ^ (r & 7)) << 4)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (live && a.lse) a.lse[packed * a.Hq + g * R + r % R] = fmaf(m, kLn2, logf(l));
            if (t0 + (i + 1) * per <= row_end) {
                tc::fence_proxy_async_smem();
                tile_sync(i);
                if ((tid & 127) == 0) {
                    for (int h = 0; h < 2; ++h)
                        tma_store_3d(&tmo, 64 * h, g * R, x.row0 + t0 + i * per, sm + L::kQ + i * kPtTile + h * kPtPanel);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                }
            } else {
                __syncwarp();
                const size_t at = packed * a.out_stride + (size_t)(g * R + r % R) * kAttnD;
                const unsigned lives = __ballot_sync(0xffffffffu, live);
#pragma unroll 4
                for (int e = 0; e < 16; ++e) {
                    const int rr = 2 * e + (lane >> 4), piece = lane & 15;
                    const size_t to = __shfl_sync(0xffffffffu, at, rr);
                    if (lives >> rr & 1u)
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + to + 8 * piece) =
                            *reinterpret_cast<const uint4*>(sm + L::kQ + i * kPtTile + (piece >> 3) * kPtPanel +
                                                            ((r & ~31) + rr) * 128 + (((piece & 7) ^ (rr & 7)) << 4));
                }
            }
        } else {
            tiles_sync();  // the ring is read: the tiles' products are done
            const int row = 128 * i + r;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                float v[32];
                if (some) {
                    tmem_ld32(tO + 32 * q, v);
                    tc::tmem_wait_ld();
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = 0.f;
                }
                // 16-byte pieces rotated by the row, so that a warp's rows do not meet in one bank
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<float4*>(sm + L::kRing + row * kAttnD * 4 + (((8 * q + k + row) & 31) << 4)) =
                        make_float4(v[4 * k] + poison, v[4 * k + 1] + poison, v[4 * k + 2] + poison, v[4 * k + 3] + poison);
            }
            *reinterpret_cast<float2*>(sm + L::kMl + row * 8) = make_float2(m, l);
        }
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    if (*flag) {  // (the same in the whole CTA)
        // the copies in flight must land and every product issued must be done
        // before the tensor memory is freed and the CTA exits (all bounded)
        if (warp == 0 && tc::elect_one()) {
            tc::mbar_wait(qbar, 0, 100000000ull);
            for (int i = 0; i < kPtStages; ++i)
                tc::mbar_wait(full + i, 0, 100000000ull), tc::mbar_wait(full + i, 1, 100000000ull);
            for (int i = 0; i < kPtCut; ++i) tc::mbar_wait(cutfull + i, 0, 100000000ull);
        } else if (warp == 1 && tc::elect_one()) {
            tc::mma_commit(endbar);
            tc::mbar_wait(endbar, 0, 100000000ull);
        }
        __syncthreads();
    }
    if (warp == 1) tc::tmem_dealloc(tm, 512);
    if (W == 1) return;
    tc::cluster_wait();    // (pairs with the arrival at the start)
    tc::cluster_arrive();  // every CTA's rows are in its shared memory ...
    tc::cluster_wait();
    merge_rows(a, sm, W, wk, row_end, x, t0, per, g);  // ... and each reads the rows that it owns
    tc::cluster_arrive();  // nobody leaves while its memory is read
    tc::cluster_wait();
}

// Per device, once: the kernel's attributes, and how many clusters of 1, 2, 4
// and 8 CTAs the device holds at once.
struct PtSetup {
    bool done;
    int held[4];
};

cudaError_t prompt_setup(const PtSetup** out) {
    static std::mutex mutex;
    static PtSetup per_device[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mutex);
    PtSetup& u = per_device[dev & 63];
    if (!u.done) {
        // the warps' register split draws on what the launch gives
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, attn_prompt_tile_kernel);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < kRegsLaunch) return cudaErrorLaunchOutOfResources;
        e = cudaFuncSetAttribute(attn_prompt_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PtSmem::kBytes);
        if (e != cudaSuccess) return e;
        u.held[0] = 152;
        for (int k = 1; k < 4; ++k) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(1u << k);
            cfg.blockDim = dim3(kPtThreads);
            cfg.dynamicSmemBytes = PtSmem::kBytes;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1u << k;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int held = 0;
            if (cudaOccupancyMaxActiveClusters(&held, attn_prompt_tile_kernel, &cfg) != cudaSuccess) held = 0;
            u.held[k] = held;
        }
        (void)cudaGetLastError();  // a refused query leaves no sticky error
        u.done = true;
    }
    *out = &u;
    return cudaSuccess;
}

// bf16 rows of 128 dims as [outer][middle][128], boxes of 64 dims x mid x out.
cudaError_t make_map(const void* p, cuuint64_t mid, cuuint64_t out, cuuint64_t mid_bytes, cuuint64_t out_bytes, int box_mid,
                     int box_out, CUtensorMap* map) {
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

}  // namespace

cudaError_t launch_attn_prompt_tiles(const PromptArgs& a, cudaStream_t st) {
    const PtSetup* setup = nullptr;
    cudaError_t e = prompt_setup(&setup);
    if (e != cudaSuccess) return e;
    const int R = a.Hq / a.Hkv, per = kPtRows / R;
    CUtensorMap tmq, tmk, tmv, tmo;
    const cuuint64_t row = kAttnD * 2;
    e = make_map(a.q, a.Hq, a.rows, row, (cuuint64_t)a.q_stride * 2, R, per, &tmq);
    if (e == cudaSuccess) e = make_map(a.k_cache, a.Tmax, (cuuint64_t)a.S * a.Hkv, row, row * a.Tmax, kPtPos, 1, &tmk);
    if (e == cudaSuccess) e = make_map(a.v_cache, a.Tmax, (cuuint64_t)a.S * a.Hkv, row, row * a.Tmax, kPtPos, 1, &tmv);
    if (e == cudaSuccess) e = make_map(a.out, a.Hq, a.rows, row, (cuuint64_t)a.out_stride * 2, R, per, &tmo);
    if (e != cudaSuccess) return e;
    const long pairs = most_tiles(a.S, a.rows, 2 * per) * a.Hkv;
    int W = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(W * pairs));
    cfg.blockDim = dim3(kPtThreads);
    cfg.dynamicSmemBytes = PtSmem::kBytes;
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
    return cudaLaunchKernelEx(&cfg, attn_prompt_tile_kernel, a, tmq, tmk, tmv, tmo, W);
}

}  // namespace m2
