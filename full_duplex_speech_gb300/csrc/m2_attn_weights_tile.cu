// The weights that cached positions receive from a packed prompt, in bf16 on the
// tcgen05 tensor cores (the operator and its formulas are those of
// m2_attn_weights.cu).
//
// One CTA takes 256 positions of one (session, kv head), two tiles of 128, and
// walks the window's rows that see any of them, up to 256 (row, head) pairs at a
// time: two tiles of floor(128 / R) packed rows, each a box of a tensor map. Per
// step and tile of positions:
//   S^T = K Q^T     kind::f16, M 128 positions x N 256 pairs, so that an operand
//                   is read from shared memory at 96 bytes a cycle of the 128
//                   that it gives (two products of N 128 need all of them);
//   sum += e^(S scale - lse)    one thread a position: a pair's lse is the same for
//                   all threads (read by broadcast), and the sum over the pairs
//                   stays in the thread, added up step by step in a fixed order.
//                   The exponent is S (scale log2 e) -
//                   (lse log2 e), the second product rounded once for all.
// The products of one tile run under the other's exponentials.
//
// Warps: 0 copies keys once and queries through a ring, 1 issues the products, 2
// fetches the rows' lse, 4-7 and 8-11 the sums of the tiles of positions: 32 pairs
// at a time, while the next 32 products and lse are on their way. (Shared memory
// answers late beside the products' own reads of it: four warps more a tile that
// waited for each other's 32 took 313 us where this takes XXX.)
#include <math.h>

#include "m2_dense_dev.cuh"
#include "m2_tc.cuh"

namespace m2 {

namespace {

constexpr int kWtThreads = 384;
constexpr int kWtPos = 128;                        // positions a tile
constexpr uint32_t kWtPanel = 128 * 128;           // 128 rows x 64 dims of bf16
constexpr uint32_t kWtKeys = 2 * kWtPanel;
constexpr uint32_t kWtStage = 4 * kWtPanel;        // 256 rows of queries
constexpr int kWtStages = 2;
constexpr int kWtRaw = 4;                          // steps whose lse is on its way

struct WtSmem {
    static constexpr uint32_t kK = 0;                                 // [tile][panel] K-major, 128-byte swizzle
    static constexpr uint32_t kQ = kK + 2 * kWtKeys;                  // [stage][panel][256 rows], likewise
    static constexpr uint32_t kL = kQ + kWtStages * kWtStage;         // float [stage][256]: the pairs' -lse log2 e
    static constexpr uint32_t kRaw = kL + kWtStages * 256 * 4;                // float [kWtRaw][256]: lse on its way
    static constexpr uint32_t kBar = kRaw + kWtRaw * 256 * 4;
    // k, qfull[stages], qempty[stages], lfull[stages], lempty[stages], d[2], dempty[2], end
    static constexpr int kBars = 4 * kWtStages + 6;
    static constexpr uint32_t kTmem = kBar + kBars * 8;
    static constexpr uint32_t kFlag = kTmem + 4;
    static constexpr uint32_t kBytes = kFlag + 4 + 1024;              // + slack to align to 1024
    static_assert(kBytes <= 227 * 1024, "one CTA an SM");
};

// grid: (position tiles of 256) x Hkv x S, the first tiles, which most rows see, first
__global__ void __launch_bounds__(kWtThreads, 1)
    attn_weights_tile_kernel(PromptArgs a, PromptSums w, const __grid_constant__ CUtensorMap tmq,
                             const __grid_constant__ CUtensorMap tmk) {
    using L = WtSmem;
    extern __shared__ uint8_t wt_raw[];
    uint8_t* sm = wt_raw + ((1024u - (tc::smem_u32(wt_raw) & 1023u)) & 1023u);
    float* sL = reinterpret_cast<float*>(sm + L::kL);
    uint64_t* kbar = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint64_t *qfull = kbar + 1, *qempty = qfull + kWtStages, *lfull = qempty + kWtStages, *lempty = lfull + kWtStages,
             *dfull = lempty + kWtStages, *dempty = dfull + 2, *endbar = dempty + 2;
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + L::kTmem);
    volatile uint32_t* flag = reinterpret_cast<uint32_t*>(sm + L::kFlag);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int R = a.Hq / a.Hkv, per = 128 / R;  // packed rows a tile of pairs
    const int heads = a.Hkv * a.S, p0 = (int)(blockIdx.x / heads) * 2 * kWtPos;
    const int g = blockIdx.x % heads % a.Hkv, s = blockIdx.x % heads / a.Hkv;

    if (tid == 0) prefetch_map(&tmq), prefetch_map(&tmk);
    pdl_wait();
    Session x;
    const bool rows_ok = session_of(a, s, &x);
    if (!rows_ok || !x.ok) {
        if (tid == 0 && p0 == 0) record_error(a.err, rows_ok ? ERR_ATTN_LENGTH : ERR_ROW_START);
        return;
    }
    const int total = x.before + x.n;
    if (p0 >= total) return;
    // the window's rows that see a position of the CTA: first .. n - 1, in steps of 2 per
    const int first = max(max(0, x.n - w.window), p0 - x.before);
    const int steps = first < x.n ? (x.n - first + 2 * per - 1) / (2 * per) : 0;
    const int tiles = p0 + kWtPos < total ? 2 : 1;  // of positions
    const size_t head = ((size_t)s * a.Hkv + g) * a.Tmax;

    if (tid == 0) {
        tc::mbar_init(kbar, 1);
        for (int i = 0; i < kWtStages; ++i) {
            tc::mbar_init(qfull + i, 1), tc::mbar_init(qempty + i, 1);
            tc::mbar_init(lfull + i, 1), tc::mbar_init(lempty + i, 4 * tiles);
        }
        for (int i = 0; i < 2; ++i) tc::mbar_init(dfull + i, 1), tc::mbar_init(dempty + i, 4);
        tc::mbar_init(endbar, 1);
        tc::fence_mbar_init();
        *flag = 0;
    }
    if (warp == 1) {
        tc::tmem_alloc(sTmem, 512);
        tc::tmem_relinquish();
    }
    // Rows of a tile of pairs that no packed row fills: zeros (and an lse that gives them no weight).
    if (warp >= 4) {
        const int dead = 128 - per * R, each = dead * 8;  // 16-byte pieces of a tile's panel
        for (int i = tid - 128; i < kWtStages * 4 * each; i += kWtThreads - 128) {
            const int panel = i / each, row = per * R + i % each / 8;  // (stage, panel, tile)
            *reinterpret_cast<uint4*>(sm + L::kQ + panel * kWtPanel + row * 128 + i % 8 * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        tc::fence_proxy_async_smem();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = *sTmem;
    pdl_trigger();  // not before the tensor memory is held: the next kernel may take some before it waits for this one

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
    auto stage = [](int j) { return j % kWtStages; };
    auto phase = [](int j) { return (uint32_t)(j / kWtStages) & 1u; };
    // tiles of pairs of step j that have rows
    auto filled = [&](int j) { return first + (2 * j + 1) * per < x.n ? 2 : 1; };

    float sum = 0.f;
    if (warp == 0) {
        // ---------------------------------------------------------------- copies
        if (steps > 0 && tc::elect_one()) {
            tc::mbar_arrive_expect_tx(kbar, (uint32_t)tiles * kWtKeys);
            for (int i = 0; i < tiles; ++i)
                for (int h = 0; h < 2; ++h)
                    tc::tma_load_3d(sm + L::kK + i * kWtKeys + h * kWtPanel, &tmk, 64 * h, p0 + i * kWtPos, s * a.Hkv + g, kbar);
        }
        __syncwarp();
        for (int j = 0; j < steps; ++j) {
            if (j >= kWtStages && !warp_ok(qempty + stage(j), phase(j - kWtStages))) break;
            if (tc::elect_one()) {
                const int n = filled(j);
                tc::mbar_arrive_expect_tx(qfull + stage(j), (uint32_t)(n * 2 * per * R * 128));
                for (int i = 0; i < n; ++i)
                    for (int h = 0; h < 2; ++h)
                        tc::tma_load_3d(sm + L::kQ + stage(j) * kWtStage + (2 * h + i) * kWtPanel, &tmq, 64 * h, g * R,
                                        x.row0 + first + (2 * j + i) * per, qfull + stage(j));
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        // -------------------------------------------------------------- products
        const bool leader = tc::elect_one();
        const uint32_t sbase = tc::smem_u32(sm);
        bool good = steps > 0 && warp_ok(kbar, 0);
        for (int j = 0; good && j < steps; ++j) {
            good = warp_ok(qfull + stage(j), phase(j));
            for (int i = 0; good && i < tiles; ++i) {
                if (j > 0) good = warp_ok(dempty + i, (uint32_t)(j - 1) & 1u);
                if (!good) break;
                tc::tc_fence_after();
                if (leader) {
                    const uint64_t ad = tc::sdesc(sbase + L::kK + i * kWtKeys, 0, 1024, 2);
                    const uint64_t bd = tc::sdesc(sbase + L::kQ + stage(j) * kWtStage, 0, 1024, 2);
                    const uint32_t id = filled(j) == 2 ? tc::idesc_bf16(128, 256, 0, 0) : tc::idesc_bf16(128, 128, 0, 0);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        tc::mma_bf16(tm + 256 * i, ad + (uint64_t)(((q >> 2) * kWtPanel + (q & 3) * 32) >> 4),
                                     bd + (uint64_t)(((q >> 2) * 2 * kWtPanel + (q & 3) * 32) >> 4), id, q > 0 ? 1u : 0u);
                    tc::mma_commit(dfull + i);
                    if (i == tiles - 1) tc::mma_commit(qempty + stage(j));
                }
                __syncwarp();
            }
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------- rows' lse
        // (a lane's own copies, kWtRaw steps ahead: loaded step by step they took 550 us of the size below)
        float* raw = reinterpret_cast<float*>(sm + L::kRaw) + lane;
        auto fetch = [&](int j) {
            const int t0 = first + 2 * j * per;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = 32 * e + lane, r = c & 127, t = t0 + (c >> 7) * per + r / R;
                if (j < steps && r < per * R && t < x.n)
                    cp_async4(raw + j % kWtRaw * 256 + 32 * e, a.lse + (size_t)(x.row0 + t) * a.Hq + g * R + r % R);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int j = 0; j < kWtRaw - 1; ++j) fetch(j);
        for (int j = 0; j < steps; ++j) {
            fetch(j + kWtRaw - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kWtRaw - 1) : "memory");
            if (j >= kWtStages && !warp_ok(lempty + stage(j), phase(j - kWtStages))) break;
#pragma unroll
            for (int e = 0; e < 8; ++e) {  // (a row that the tile does not have gets no weight)
                const int c = 32 * e + lane;
                sL[stage(j) * 256 + c] = (c & 127) < per * R ? -raw[j % kWtRaw * 256 + 32 * e] * kLog2e : -INFINITY;
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(lfull + stage(j));
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= 4 && (warp - 4) >> 2 < tiles) {
        // ------------------------------------------ sums, one position a thread
        const int i = (warp - 4) >> 2, p = p0 + tid - 128;
        const uint32_t tD = tm + ((uint32_t)((warp & 3) * 32) << 16) + 256 * i;
        const float sl2 = a.scale * kLog2e;
        const float2 c2 = make_float2(sl2, sl2);
        for (int j = 0; j < steps; ++j) {
            if (!warp_ok(lfull + stage(j), phase(j))) break;
            const float* nl = sL + stage(j) * 256;
            // pairs lo .. hi - 1 of the step's (of a tile, with those of the other behind them) see the position
            const int t = first + 2 * j * per;
            const bool part = __any_sync(0xffffffffu, p - x.before > t) || x.n < t + 2 * per;
            float2 s0 = make_float2(0.f, 0.f), s1 = s0;
            // the step's sum; kPart: some pairs do not see the position (in code of its own: with the
            // question asked for every pair, the others took twice the instructions)
            auto add_step = [&](auto kPart) -> bool {
                float v[2][32];
                float4 l4[2][8];
#pragma unroll
                for (int e = 0; e < 8; ++e) l4[0][e] = reinterpret_cast<const float4*>(nl)[e];
                if (!warp_ok(dfull + i, (uint32_t)j & 1u)) return false;
                tc::tc_fence_after();
                tmem_ld32(tD, v[0]);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int at = q & 1, to = at ^ 1;
                    tc::tmem_wait_ld();
                    if (q < 7) {
                        tmem_ld32(tD + 32 * (q + 1), v[to]);
#pragma unroll
                        for (int e = 0; e < 8; ++e) l4[to][e] = reinterpret_cast<const float4*>(nl + 32 * (q + 1))[e];
                    } else {
                        tc::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(dempty + i), tc::mbar_arrive(lempty + stage(j));
                    }
                    const int tq = t + (q >> 2) * per, lo = (p - x.before - tq) * R - 32 * (q & 3),
                              hi = min(x.n - tq, per) * R - 32 * (q & 3);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 l = l4[at][e];
                        float2 x0 = fma2(make_float2(v[at][4 * e], v[at][4 * e + 1]), c2, make_float2(l.x, l.y));
                        float2 x1 = fma2(make_float2(v[at][4 * e + 2], v[at][4 * e + 3]), c2, make_float2(l.z, l.w));
                        if constexpr (decltype(kPart)::value) {
                            const int c = 4 * e;
                            x0.x = c >= lo && c < hi ? x0.x : -INFINITY, x0.y = c + 1 >= lo && c + 1 < hi ? x0.y : -INFINITY;
                            x1.x = c + 2 >= lo && c + 2 < hi ? x1.x : -INFINITY, x1.y = c + 3 >= lo && c + 3 < hi ? x1.y : -INFINITY;
                        }
                        s0 = add2(s0, make_float2(ex2_approx(x0.x), ex2_approx(x0.y)));
                        s1 = add2(s1, make_float2(ex2_approx(x1.x), ex2_approx(x1.y)));
                    }
                }
                return true;
            };
            if (!(part ? add_step(std::true_type()) : add_step(std::false_type()))) break;
            sum += (s0.x + s0.y) + (s1.x + s1.y);  // (a step's terms first, then the steps: no long chain of roundings)
        }
        if (p < total) w.acc_out[head + p] = (p < x.before ? w.acc[head + p] : 0.f) + sum;
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    if (*flag) {  // (the same in the whole CTA)
        // the copies in flight must land and every product issued must be done
        // before the tensor memory is freed and the CTA exits (all bounded)
        if (warp == 0 && tc::elect_one()) {
            tc::mbar_wait(kbar, 0, 100000000ull);
            for (int i = 0; i < kWtStages; ++i)
                tc::mbar_wait(qfull + i, 0, 100000000ull), tc::mbar_wait(qfull + i, 1, 100000000ull);
        } else if (warp == 1 && tc::elect_one()) {
            tc::mma_commit(endbar);
            tc::mbar_wait(endbar, 0, 100000000ull);
        }
        __syncthreads();
    }
    if (warp == 1) tc::tmem_dealloc(tm, 512);
}

}  // namespace

cudaError_t launch_attn_weights_tiles(const PromptArgs& a, const PromptSums& w, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(attn_weights_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)WtSmem::kBytes);
    if (e != cudaSuccess) return e;
    const int R = a.Hq / a.Hkv, per = 128 / R;
    CUtensorMap tmq, tmk;
    const unsigned long long row = kAttnD * 2;
    // (a call without rows has no queries to copy: any map will do)
    e = make_rows_map(a.q, a.Hq, a.rows > 0 ? a.rows : 1, row, (unsigned long long)a.q_stride * 2, R, per, &tmq);
    if (e == cudaSuccess) e = make_rows_map(a.k_cache, a.Tmax, (unsigned long long)a.S * a.Hkv, row, row * a.Tmax, kWtPos, 1, &tmk);
    if (e != cudaSuccess) return e;
    const long blocks = (long)((a.Tmax + 2 * kWtPos - 1) / (2 * kWtPos)) * a.Hkv * a.S;
    return launch_pdl(attn_weights_tile_kernel, dim3((unsigned)blocks), dim3(kWtThreads), WtSmem::kBytes, st, a, w, tmq, tmk);
}

}  // namespace m2
