// The weights that cached positions receive from a packed prompt, in bf16 on the
// tcgen05 tensor cores (the operator and its formulas are those of
// m2_attn_weights.cu).
//
// One CTA takes 256 positions of one (session, kv head), two tiles of 128, and
// walks the window's rows that see any of them, up to 256 (row, head) pairs at a
// time: two tiles of floor(128 / R) packed rows, each a box of a tensor map. Per
// step, tile of positions and tile of pairs:
//   S^T = [K 1] [Q e]^T    kind::f16, M 128 positions x N 128 pairs, K from tensor
//                   memory, where it stays (from shared memory, read anew with
//                   every product, a product took 1,000 cycles for its 580, and the
//                   whole 361 us of the size below where it then took 331); 16 more of the products'
//                   inner dim bring a pair's e = -lse / scale, as three bf16 terms
//                   (24 bits) times ones, so that
//   sum += 2^(S^T scale log2 e)    needs nothing but S^T: one thread a position, whose
//                   sum over the pairs stays in it, added up step by step in a fixed
//                   order. (With the lse read from shared memory, the same for
//                   all threads, its 512 bytes a warp and read cost as much of
//                   shared memory's time as the products: 314 us where the two together
//                   and what follows take 281.)
// The products' sums are fp32, but cut off, not rounded, as they are added; kCutOff takes
// back what that does on average: the sums of the size below, and of the last 32 rows of six
// sessions of up to 2048, are within 4e-7 and 5e-7 of their 2-norm (1.2e-6 and 1.3e-6 without it; single
// scores of 80 may still be off by 1e-6 of a weight).
// The products go to three buffers of tensor memory in turn; two are added up while
// the third is filled.
//
// Warps: 0 copies queries through a ring, 1 issues the products, 2 and 3 make the
// pairs' e, 4-7 and 8-11 the sums of the tiles of positions, whose keys they bring;
// 12 waits for what the next products need while these are issued (an issue lasts as
// long as the products, and a look at a barrier in shared memory some 200 cycles
// more: 331 us without it, 287 with).
//   Measured: 4 sessions of 4096 rows, 40 query and 8 kv heads, all rows, 344 GFLOP: 262
// us replayed from a graph, 1.31 PFLOP/s (69 % of a bf16 library product's measured rate);
// 287 in a loop of eager calls of half a second, 1.20. A step of 256
// pairs took 2,650 cycles when the whole took 284 us: 2,300 of products (2,050 without e), and the
// exponentials' unit is busy for 2,050 of them; a CTA's start and its first steps,
// which some positions do not see, are another fifth.
#include <math.h>

#include "m2_dense_dev.cuh"
#include "m2_tc.cuh"

namespace m2 {

namespace {

constexpr int kWtThreads = 416;
constexpr int kWtPos = 128;                        // positions a tile
constexpr uint32_t kWtPanel = 128 * 128;           // 128 rows x 64 dims of bf16
constexpr uint32_t kWtStage = 4 * kWtPanel;        // 256 rows of queries
constexpr int kWtStages = 3;
constexpr int kWtBuffers = 3;                      // of 128 columns of tensor memory
constexpr uint32_t kWtColK = 128 * kWtBuffers;     // behind them the keys, 64 columns a tile
constexpr int kWtRaw = 4;                          // steps whose lse is on its way

constexpr uint32_t kWtExtra = 128 * 32;            // 128 rows x 16 of bf16, 8 x 8 blocks: rows by 128 bytes, the second 8 2 KB on
struct WtSmem {
    static constexpr uint32_t kQ = 0;                                 // [stage][panel][256 rows] K-major, 128-byte swizzle
    static constexpr uint32_t kE = kQ + kWtStages * kWtStage;         // [stage][tile of pairs]: e, K-major, no swizzle
    static constexpr uint32_t kOne = kE + kWtStages * 2 * kWtExtra;   // the ones they are multiplied by, likewise
    static constexpr uint32_t kRaw = kOne + kWtExtra;                 // float [kWtRaw][256]: lse on its way
    static constexpr uint32_t kBar = kRaw + kWtRaw * 256 * 4;
    // kload, k, qfull[stages], qempty[stages], efull[stages], d[buffers], dempty[buffers], end
    static constexpr int kBars = 3 * kWtStages + 2 * kWtBuffers + 3;
    static constexpr uint32_t kTmem = kBar + kBars * 8;
    static constexpr uint32_t kFlag = kTmem + 4;
    static constexpr uint32_t kSum = (kFlag + 4 + 15) / 16 * 16;      // float [256]: the CTA's part of the positions' sums
    static constexpr uint32_t kBytes = kSum + 2 * kWtPos * 4 + 1024;  // + slack to align to 1024
    static_assert(kBytes <= 227 * 1024, "one CTA an SM");
};

// The warp that issues the products and the one that waits for their operands, once
// a product.
__device__ __forceinline__ void products_meet() { asm volatile("barrier.sync 1, 64;" ::: "memory"); }

// grid: n x Hkv x S x W, a CTA for every n-th tile of 256 positions; the first tiles, which most rows see, first.
// W > 1: a cluster takes a tile, a CTA a run of its steps.
__global__ void __launch_bounds__(kWtThreads, 1)
    attn_weights_tile_kernel(PromptArgs a, PromptSums w, const __grid_constant__ CUtensorMap tmq,
                             const __grid_constant__ CUtensorMap tmk, int W) {
    using L = WtSmem;
    extern __shared__ uint8_t wt_raw[];
    uint8_t* sm = wt_raw + ((1024u - (tc::smem_u32(wt_raw) & 1023u)) & 1023u);
    uint64_t* kload = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint64_t *kbar = kload + 1, *qfull = kbar + 1, *qempty = qfull + kWtStages, *efull = qempty + kWtStages,
             *dfull = efull + kWtStages, *dempty = dfull + kWtBuffers, *endbar = dempty + kWtBuffers;
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + L::kTmem);
    volatile uint32_t* flag = reinterpret_cast<uint32_t*>(sm + L::kFlag);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int R = a.Hq / a.Hkv, per = 128 / R;  // packed rows a tile of pairs
    const int heads = a.Hkv * a.S, stride = gridDim.x / W / heads;  // tiles of 256 positions: this CTA's first, and from one to the next
    const int wk = blockIdx.x % W, block = blockIdx.x / W, tile0 = block / heads;
    const int g = block % heads % a.Hkv, s = block % heads / a.Hkv;

    if (tid == 0) prefetch_map(&tmq), prefetch_map(&tmk);
    pdl_wait();
    const int ahead = load_ahead(a, s);
    Session x;
    const bool within = session_of(a, s, &x), rows_ok = block_begins_behind(a, s, ahead) && within;
    if (!rows_ok || !x.ok) {
        if (tid == 0 && tile0 == 0) record_error(a.err, rows_ok ? ERR_ATTN_LENGTH : ERR_ROW_START);
        return;
    }
    const int total = x.before + x.n;
    if (tile0 * 2 * kWtPos >= total) return;
    const size_t head = ((size_t)s * a.Hkv + g) * a.Tmax;

    if (tid == 0) {
        tc::mbar_init(kload, 1), tc::mbar_init(kbar, 8);
        for (int i = 0; i < kWtStages; ++i) {
            tc::mbar_init(qfull + i, 1), tc::mbar_init(qempty + i, 1), tc::mbar_init(efull + i, 2);
        }
        for (int i = 0; i < kWtBuffers; ++i) tc::mbar_init(dfull + i, 1), tc::mbar_init(dempty + i, 4);
        tc::mbar_init(endbar, 1);
        tc::fence_mbar_init();
        *flag = 0;
    }
    if (warp == 1) {
        tc::tmem_alloc(sTmem, 512);
        tc::tmem_relinquish();
    }
    // The ones: three of 16; what e's last 13 are is zeros. (Rows of a tile of pairs that no packed row
    // fills hold anything: their columns of the products are not added up.)
    if (warp >= 4) {
        for (int i = tid - 128; i < (int)((2 * kWtStages + 1) * kWtExtra / 16); i += kWtThreads - 128) {
            const bool ones = i >= (int)(2 * kWtStages * kWtExtra / 16) && i % (int)(kWtExtra / 16) < 128;
            *reinterpret_cast<uint4*>(sm + L::kE + i * 16) = ones ? make_uint4(0x3F803F80u, 0x3F80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
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
    // A tile of 256 positions: the window's rows that see any of them, first .. n - 1, in steps of 2 per.
    struct Item {
        int p0, first, steps, tiles;  // tiles: of 128 positions
    };
    auto item = [&](int tile) {
        Item it;
        it.p0 = tile * 2 * kWtPos;
        it.first = max(max(0, x.n - w.window), it.p0 - x.before);
        const int steps = it.first < x.n ? (x.n - it.first + 2 * per - 1) / (2 * per) : 0, run = (steps + W - 1) / W;
        it.first += wk * run * 2 * per;  // this CTA's run of them
        it.steps = min(max(steps - wk * run, 0), run);
        it.tiles = it.p0 + kWtPos < total ? 2 : 1;
        return it;
    };
    // tiles of pairs of step j that have rows
    auto filled = [&](const Item& it, int j) { return it.first + (2 * j + 1) * per < x.n ? 2 : 1; };
    // Each warp's loop over the CTA's tiles of positions that have steps: role(it, k of them and J steps before)
    auto every_item = [&](auto role) {
        for (int tile = tile0, k = 0, J = 0; tile * 2 * kWtPos < total; tile += stride) {
            const Item it = item(tile);
            role(it, k, J);
            k += it.steps > 0;
            J += it.steps;
        }
    };

    if (warp == 0) {
        // ---------------------------------------------------------------- copies
        bool good = true;
        every_item([&](const Item& it, int k, int J) {
            if (it.steps == 0 || !good) return;
            // the keys go by way of the stage of the third step
            const int ks = stage(J + kWtStages - 1);
            if (J > 0) good = warp_ok(qempty + stage(J - 1), phase(J - 1));
            if (good && tc::elect_one()) {
                tc::mbar_arrive_expect_tx(kload, (uint32_t)it.tiles * 2 * kWtPanel);
                for (int i = 0; i < it.tiles; ++i)
                    for (int h = 0; h < 2; ++h)
                        tc::tma_load_3d(sm + L::kQ + ks * kWtStage + (2 * i + h) * kWtPanel, &tmk, 64 * h, it.p0 + i * kWtPos,
                                        s * a.Hkv + g, kload);
            }
            __syncwarp();
            for (int j = 0; j < it.steps || j < kWtStages; ++j) {
                if (j == kWtStages - 1) good = good && warp_ok(kbar, (uint32_t)k & 1u);  // the keys are read
                if (j >= it.steps) continue;
                const int at = stage(J + j);
                if (J + j >= kWtStages) good = good && warp_ok(qempty + at, phase(J + j - kWtStages));
                if (good && tc::elect_one()) {
                    const int n = filled(it, j);
                    tc::mbar_arrive_expect_tx(qfull + at, (uint32_t)(n * 2 * per * R * 128));
                    for (int i = 0; i < n; ++i)
                        for (int h = 0; h < 2; ++h)
                            tc::tma_load_3d(sm + L::kQ + at * kWtStage + (2 * h + i) * kWtPanel, &tmq, 64 * h, g * R,
                                            x.row0 + it.first + (2 * j + i) * per, qfull + at);
                }
                __syncwarp();
            }
        });
    } else if (warp == 1) {
        // -------------------------------------------------------------- products
        const bool leader = tc::elect_one();
        const uint32_t sbase = tc::smem_u32(sm);
        int m = 0;  // products so far
        every_item([&](const Item& it, int, int J) {
            for (int j = 0; j < it.steps; ++j) {
                const int n = filled(it, j), at = stage(J + j);
                for (int d = 0; d < n * it.tiles; ++d, ++m) {
                    const int i = it.tiles == 2 ? d & 1 : 0, h = it.tiles == 2 ? d >> 1 : d, b = m % kWtBuffers;
                    products_meet();
                    tc::tc_fence_after();
                    if (leader) {
                        const uint64_t bd = tc::sdesc(sbase + L::kQ + at * kWtStage + h * kWtPanel, 0, 1024, 2);
                        const uint32_t to = tm + 128 * b, id = tc::idesc_bf16(128, 128, 0, 0);
    #pragma unroll
                        for (int q = 0; q < 8; ++q)
                            tc::mma_bf16_tmem_a(to, tm + kWtColK + 64 * i + 8 * q,
                                                bd + (uint64_t)(((q >> 2) * 2 * kWtPanel + (q & 3) * 32) >> 4), id, q > 0 ? 1u : 0u);
                        // (e last: the sums are cut off at the size of what they have reached)
                        tc::mma_bf16(to, tc::sdesc(sbase + L::kOne, kWtExtra / 2, 128, 0),
                                     tc::sdesc(sbase + L::kE + (2 * at + h) * kWtExtra, kWtExtra / 2, 128, 0), id, 1u);
                        tc::mma_commit(dfull + b);
                        if (d == n * it.tiles - 1) tc::mma_commit(qempty + at);
                    }
                    __syncwarp();
                }
            }
        });
    } else if (warp == 12) {
        // -------------------------------------- waits on behalf of the products
        // (after one that gave up, what the products read is there, if not what it should be, and the
        // error is recorded; every meeting takes place)
        bool good = true;
        int m = 0;
        every_item([&](const Item& it, int k, int J) {
            if (it.steps > 0) good = good && warp_ok(kbar, (uint32_t)k & 1u);
            for (int j = 0; j < it.steps; ++j) {
                const int at = stage(J + j);
                good = good && warp_ok(qfull + at, phase(J + j)) && warp_ok(efull + at, phase(J + j));
                const int products = filled(it, j) * it.tiles;
                for (int d = 0; d < products; ++d, ++m) {
                    if (m >= kWtBuffers) good = good && warp_ok(dempty + m % kWtBuffers, (uint32_t)(m / kWtBuffers - 1) & 1u);
                    tc::tc_fence_before();
                    products_meet();
                }
            }
        });
    } else if (warp < 4) {
        // ------------------------------------- the pairs' e, a tile of pairs a warp
        // (a lane's own copies of lse, kWtRaw steps ahead: loaded step by step they took 550 us of the
        // size below, and with one warp, which has a step's time for 256 of them, 357)
        const int h = warp - 2;
        float* raw = reinterpret_cast<float*>(sm + L::kRaw) + 128 * h + lane;
        const float by = -1.f / (a.scale * kCutOff), none = a.scale > 0.f ? -INFINITY : INFINITY;
        bool good = true;
        every_item([&](const Item& it, int, int J) {
            const float* from[4];  // a lane's pairs 32 e + lane, step by step
            int t[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 32 * e + lane;
                t[e] = r < per * R ? it.first + h * per + r / R : x.n;  // (a row that the tile does not have: never)
                from[e] = a.lse + (size_t)(x.row0 + it.first + h * per + r / R) * a.Hq + g * R + r % R;
            }
            auto fetch = [&](int j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (t[e] < x.n) cp_async4(raw + (J + j) % kWtRaw * 256 + 32 * e, from[e]);
                    t[e] += 2 * per, from[e] += (size_t)2 * per * a.Hq;
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            if (it.steps == 0) return;
            for (int j = 0; j < kWtRaw - 1; ++j) fetch(j);
            for (int j = 0; j < it.steps; ++j) {
                const int at = stage(J + j);
                fetch(j + kWtRaw - 1);
                asm volatile("cp.async.wait_group %0;" ::"n"(kWtRaw - 1) : "memory");
                if (J + j >= kWtStages) good = good && warp_ok(qempty + at, phase(J + j - kWtStages));
                if (!good) break;
#pragma unroll 1
                for (int e = 0; e < 4; ++e) {
                    const int r = 32 * e + lane;
                    const float z = r < per * R ? raw[(J + j) % kWtRaw * 256 + 32 * e] * by : none;  // (no weight)
                    // hi + mid + lo, each what the ones before it leave, rounded; of an infinity hi alone
                    const uint32_t hi = float_to_bf16_bits(z);
                    const float top = bf16_bits_to_float(hi), rest = fabsf(top) < INFINITY ? z - top : 0.f;
                    const uint32_t mid = float_to_bf16_bits(rest), lo = float_to_bf16_bits(rest - bf16_bits_to_float(mid));
                    *reinterpret_cast<uint2*>(sm + L::kE + (2 * at + h) * kWtExtra + (r >> 3) * 128 + (r & 7) * 16) =
                        make_uint2(hi | mid << 16, lo);
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(efull + at);
            }
        });
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // ------------------------------------------ sums, one position a thread
        const int i = (warp - 4) >> 2;
        const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
        const float sl2 = a.scale * kLog2e * kCutOff;
        const float2 c2 = make_float2(sl2, sl2);
        int done = 0;  // products before the step's
        every_item([&](const Item& it, int k, int J) {
            const int p = it.p0 + tid - 128, tiles = it.tiles;
            if (it.steps > 0) {
                // its key, two dims a column (read from the cache, a row a thread, it took 2 us more); the
                // products with the one before are done
                warp_ok(kload, (uint32_t)k & 1u);
                if (i < tiles) {
                    const uint8_t* key = sm + L::kQ + stage(J + kWtStages - 1) * kWtStage + 2 * i * kWtPanel + (tid & 127) * 128;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t v[16];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint4 u = *reinterpret_cast<const uint4*>(key + (q >> 1) * kWtPanel +
                                                                            (((4 * (q & 1) + e) ^ (tid & 7)) << 4));
                            v[4 * e] = u.x, v[4 * e + 1] = u.y, v[4 * e + 2] = u.z, v[4 * e + 3] = u.w;
                        }
                        tmem_st16(lanes + kWtColK + 64 * i + 16 * q, v);
                    }
                    tc::fence_proxy_async_smem();  // (read before the stage's queries come)
                    tc::tmem_wait_st();
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(kbar);
            }
            float sum = 0.f;
            for (int j = 0; j < (i < tiles ? it.steps : 0); ++j) {
                const int t0 = it.first + 2 * j * per, p_last = p - lane + 31;
                float2 s0 = make_float2(0.f, 0.f), s1 = s0;
                // The step's sum; kPart: some of its pairs do not see some of the warp's positions. (Code of its
                // own: asked for every pair, or between the 32s, of every step, that cost them all a quarter.)
                auto add_step = [&](auto kPart) -> bool {
                    constexpr bool kAsk = decltype(kPart)::value;
                    const int n = kAsk ? filled(it, j) : 2;
#pragma unroll 1  // (twice the code: 284 us of the size above)
                    for (int h = 0; h < 2; ++h) {
                        if (kAsk && h == n) break;
                        const int m = done + h * tiles + i, b = m % kWtBuffers;  // the product
                        const uint32_t tD = lanes + 128 * b;
                        if (!warp_ok(dfull + b, (uint32_t)(m / kWtBuffers) & 1u)) return false;
                        tc::tc_fence_after();
                        float v[2][32];
                        tmem_ld32(tD, v[0]);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int at = q & 1;
                            tc::tmem_wait_ld();
                            if (q < 3) {
                                tmem_ld32(tD + 32 * (q + 1), v[at ^ 1]);
                            } else {  // the buffer is read
                                tc::tc_fence_before();
                                __syncwarp();
                                if (lane == 0) tc::mbar_arrive(dempty + b);
                            }
                            // pairs lo .. hi - 1 of these 32 see the position
                            const int t = t0 + h * per, hi = min(x.n - t, per) * R - 32 * q;
                            const int lo = (p - x.before - t) * R - 32 * q, lo0 = lo - lane * R;
                            if (kAsk && (hi <= 0 || lo0 >= 32)) continue;  // none of the warp's
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float2 x0 = mul2(make_float2(v[at][4 * e], v[at][4 * e + 1]), c2);
                                float2 x1 = mul2(make_float2(v[at][4 * e + 2], v[at][4 * e + 3]), c2);
                                // the columns that no packed row fills, three at most
                                if (!kAsk && q == 3 && e == 7) {
                                    x0.y = per * R > 125 ? x0.y : -INFINITY;
                                    x1.x = per * R > 126 ? x1.x : -INFINITY, x1.y = per * R > 127 ? x1.y : -INFINITY;
                                }
                                if (kAsk) {
                                    const int c = 4 * e;
                                    x0.x = c >= lo && c < hi ? x0.x : -INFINITY, x0.y = c + 1 >= lo && c + 1 < hi ? x0.y : -INFINITY;
                                    x1.x = c + 2 >= lo && c + 2 < hi ? x1.x : -INFINITY, x1.y = c + 3 >= lo && c + 3 < hi ? x1.y : -INFINITY;
                                }
                                s0 = add2(s0, make_float2(ex2_approx(x0.x), ex2_approx(x0.y)));
                                s1 = add2(s1, make_float2(ex2_approx(x1.x), ex2_approx(x1.y)));
                            }
                        }
                    }
                    done += n * tiles;
                    return true;
                };
                const bool part = p_last - x.before > t0 || x.n < t0 + 2 * per;  // (the same in the whole warp)
                if (!(part ? add_step(std::true_type()) : add_step(std::false_type()))) break;
                sum += (s0.x + s0.y) + (s1.x + s1.y);  // (a step's terms first, then the steps: no long chain of roundings)
            }
            if (W > 1)
                reinterpret_cast<float*>(sm + L::kSum)[tid - 128] = sum;
            else if (p < total)
                w.acc_out[head + p] = (p < x.before ? w.acc[head + p] : 0.f) + sum;
        });
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    if (*flag) {  // (the same in the whole CTA)
        // the copies in flight must land and every product issued must be done
        // before the tensor memory is freed and the CTA exits (all bounded)
        if (warp == 0 && tc::elect_one()) {
            tc::mbar_wait(kload, 0, 100000000ull), tc::mbar_wait(kload, 1, 100000000ull);
            for (int i = 0; i < kWtStages; ++i)
                tc::mbar_wait(qfull + i, 0, 100000000ull), tc::mbar_wait(qfull + i, 1, 100000000ull);
        } else if (warp == 1 && tc::elect_one()) {
            tc::mma_commit(endbar);
            tc::mbar_wait(endbar, 0, 100000000ull);
        }
        __syncthreads();
    }
    if (warp == 1) tc::tmem_dealloc(tm, 512);
    if (W == 1) return;
    tc::cluster_arrive();  // every CTA's sums are in its shared memory ...
    tc::cluster_wait();
    // ... and each adds up its share of the positions', in order
    const int share = 2 * kWtPos / W, p = tile0 * 2 * kWtPos + wk * share + tid;
    if (tid < share && p < total) {
        float sum = 0.f;
        for (int c = 0; c < W; ++c) sum += ld_cluster_f32(tc::cluster_map(tc::smem_u32(sm) + L::kSum + (wk * share + tid) * 4, c));
        w.acc_out[head + p] = (p < x.before ? w.acc[head + p] : 0.f) + sum;
    }
    tc::cluster_arrive();  // nobody leaves while its memory is read
    tc::cluster_wait();
}

}  // namespace

cudaError_t launch_attn_weights_tiles(const PromptArgs& a, const PromptSums& w, cudaStream_t st) {
    cudaError_t e = allow_shared<1>((const void*)attn_weights_tile_kernel, (int)WtSmem::kBytes);
    if (e != cudaSuccess) return e;
    const int R = a.Hq / a.Hkv, per = 128 / R;
    CUtensorMap tmq, tmk;
    const unsigned long long row = kAttnD * 2;
    // (a call without rows has no queries to copy: any map will do)
    e = make_rows_map(a.q, a.Hq, a.rows > 0 ? a.rows : 1, row, (unsigned long long)a.q_stride * 2, R, per, &tmq);
    if (e == cudaSuccess) e = make_rows_map(a.k_cache, a.Tmax, (unsigned long long)a.S * a.Hkv, row, row * a.Tmax, kWtPos, 1, &tmk);
    if (e != cudaSuccess) return e;
    // A CTA a tile of positions while that is some four an SM, or two where a tile has a step or two (six sessions
    // of 75 rows behind up to 3,001, the last 32: 14.7 us, 17.0 with four; four sessions of 4096, all rows: 262
    // with four, 289 with two); past that, where many tiles of many sessions may lie behind their last positions, a
    // CTA takes every n-th of a (session, kv head).
    const long window = w.window < a.rows ? w.window : a.rows, steps = (window + 2 * per - 1) / (2 * per);
    const long heads = (long)a.Hkv * a.S, reach = a.lens ? a.Tmax : a.rows < a.Tmax ? a.rows : a.Tmax;
    const long tiles = (reach + 2 * kWtPos - 1) / (2 * kWtPos), most = ((steps > 2 ? 4 : 2) * 152 + heads - 1) / heads;
    // While the tiles leave most SMs idle, up to four CTAs share a tile's steps (one session of 300, all rows: 10.2
    // us, 11.8 with two, 16.3 with one; of 600 12.4, 17.8, 25.3; eight were no faster).
    int W = 1;
    while (W < 4 && 2 * W <= steps && heads * tiles * 2 * W <= 152) W *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(W * heads * (tiles < 1 ? 1 : tiles < most ? tiles : most)));
    cfg.blockDim = dim3(kWtThreads);
    cfg.dynamicSmemBytes = WtSmem::kBytes;
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
    return cudaLaunchKernelEx(&cfg, attn_weights_tile_kernel, a, w, tmq, tmk, W);
}

}  // namespace m2
