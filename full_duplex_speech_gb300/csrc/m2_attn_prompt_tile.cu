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
// Warps: 0 copies (a ring of K and V by TMA), 1 issues the products, 2 waits for
// their operands, 3 looks them over as they land and mends the values of chunks
// that some rows see only partly: positions behind the last count as zeros, and
// so do values that are not finite, which must not reach the rows that do not see
// them (the others read NaN); 4-7 and 8-11 the softmax of the tiles. The products
// of one tile run under the other's softmax.
//
// A CTA that is done takes the place of one that has not started yet
// (clusterlaunchcontrol: in the order of blockIdx, whichever CTA is free first), and
// its copies run ahead: the next rows' queries, keys and values are under way
// while the softmax and the output of the last chunk still run. Outputs leave by way
// of a piece of the ring a tile. A tile's softmax goes on to the next rows by itself.
// (With a CTA started for each pair of tiles, 535 us of the size below where it then took 490.)
//
// Where few pairs would leave SMs idle, W CTAs of a cluster share the positions
// of one pair of tiles and merge through distributed shared memory; they take one
// pair each.
// Code length alone costs time here, as where instructions do not stay in the nearest
// caches: what runs every chunk is kept short, and the softmax comes first (with the
// others first, the mending unrolled by eight and no way past it for most pieces 490 us of
// the size below and 74 of nine prompts of up to 750, which now take 70.5).
//   Measured: 4 sessions of 4096 rows, 40 query and 8 kv heads, causal, 687 GFLOP: 464
// us with the append (24 alone) replayed from a graph, 1.48 PFLOP/s, 78 % of a bf16 library
// product's measured rate; 505 in a loop of eager calls of half a second, 1.36. A chunk of a pair took 2,600
// cycles when the whole took 490 us: 2 x 1,150 of products (2,050 at their rate; what is
// left waits for shared memory, which they and the copies read and write for 2,000
// cycles), each tile's softmax 1,000 and its hand-overs some 450.
#include <limits.h>
#include <math.h>

#include <mutex>

#include "m2_dense_dev.cuh"
#include "m2_prompt_ring.h"
#include "m2_tc.cuh"
#include "m2_tile_meet.h"

namespace m2 {

namespace {

constexpr int kPtThreads = 384;
constexpr int kPtRows = 128;                       // rows of a tile
constexpr int kPtPos = 128;                        // positions a chunk
constexpr uint32_t kPtPanel = 128 * 128;           // 128 rows x 64 dims of bf16
constexpr uint32_t kPtTile = 2 * kPtPanel;
constexpr int kPtStages = kRingStages;             // of a chunk's K or V, in turn
constexpr float kPtSlack = 8.f;                    // log2 by which a chunk may exceed m
constexpr int kPtCut = 3;                          // chunks that the tiles' at most 256 packed rows see partly, at most
constexpr int kPtBad = 4 * kPtCut + 1;
constexpr uint32_t kColO = 0, kColS = 256;         // tensor memory: O of the two tiles, then S (and p over it)

struct PtSmem {
    static constexpr uint32_t kQ = 0;                                // [tile][panel] K-major
    static constexpr uint32_t kRing = kQ + 2 * kPtTile;              // K: K-major, V: MN-major; two panels each
    static constexpr uint32_t kBar = kRing + kPtStages * kPtTile;
    // full[stages], empty[stages], ready[stages], qfull, qempty, s[2], o[2], next, passed, end
    static constexpr int kBars = 3 * kPtStages + 9;
    static constexpr uint32_t kBad = kBar + kBars * 8;               // values that are not finite: a bit a position, and
                                                                     // whether any; for the pairs in turn
    static constexpr uint32_t kNext = (kBad + 2 * kPtBad * 4 + 15) / 16 * 16;  // the answer of clusterlaunchcontrol
    static constexpr uint32_t kWork = kNext + 16;                    // PtWork, in turn
    static constexpr uint32_t kTmem = kWork + 2 * 32;
    static constexpr uint32_t kFlag = kTmem + 4;
    static constexpr uint32_t kBytes = kFlag + 4 + 1024;             // + slack to align to 1024
    // after the walk, over the ring: 256 rows x 128 floats, then their (m, l)
    static constexpr uint32_t kMl = kRing + 2 * kPtRows * kAttnD * 4;
    static_assert(kMl + 2 * kPtRows * 8 <= kBar, "the merge fits in the ring");
    static_assert(kBytes <= 227 * 1024, "one CTA an SM");
};

// A pair of tiles (or one tile, where there are few): a session (-1: none is left) and its rows,
// the pair of it, the kv head.
struct PtWork {
    int s, row0, n, before, pair, g;
};
static_assert(sizeof(PtWork) <= 32, "a slot of kWork");

constexpr int kRegsLaunch = 168, kRegsFew = 88, kRegsMany = 208;
static_assert(128 * kRegsFew + 256 * kRegsMany <= kPtThreads * kRegsLaunch, "the split is covered by the launch's registers");
// the threads of a tile's softmax; of both tiles'
__device__ __forceinline__ void tile_sync(int i) { asm volatile("barrier.sync %0, 128;" ::"r"(4 + i) : "memory"); }
__device__ __forceinline__ void tiles_sync() { asm volatile("barrier.sync 6, 256;" ::: "memory"); }

// The next pair of tiles is known: warp 0 says so without waiting, and the softmax
// of tile 0, that of tile 1 and the warps 1 to 3 wait for it, each for themselves.
__device__ __forceinline__ void pair_known() {
    asm volatile("barrier.arrive 7, 160;\n\tbarrier.arrive 8, 160;\n\tbarrier.arrive 9, 128;" ::: "memory");
}
__device__ __forceinline__ void pair_wait(int warp) {
    asm volatile("barrier.sync %0, %1;" ::"r"(warp < 4 ? 9 : warp < 8 ? 7 : 8), "r"(warp < 4 ? 128 : 160) : "memory");
}

// Asks for the block index of a CTA that has not started, to run in its place;
// the answer comes to `to`, counted on `bar`. Not to be asked again after a refusal.
__device__ __forceinline__ void ask_next(void* to, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     tc::smem_u32(to)),
                 "r"(tc::smem_u32(bar))
                 : "memory");
}
// The answer: its blockIdx.x, or -1.
__device__ __forceinline__ int answer_next(const void* from) {
    uint32_t ok, x;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
        : "=r"(ok), "=r"(x)
        : "r"(tc::smem_u32(from))
        : "memory");
    return ok ? (int)x : -1;
}

// A box of shared memory out to a tensor map's coordinates.
__device__ __forceinline__ void tma_store_3d(const void* tmap, int x, int y, int z, const void* src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(tmap), "r"(x),
                 "r"(y), "r"(z), "r"(tc::smem_u32(src))
                 : "memory");
}

// The pair of tiles `at` of all the sessions' pairs of `per` packed rows each,
// found by a warp, four sessions a lane at a time (a session's last pair first:
// it sees the most positions). A session whose rows do not lie within the call's, or
// begin before an entry ahead of them, has none (the append records it). `from`: the sessions
// and pairs that lie before, and, once an entry is below the one ahead of it, the
// largest of theirs, for the next time.
struct PtFound {
    int s0, base;
    bool fell;
    int top;
};
__device__ __forceinline__ PtWork find_pair(const PromptArgs& a, int per, int at, PtFound* from) {
    constexpr int kEach = 4;
    const int lane = threadIdx.x & 31;
    PtWork y = {-1, 0, 0, 0, 0, at % a.Hkv};
    at /= a.Hkv;
    if (at < from->base) *from = {0, 0, false, 0};
    int base = from->base, top = from->top;
    bool fell = from->fell;
    for (int s0 = from->s0; s0 < a.S; s0 += 32 * kEach) {
        *from = {s0, base, fell, top};
        int b[kEach + 1], before[kEach], n[kEach], mine = 0;
        const int first = s0 + lane * kEach;
#pragma unroll
        for (int i = 0; i <= kEach; ++i) b[i] = first + i <= a.S ? a.start[first + i] : 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) before[i] = a.lens && first + i < a.S ? a.lens[first + i] : 0;
        bool falls = false;
#pragma unroll
        for (int i = 0; i < kEach; ++i) falls = falls || (first + i < a.S && b[i + 1] < b[i]);
        unsigned before_them = 0;  // a bit a session that begins before an entry ahead of its first
        if (__builtin_expect(fell || __any_sync(0xffffffffu, falls), 0)) {
            if (!fell) top = __shfl_sync(0xffffffffu, b[0], 0);
            fell = true;
            int largest = INT_MIN;
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (first + i < a.S) largest = max(largest, b[i]);
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int below = __shfl_up_sync(0xffffffffu, largest, off);
                if (lane >= off) largest = max(largest, below);
            }
            const int below = __shfl_up_sync(0xffffffffu, largest, 1);
            int ahead = lane > 0 ? max(top, below) : top;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                if (b[i] < ahead) before_them |= 1u << i;
                ahead = max(ahead, b[i]);
            }
            top = max(top, __shfl_sync(0xffffffffu, largest, 31));
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            n[i] = 0;
            if (first + i < a.S && b[i] >= 0 && b[i + 1] >= b[i] && b[i + 1] <= a.rows && !(before_them >> i & 1u))
                n[i] = (b[i + 1] - b[i] + per - 1) / per;
            mine += n[i];
        }
        int upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int below = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += below;
        }
        int ahead = base + upto - mine;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (at >= ahead && at < ahead + n[i])
                y.s = first + i, y.row0 = b[i], y.n = b[i + 1] - b[i], y.before = before[i], y.pair = n[i] - 1 - (at - ahead);
            ahead += n[i];
        }
        const unsigned who = __ballot_sync(0xffffffffu, y.s >= 0);
        if (who) {
            const int src = __ffs(who) - 1;
            y.s = __shfl_sync(0xffffffffu, y.s, src);
            y.row0 = __shfl_sync(0xffffffffu, y.row0, src);
            y.n = __shfl_sync(0xffffffffu, y.n, src);
            y.before = __shfl_sync(0xffffffffu, y.before, src);
            y.pair = __shfl_sync(0xffffffffu, y.pair, src);
            return y;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
    return y;
}

// A pair's rows and the run of chunks that CTA wk of W takes.
struct PtRun {
    int t0, row_end;     // packed rows t0 .. row_end - 1 of the session
    int all, total;      // positions that every row sees, and that the last one does
    int cb, nc;          // this CTA's run of chunks, cb .. cb + nc - 1
    int nc0, nc1;        // ... of which tile 0 and tile 1 take so many
    int pieces;          // of the ring: K and V of each chunk in turn, and (W == 1) room for each tile's output
    int cut;             // the first of them that is not whole for every row
    bool ok;             // the session's positions fit the cache (otherwise no chunks)
    __device__ __forceinline__ PtRun(const PromptArgs& a, const PtWork& y, int per, int span, int W, int wk) {
        ok = y.before >= 0 && (long)y.before + y.n <= a.Tmax;
        t0 = y.pair * span;
        row_end = min(t0 + span, y.n);
        all = y.before + t0 + 1;
        total = y.before + row_end;
        const int total0 = y.before + min(t0 + per, row_end);
        const int nch = ok ? (total + kPtPos - 1) / kPtPos : 0, cpw = W == 1 ? nch : (nch + W - 1) / W;
        cb = min(wk * cpw, nch);
        nc = min(cpw, nch - cb);
        nc0 = ok ? min(max((total0 + kPtPos - 1) / kPtPos - cb, 0), nc) : 0;
        nc1 = row_end > t0 + per ? nc : 0;
        cut = max(all / kPtPos, cb);
        pieces = ring_pieces(nc, W > 1 ? 0 : row_end > t0 + per ? 2 : 1);
    }
};

// The CTA's ring as m2_prompt_ring.h sees it; the calling warp is converged.
template <typename WarpOk> struct PtRing {
    uint64_t *full, *empty, *ready;
    WarpOk ok;
    static __device__ __forceinline__ int at(int piece) { return piece % kPtStages; }
    static __device__ __forceinline__ uint32_t turn(int piece) { return (uint32_t)(piece / kPtStages) & 1u; }
    __device__ __forceinline__ bool wait_full(int piece) { return ok(full + at(piece), turn(piece)); }
    __device__ __forceinline__ bool wait_empty(int piece) { return ok(empty + at(piece), turn(piece)); }
    __device__ __forceinline__ bool wait_ready(int piece) { return ok(ready + at(piece), turn(piece)); }
    __device__ __forceinline__ void arrive_ready(int piece) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) tc::mbar_arrive(ready + at(piece));
    }
};

// The merge of a cluster's W parts of the rows that CTA wk owns, a warp a row,
// four dims a lane:
//     out = sum_w 2^(m_w - M) O_w / sum_w 2^(m_w - M) l_w
// Lane i holds the (m, l) of part i % W of the warp's row i / W; eight pieces of
// a row's parts are on their way together (a row after the other, a part after the
// other, took 8 us more of 35 with W = 2).
template <int W>
__device__ __forceinline__ void merge_rows(const PromptArgs& a, uint8_t* sm, int wk, const PtWork& y, const PtRun& run, int per) {
    constexpr int kWarps = kPtThreads / 32, kShare = 2 * kPtRows / W, kRows = (kShare + kWarps - 1) / kWarps, kBatch = 8 / W;
    static_assert(kRows * W <= 32, "a warp's parts, a lane each");
    const int lane = threadIdx.x & 31, R = a.Hq / a.Hkv, first = wk * kShare + (int)(threadIdx.x >> 5);
    const uint32_t here = tc::smem_u32(sm);
    auto row_of = [&](int n) { return min(first + kWarps * n, 2 * kPtRows - 1); };  // the warp's n-th row
    const float2 ml = ld_cluster_f32x2(tc::cluster_map(here, (uint32_t)(lane % W)) + PtSmem::kMl + row_of(lane / W) * 8);
    float M = ml.x;
#pragma unroll
    for (int off = 1; off < W; off <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    const float f = ex2_approx(ml.x - M);
    float L = f * ml.y;
#pragma unroll
    for (int off = 1; off < W; off <<= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
#pragma unroll 1
    for (int n0 = 0; n0 < kRows; n0 += kBatch) {
        float4 v[kBatch][W];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const int row = row_of(n0 + b);
                v[b][w] = ld_cluster_f32x4(tc::cluster_map(here, (uint32_t)w) + PtSmem::kRing + row * kAttnD * 4 +
                                           (((lane + row) & 31) << 4));
            }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int n = n0 + b, row = row_of(n), from = min(n * W, 31);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float fw = __shfl_sync(0xffffffffu, f, min(from + w, 31));
                const float4 x = v[b][w];
                o.x = fmaf(fw, x.x, o.x), o.y = fmaf(fw, x.y, o.y), o.z = fmaf(fw, x.z, o.z), o.w = fmaf(fw, x.w, o.w);
            }
            const float Lr = __shfl_sync(0xffffffffu, L, from), Mr = __shfl_sync(0xffffffffu, M, from);
            const int r = row & 127, t = run.t0 + (row >> 7) * per + r / R;
            if (n >= kRows || first + kWarps * n >= (wk + 1) * kShare || r >= per * R || t >= run.row_end)
                continue;  // (the same in the whole warp)
            const float inv = run.ok ? 1.f / Lr : 0.f;  // (a refused session: zeros)
            const size_t packed = (size_t)y.row0 + t;
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + packed * a.out_stride + (size_t)(y.g * R + r % R) * kAttnD +
                                      4 * lane) =
                run.ok ? make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv)) : make_uint2(0u, 0u);
            if (a.lse && lane == 0) a.lse[packed * a.Hq + y.g * R + r % R] = fmaf(Mr, kLn2, logf(Lr));
        }
    }
}

// grid (W x Hkv x pairs of tiles), a cluster of W CTAs when W > 1
__global__ void __launch_bounds__(kPtThreads, 1)
    attn_prompt_tile_kernel(PromptArgs a, const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmo,
                            const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                            const __grid_constant__ CUtensorMap tmkn, const __grid_constant__ CUtensorMap tmvn, int W, int tiles) {
    using L = PtSmem;
    extern __shared__ uint8_t pt_raw[];
    uint8_t* sm = pt_raw + ((1024u - (tc::smem_u32(pt_raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint64_t *empty = full + kPtStages, *ready = empty + kPtStages, *qfull = ready + kPtStages, *qempty = qfull + 1,
             *sfull = qempty + 1, *ofull = sfull + 2, *next = ofull + 2, *passed = next + 1, *endbar = passed + 1;
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + L::kTmem);
    volatile uint32_t* flag = reinterpret_cast<uint32_t*>(sm + L::kFlag);
    auto bad_of = [&](int k) { return reinterpret_cast<uint32_t*>(sm + L::kBad) + (k & 1) * kPtBad; };
    auto work = [&](int k) { return reinterpret_cast<PtWork*>(sm + L::kWork + (k & 1) * 32); };  // of the CTA's k-th pair
    const int wk = (int)blockIdx.x % W;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int R = a.Hq / a.Hkv, per = kPtRows / R, span = tiles * per;  // packed rows a tile, a pair of tiles

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
    // The ring's pieces, counted over all of the CTA's pairs.
    PtRing<decltype(warp_ok)> ring{full, empty, ready, warp_ok};
    auto stage = [](int piece) { return piece % kPtStages; };

    if (W > 1) tc::cluster_arrive_relaxed();  // waited on before the first remote access: every CTA has started
    bool good = true;                         // warp 0: no wait has run out, and copies may go on
    PtFound found = {0, 0, false, 0};                   // warp 0: where it has looked for pairs
    bool appended = false;                    // warp 0: the append has been waited for
    // warp 0: a pair's queries, behind those of q pairs before; and its pieces p .. end - 1 of the ring,
    // where `first` is the first of them
    auto copy_q = [&](const PtWork& y, const PtRun& run, int q) {
        if (run.nc == 0) return;
        if (q > 0) good = good && warp_ok(qempty, (uint32_t)(q - 1) & 1u);
        if (good && tc::elect_one()) {
            const int boxes = run.nc1 > 0 ? 2 : 1;
            tc::mbar_arrive_expect_tx(qfull, (uint32_t)(boxes * 2 * per * R * 128));
            for (int i = 0; i < boxes; ++i)
                for (int h = 0; h < 2; ++h)
                    tc::tma_load_3d(sm + L::kQ + i * kPtTile + h * kPtPanel, &tmq, 64 * h, y.g * R, y.row0 + run.t0 + i * per, qfull);
        }
        __syncwarp();
    };
    auto copy_pieces = [&](const PtWork& y, const PtRun& run, int first, int p, int end) {
        if (y.before > 0 && !appended) pdl_wait(), appended = true;
        good = good && ring_fill(ring, first, p, end, [&](int p) {
            const int at = stage(first + p);
            if (tc::elect_one()) {
                if (p >= 2 * run.nc) {  // room for an output
                    tc::mbar_arrive(full + at);
                } else {
                    tc::mbar_arrive_expect_tx(full + at, kPtTile);
                    uint8_t* to = sm + L::kRing + at * kPtTile;
                    const int p0 = (run.cb + (p >> 1)) * kPtPos;
                    for (int h = 0; h < 2; ++h)
                        if (y.before > 0)  // from the caches
                            tc::tma_load_3d(to + h * kPtPanel, p & 1 ? &tmv : &tmk, 64 * h, p0, y.s * a.Hkv + y.g, full + at);
                        else  // from the rows themselves
                            tc::tma_load_3d(to + h * kPtPanel, p & 1 ? &tmvn : &tmkn, 64 * h, y.g, y.row0 + p0, full + at);
                }
            }
            __syncwarp();
        });
    };
    // pieces that are copied before the pair ahead of theirs ends (they wait for nothing of their own pair's)
    constexpr int kAhead = 3;

    if (warp == 0) {
        if (lane == 0) {
            prefetch_map(&tmq), prefetch_map(&tmo);
            prefetch_map(&tmk), prefetch_map(&tmv), prefetch_map(&tmkn), prefetch_map(&tmvn);
            for (int i = 0; i < kPtStages; ++i) tc::mbar_init(full + i, 1), tc::mbar_init(empty + i, 1), tc::mbar_init(ready + i, 1);
            tc::mbar_init(qfull, 1), tc::mbar_init(qempty, 1), tc::mbar_init(next, 1), tc::mbar_init(endbar, 1);
            tc::mbar_init(passed, kPtThreads / 32 - 1);
            for (int i = 0; i < 2; ++i) tc::mbar_init(sfull + i, 1), tc::mbar_init(ofull + i, 1);
            tc::fence_mbar_init();
            *flag = 0;
        }
        __syncwarp();
        // (The kernel before this one is this call's append, which has waited for what came before
        // it: only the caches are its own. They are waited for where they are read, and at the end,
        // so that whoever waits for this kernel has waited for the append too.)
        const PtWork y = find_pair(a, span, (int)blockIdx.x / W, &found);
        if (lane == 0) *work(0) = y;
        if (y.s >= 0) {
            const PtRun run(a, y, per, span, W, wk);
            copy_q(y, run, 0);
        }
    } else if (warp == 1) {
        tc::tmem_alloc(sTmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tm = *sTmem;
    pdl_trigger();  // not before the tensor memory is held: the next kernel may take some before it waits for this one

    // Each warp's loop over the CTA's pairs: role(y, run, k, q pairs with chunks before, first piece).
    // A tile's softmax goes on to the next pair by itself; warp 0 lets no warp fall two pairs behind.
    auto every_pair = [&](auto role) {
        PtWork y = *work(0);
        for (int k = 0, q = 0, first = 0; y.s >= 0; ++k) {
            const PtRun run(a, y, per, span, W, wk);
            role(y, run, k, q, first);
            first += run.pieces;
            q += run.nc > 0;
            __syncwarp();
            if (W > 1) break;
            if (warp > 0) pair_wait(warp);
            y = *work(k + 1);
            __syncwarp();
            if (warp > 0 && lane == 0) tc::mbar_arrive(passed);
        }
    };
    if (warp >= 4) {
        regs_up<kRegsMany>();
        int chunks = 0, walks = 0;  // of the tile so far
        const int i = (warp - 4) >> 2, r = tid - 128 - 128 * i;  // tile, row of it
        const int rt = i * per + r / R, rt0 = i * per + (r & ~31) / R;  // its packed row of the pair's, and the warp's first
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tm + lanes + kColS + 128 * i, tO = tm + lanes + kColO + 128 * i;
        const int head = r % R;
        uint64_t* leaving = nullptr;  // thread 0 of the tile: the piece whose rows are still being copied out
        auto left = [&] {
            if (!leaving) return;
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            tc::mbar_arrive(leaving);
            leaving = nullptr;
        };
        every_pair([&](const PtWork& y, const PtRun& run, int k, int before, int first) {
            // -------------------------------------- softmax, one row a thread
            const int t = run.t0 + rt;
            // The last position seen. (A row behind the tile's last goes with what the last one sees:
            // hiding all from it took its warp 700 cycles more a chunk, and 80 us of the size below.)
            const int lim = min(y.before + t, run.total - 1);
            // ... and the fewest that a row of the warp sees
            const int least = min(y.before + run.t0 + rt0, run.total - 1);
            const int nci = i ? run.nc1 : run.nc0;
            // (Not 0, since hidden scores are -infinity: a scale of 0 counts as the least number above it, which
            // leaves any finite product below 1e-6.)
            const float cs = fmaxf(fabsf(a.scale) * kLog2e * kCutOff, FLT_TRUE_MIN);
            bool here = true;
            float m = kNone;
            float2 l0 = make_float2(0.f, 0.f), l1 = l0;  // the row's sum, in four parts
            // the weights of the run's chunk j from its scores
            auto softmax_chunk = [&](int j) -> bool {
                if (!warp_ok(sfull + i, (uint32_t)(chunks + j) & 1u)) return false;
                tc::tc_fence_after();
                const int p0 = (run.cb + j) * kPtPos, see = lim - p0;  // columns 0 .. see are seen
                float v[kPtPos], tops[8];                              // the scores, and their maxima
#pragma unroll
                for (int b = 0; b < 8; ++b) tmem_ld16_max(tS + 16 * b, v + 16 * b, tops[b]);
                tc::tmem_wait_ld();
                if (least - p0 < kPtPos - 1) {
#pragma unroll
                    for (int b = 0; b < 8; ++b) {
                        if (least - p0 >= 16 * b + 15) continue;  // (the same in the whole warp)
                        float* w = v + 16 * b;
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = 16 * b + e <= see ? w[e] : -INFINITY;
                        tops[b] = max3(max3(max3(w[0], w[1], w[2]), max3(w[3], w[4], w[5]), max3(w[6], w[7], w[8])),
                                       max3(w[9], w[10], w[11]), max3(fmaxf(w[12], w[13]), w[14], w[15]));
                    }
                }
                const float mx =
                    max3(max3(tops[0], tops[1], tops[2]), max3(tops[3], tops[4], tops[5]), fmaxf(tops[6], tops[7])) * cs;
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
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[h][e] * f);
                            tmem_st16(tO + 32 * q + 16 * h, w);
                        }
                    }
                }
                const float2 nm = make_float2(-m, -m), c2 = make_float2(cs, cs);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 x = fma2(make_float2(v[32 * q + 2 * e], v[32 * q + 2 * e + 1]), c2, nm);
                        const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                        if (e & 1)
                            l1 = add2(l1, p);
                        else
                            l0 = add2(l0, p);
                        w[e] = pack_bf16x2(p.x, p.y);
                    }
                    tmem_st16(tS + 16 * q, w);  // over S, which is read
                }
                tc::tmem_wait_st();
                return true;
            };
            left();
            tc::tc_fence_before();
            tile_rows_meet(TileBarriers(), i, nci, [&](int j) {
                here = here && softmax_chunk(j);
                tc::tc_fence_before();
            });
            chunks += nci;
            float l = (l0.x + l0.y) + (l1.x + l1.y);
            if (nci > 0) {
                here = here && warp_ok(ofull + i, (uint32_t)walks++ & 1u);
                tc::tc_fence_after();
            }
            // -------------------------------------------------------- O out
            const bool live = r < per * R && t < run.row_end;
            float poison = 0.f;  // NaN where the row sees a value that was not finite
            const uint32_t* bads = bad_of(k);
            if (nci > 0 && bads[kPtBad - 1]) {
                for (int e = 0; e < 4 * (run.cb + run.nc - run.cut); ++e) {
                    const int see = lim - run.cut * kPtPos - 32 * e;
                    const uint32_t off = bads[e];
                    if (see >= 0 && (off & (see >= 31 ? ~0u : (2u << see) - 1u))) poison = NAN;
                }
            }
            if (W == 1) {
                if (run.t0 + i * per >= run.row_end) return;  // the tile has no rows
                const size_t packed = (size_t)y.row0 + t;
                if (!run.ok) {  // a refused session has no pieces of the ring: each row's zeros from its own thread
                    if (!live) return;
                    uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + packed * a.out_stride +
                                                         (size_t)(y.g * R + head) * kAttnD);
#pragma unroll 1
                    for (int e = 0; e < kAttnD / 8; ++e) to[e] = make_uint4(0u, 0u, 0u, 0u);
                    if (a.lse) a.lse[packed * a.Hq + y.g * R + head] = -INFINITY;
                    return;
                }
                // in bf16 to a piece of the ring, laid out as the queries were; a whole tile leaves by two
                // copies of a thread, the last of a session two rows at a time (16 lanes a row)
                // (The stage's turn before is over: that was a key or value of this pair that the tile's
                // products have read, or a piece ahead of one.)
                const int piece = first + 2 * run.nc + i, at = stage(piece);
                here = ring_room(ring, piece) && here;
                uint8_t* mine = sm + L::kRing + at * kPtTile;
                const float f = 1.f / l + poison;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    float v[32];
                    tmem_ld32(tO + 32 * q, v);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int h = 0; h < 4; ++h) w[h] = pack_bf16x2(v[e + 2 * h] * f, v[e + 2 * h + 1] * f);
                        *reinterpret_cast<uint4*>(mine + (q >> 1) * kPtPanel + r * 128 + (((4 * (q & 1) + e / 8) ^ (r & 7)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                if (live && a.lse) a.lse[packed * a.Hq + y.g * R + head] = fmaf(m, kLn2, logf(l));
                if (run.t0 + (i + 1) * per <= run.row_end) {
                    tc::fence_proxy_async_smem();
                    tile_sync(i);
                    if (r == 0) {
                        for (int h = 0; h < 2; ++h)
                            tma_store_3d(&tmo, 64 * h, y.g * R, y.row0 + run.t0 + i * per, mine + h * kPtPanel);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        leaving = empty + at;
                    }
                } else {
                    __syncwarp();
                    const size_t to_row = packed * a.out_stride + (size_t)(y.g * R + head) * kAttnD;
                    const unsigned lives = __ballot_sync(0xffffffffu, live);
#pragma unroll 1
                    for (int e = 0; e < 16; ++e) {
                        const int rr = 2 * e + (lane >> 4), col = lane & 15;
                        const size_t to = __shfl_sync(0xffffffffu, to_row, rr);
                        if (lives >> rr & 1u)
                            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + to + 8 * col) =
                                *reinterpret_cast<const uint4*>(mine + (col >> 3) * kPtPanel + ((r & ~31) + rr) * 128 +
                                                                (((col & 7) ^ (rr & 7)) << 4));
                    }
                    tc::fence_proxy_async_smem();  // (read before a copy may come over it)
                    tile_sync(i);
                    if (r == 0) tc::mbar_arrive(empty + at);
                }
            } else {
                const bool some = here && nci > 0;  // (the same in the whole warp)
                if (!some) m = kNone, l = 0.f;
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
                        for (int e = 0; e < 32; ++e) v[e] = 0.f;
                    }
                    // 16-byte pieces rotated by the row, so that a warp's rows do not meet in one bank
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<float4*>(sm + L::kRing + row * kAttnD * 4 + (((8 * q + e + row) & 31) << 4)) =
                            make_float4(v[4 * e] + poison, v[4 * e + 1] + poison, v[4 * e + 2] + poison, v[4 * e + 3] + poison);
                }
                *reinterpret_cast<float2*>(sm + L::kMl + row * 8) = make_float2(m, l);
            }
        });
        left();
        } else {
        regs_down<kRegsFew>();
        every_pair([&](const PtWork& y, const PtRun& run, int k, int before, int first) {
            if (warp == 0) {
                // -------------------------------------------------------- copies
                if (W == 1 && lane == 0) {
                    tc::mbar_arrive_expect_tx(next, 16);
                    ask_next(sm + L::kNext, next);
                }
                __syncwarp();
                // (first what need not wait for this pair's products, then the next pair, then the rest)
                const int had = k > 0 ? min(kAhead, run.pieces) : 0, soon = min(kPtStages, run.pieces);
                copy_pieces(y, run, first, had, soon);
                PtWork z = {-1, 0, 0, 0, 0, 0};
                if (W == 1) {
                    good = good && warp_ok(next, (uint32_t)k & 1u);
                    const int x = good ? answer_next(sm + L::kNext) : -1;
                    tc::fence_proxy_async_smem();  // (the answer is read before another may come)
                    __syncwarp();
                    if (x >= 0) z = find_pair(a, span, x, &found);
                    // (where the wait runs out, the others' waits end as soon as that is known: a second
                    // one sees them pass)
                    if (k > 0 && !warp_ok(passed, (uint32_t)(k - 1) & 1u)) good = false, tc::mbar_wait(passed, (uint32_t)(k - 1) & 1u);
                    if (lane == 0) *work(k + 1) = z;
                    __syncwarp();
                    pair_known();
                }
                copy_pieces(y, run, first, soon, run.pieces);
                if (z.s >= 0) {
                    const PtRun then(a, z, per, span, W, wk);
                    copy_q(z, then, before + (run.nc > 0));
                    copy_pieces(z, then, first + run.pieces, 0, min(kAhead, then.pieces));
                }
            } else if (warp == 1) {
                // ------------------------------------------------------ products
                const bool leader = tc::elect_one();
                const uint32_t sbase = tc::smem_u32(sm);
                // (a scale's sign goes into the products, so that the maxima are those of S)
                const uint32_t scores = tc::idesc_bf16(kPtRows, kPtPos, 0, 0) | (a.scale < 0.f ? tc::kIdescNegateA : 0u);
                tile_turns_meet(TileBarriers(), run.nc, run.nc0, run.nc1, [](int) {}, [&](int i, int j) {
                    const int nci = i ? run.nc1 : run.nc0;
                    // the last of the tiles that read this chunk (tile 1 takes every one, where there is one)
                    const bool last = i == 1 || run.nc1 == 0;
                    tc::tc_fence_after();
                    if (leader) {
                        if (j > 0) {  // O += p V of chunk j - 1
                            const int at = stage(first + 2 * j - 1);
                            const uint64_t bd = tc::sdesc(sbase + L::kRing + at * kPtTile, kPtPanel, 1024, 2);
    #pragma unroll
                            for (int q = 0; q < 8; ++q)
                                tc::mma_bf16_tmem_a(tm + kColO + 128 * i, tm + kColS + 128 * i + 8 * q, bd + (uint64_t)(q * 2048 >> 4),
                                                    tc::idesc_bf16(kPtRows, kAttnD, 0, 1), (j > 1 || q > 0) ? 1u : 0u);
                            if (last) tc::mma_commit(empty + at);
                        }
                        if (j < nci) {  // S = q K^T of chunk j, over the weights
                            const int at = stage(first + 2 * j);
                            const uint64_t ad = tc::sdesc(sbase + L::kQ + i * kPtTile, 0, 1024, 2);
                            const uint64_t bd = tc::sdesc(sbase + L::kRing + at * kPtTile, 0, 1024, 2);
    #pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                const uint64_t off = (uint64_t)(((q >> 2) * kPtPanel + (q & 3) * 32) >> 4);
                                tc::mma_bf16(tm + kColS + 128 * i, ad + off, bd + off, scores, q > 0 ? 1u : 0u);
                            }
                            tc::mma_commit(sfull + i);
                            if (last) tc::mma_commit(empty + at);
                            if (last && j == run.nc - 1) tc::mma_commit(qempty);
                        } else {
                            tc::mma_commit(ofull + i);
                        }
                    }
                    __syncwarp();
                });
            } else if (warp == 2) {
                // --- waits for the operands from memory on behalf of the products
                // (after one that gave up, what the products read is there, if not what it should be,
                // and the CTA's results are dropped)
                bool here = true;
                tile_turns_meet(TileBarriers(), run.nc, run.nc0, run.nc1, [&](int j) {
                    if (j == 0 && run.nc > 0) here = here && warp_ok(qfull, (uint32_t)before & 1u);
                    if (j < run.nc) here = here && ring.wait_ready(first + 2 * j);
                    if (j > 0) here = here && ring.wait_ready(first + 2 * j - 1);
                }, [](int, int) {});
            } else {
                // ---------------------------- what has landed, looked over in turn
                uint32_t* bads = bad_of(k);
                if (lane < kPtBad) bads[lane] = 0u;
                __syncwarp();
                ring_look(ring, first, run.pieces, [&](int p) {
                    const int at = stage(first + p), c = run.cb + (p >> 1);
                    if (c < run.cut) return;  // most of them: nothing to do
                    if ((p & 1) && p < 2 * run.nc) {
                        // positions of the chunk from `from` on are not seen by every row, and there is nothing from
                        // `left` on; lanes 0 .. 15 have the 16 pieces of a position, 16 .. 31 of the next
                        const int from = max(run.all - c * kPtPos, 0), left = min(run.total - c * kPtPos, kPtPos);
                        uint32_t* bad = bads + 4 * (c - run.cut);
                        uint8_t* mine = sm + L::kRing + at * kPtTile + (lane & 7) * 16 + ((lane >> 3) & 1) * kPtPanel;
                        for (int p0 = from + (lane >> 4); p0 < left; p0 += 4) {
                            uint4 w[2];
    #pragma unroll
                            for (int q = 0; q < 2; ++q)
                                if (p0 + 2 * q < left) w[q] = *reinterpret_cast<const uint4*>(mine + (p0 + 2 * q) * 128);
    #pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                if (p0 + 2 * q >= left) break;
                                const uint32_t u[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
                                bool off = false;
    #pragma unroll
                                for (int e = 0; e < 4; ++e) off |= (u[e] & 0x7F80u) == 0x7F80u || (u[e] & 0x7F800000u) == 0x7F800000u;
                                if (off) {
                                    *reinterpret_cast<uint4*>(mine + (p0 + 2 * q) * 128) = make_uint4(0u, 0u, 0u, 0u);
                                    atomicOr(bad + ((p0 + 2 * q) >> 5), 1u << ((p0 + 2 * q) & 31));
                                    bads[kPtBad - 1] = 1u;
                                }
                            }
                        }
    #pragma unroll 1
                        for (int q = left + (lane >> 4); q < kPtPos; q += 2)
                            *reinterpret_cast<uint4*>(mine + q * 128) = make_uint4(0u, 0u, 0u, 0u);
                        tc::fence_proxy_async_smem();
                    }
                });
            }
        });
    }
    if (warp == 0 && !appended) pdl_wait();
    __syncthreads();
    const PtWork y = *work(0);  // W > 1: the only one
    const bool none = y.s < 0;  // ... of the whole cluster
    if (*flag) {                // (the same in the whole CTA: nobody waits any more)
        // the copies in flight must land and every product issued must be done
        // before the tensor memory is freed and the CTA exits (all bounded)
        if (warp == 0 && tc::elect_one()) {
            for (uint32_t b = 0; b < 2; ++b) {
                tc::mbar_wait(qfull, b, 100000000ull), tc::mbar_wait(next, b, 100000000ull);
                for (int i = 0; i < kPtStages; ++i) tc::mbar_wait(full + i, b, 100000000ull);
            }
        } else if (warp == 1 && tc::elect_one()) {
            tc::mma_commit(endbar);
            tc::mbar_wait(endbar, 0, 100000000ull);
        }
        __syncthreads();
    }
    if (warp == 1) tc::tmem_dealloc(tm, 512);
    if (W == 1 || none) return;
    const PtRun run(a, y, per, span, W, wk);
    tc::cluster_wait();    // (pairs with the arrival at the start)
    tc::cluster_arrive();  // every CTA's rows are in its shared memory ...
    tc::cluster_wait();
    // ... and each reads the rows that it owns
    if (W == 2)
        merge_rows<2>(a, sm, wk, y, run, per);
    else if (W == 4)
        merge_rows<4>(a, sm, wk, y, run, per);
    else
        merge_rows<8>(a, sm, wk, y, run, per);
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

}  // namespace

cudaError_t launch_attn_prompt_tiles(const PromptArgs& a, cudaStream_t st) {
    const PtSetup* setup = nullptr;
    cudaError_t e = prompt_setup(&setup);
    if (e != cudaSuccess) return e;
    const int R = a.Hq / a.Hkv, per = kPtRows / R;
    CUtensorMap tmq, tmo, tmk, tmv, tmkn, tmvn;
    const cuuint64_t row = kAttnD * 2;
    e = make_rows_map(a.q, a.Hq, a.rows, row, (cuuint64_t)a.q_stride * 2, R, per, &tmq);
    if (e == cudaSuccess) e = make_rows_map(a.k_cache, a.Tmax, (cuuint64_t)a.S * a.Hkv, row, row * a.Tmax, kPtPos, 1, &tmk);
    if (e == cudaSuccess) e = make_rows_map(a.v_cache, a.Tmax, (cuuint64_t)a.S * a.Hkv, row, row * a.Tmax, kPtPos, 1, &tmv);
    if (e == cudaSuccess) e = make_rows_map(a.k_new, a.Hkv, a.rows, row, (cuuint64_t)a.kv_stride * 2, 1, kPtPos, &tmkn);
    if (e == cudaSuccess) e = make_rows_map(a.v_new, a.Hkv, a.rows, row, (cuuint64_t)a.kv_stride * 2, 1, kPtPos, &tmvn);
    if (e == cudaSuccess) e = make_rows_map(a.out, a.Hq, a.rows, row, (cuuint64_t)a.out_stride * 2, R, per, &tmo);
    if (e != cudaSuccess) return e;
    long pairs = most_tiles(a.S, a.rows, 2 * per) * a.Hkv;
    // CTAs that share a pair's positions: the least time, in chunks (of 1.4 us), with
    // 4 for a CTA's start and end and 2 more for the merge. One session's CTAs are all
    // alike: rounds x a CTA's time. Several sessions are mostly shorter than the caches:
    // the longest, and where not all CTAs are held at once, what the others take. (Six
    // sessions adding up to 75 rows behind up to 3001: 41 us with one CTA a pair, 30 with
    // two, 37 with four; one adding 75 behind 7400: 87, 54, 33 and 45 with eight, of which
    // the device holds less than the 16 clusters at once; 300 behind 3000: 43, 31, 42, 68;
    // one of 1500: 37, 66, 102, 224.)
    const long reach = a.lens || a.rows > a.Tmax ? a.Tmax : a.rows, chunks = (reach + kPtPos - 1) / kPtPos;
    int W = 1, at = 0;
    float best = 0.f;
    for (int k = 0, w = 1; k < 4 && (w == 1 || w <= chunks) && setup->held[k] > 0; ++k, w *= 2) {
        const float part = (float)pairs / (float)setup->held[k], walk = (float)((chunks + w - 1) / w), ends = w > 1 ? 6.f : 4.f;
        const float cost = a.S == 1 ? fmaxf(1.f, ceilf(part)) * (walk + ends)
                                    : walk + ends + (part > 1.f ? (part - 0.7f) * (0.3f * walk + ends) : 0.f);
        if (w == 1 || cost < best) best = cost, W = w, at = k;
    }
    // A tile a CTA, not a pair, while that leaves some SMs free: nothing of a chunk waits for the other tile.
    // (One session of 100: 8.4 us, 10.3 in pairs; of 300 11.2 and 11.9; of 75 behind 7400 31.2 and 32.5; where
    // they take almost every SM and the next kernel's CTAs wait for them, one of 450: 14.4 and 13.3.)
    const long single = most_tiles(a.S, a.rows, per) * a.Hkv;
    const int tiles = single * W <= 130 && single <= setup->held[at] ? 1 : 2;
    if (tiles == 1) pairs = single;
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
    return cudaLaunchKernelEx(&cfg, attn_prompt_tile_kernel, a, tmq, tmo, tmk, tmv, tmkn, tmvn, W, tiles);
}

}  // namespace m2
