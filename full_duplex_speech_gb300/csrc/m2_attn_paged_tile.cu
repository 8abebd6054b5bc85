// Attention over the paged e4m3 cache for many rows (a prefill, sessions
// catching up, cross attention of a whole sequence), bf16 activations, on the
// tcgen05 tensor cores. The operator and its formulas are those of
// m2_attn_paged.cu; a kv head's rows are its (query, head) pairs, row = t R + r.
//
// One CTA takes two tiles of 128 rows of one (session, kv head) and walks the
// positions they see, 128 at a time. Per chunk and tile:
//   S = q K^T       kind::f8f6f4 straight from the cache's codes. A query row,
//                   scaled by a power of two to a largest element in
//                   [2^11, 2^12), enters as two terms, hi in e5m2 and lo in
//                   e4m3: 8 significant bits, which is all of a bf16, for
//                   elements from 2^-13 of the largest on (hi leaves at most
//                   16 steps of the last bit, which lo holds); below, off by
//                   at most 2^-21 of the largest and 2^-3 of themselves. At
//                   the cost of one product in 16 bits and with no conversion
//                   of the keys. (Both in e4m3, the largest in [2^7, 2^8),
//                   were off by 2^-17 of it, exact from 2^-9 on.)
//   softmax         one thread a row, S read out of tensor memory in fp32 with
//                   each block's maximum (tcgen05.ld.red):
//                   x = S (scale ks), p = 2^(x - m), l += p, and the weight
//                   w = p vs 2^(m - mv + 7) to fp16 (2^-11) over S;
//   O += w V        kind::f16, w from tensor memory, V converted to fp16
//                   (exactly) by four warps.
// m and mv (the reference of the weights, a maximum of x + log2 vs) move only
// when a chunk exceeds them by more than 2^8, which p <= 2^8 in fp32 and
// w <= 2^15 in fp16 allow; only then is O rescaled in tensor memory.
//     out = 2^(mv - m - 7) O / l.
//
// Warps: 0 copies (pages by TMA through rings, scales by 4-byte asynchronous
// copies), 1 issues the products, 2 waits for their operands, 4-7 convert V,
// 8-11 and 12-15 the softmax of the tiles. One warp issues for both tiles, in
// turn: two of their own let the tiles fall into step, both in the softmax
// and then both in the products (716 us against 665 when both were tried, at
// the size below). The products of one tile run under the other's softmax.
// Where few CTAs would leave SMs idle, W CTAs of a cluster share the positions
// of one pair of tiles and merge through distributed shared memory, each the
// owner of 256 / W rows.
//   Measured: 4 sessions of 4096 positions, 40 query and 8 kv heads, causal,
// 687 GFLOP: 559 us, 1.23 PFLOP/s (66% of a bf16 library product's measured
// rate). With references that lagged by 2^15 and softmax warps that did not wait
// in the meetings it took 535, and these cycles: a chunk of a pair 2,880; the
// warp that issues is held by the products for 2,400 of them (about 272 KB pass
// through shared memory, 2,180 cycles of it); a tile's own round, its softmax
// (1,130), the hand-overs and the scales (1,200), and 1,020 of products, is as
// long as that, so that neither alone makes it shorter: an eighth of the products
// left 483 us, no exponentials 527. The scores of the next chunk during the
// softmax (one S for both tiles, the weights in columns of their own) took 567
// where this took 533: the products then wait for one another.
#include <cuda_fp8.h>
#include <float.h>
#include <math.h>

#include <mutex>

#include "m2_paged_dev.cuh"
#include "m2_tile_meet.h"

namespace m2 {

namespace {

constexpr int kTlThreads = 512;
constexpr int kTlRows = 128;                       // rows of a tile
constexpr int kTlTc = 128;                         // positions per chunk
constexpr int kTlBlocks = kTlTc / kKvBlock;        // scales of a chunk
constexpr uint32_t kTlTile = kTlTc * kKvD;         // 16 KB of codes
constexpr int kKStages = 3, kVStages = 2, kHStages = 2, kScStages = kKStages + 1;
constexpr int kQPower = 11;  // a row of q is scaled to a largest element in [2^11, 2^12)
// log2 by which a chunk may exceed m and mv, and log2 of the weight of a position
// at mv: fp16 reaches from 2^15 down to 2^-24, so that a weight is off by 2^-32 of
// the one at mv at most, and is dropped below that (a long flat rest behind one
// dominant position is many of them: with 15 and 0, which took 541 us where this
// takes 561, 2^20 positions of 2^-25 each lost an eighth of themselves; 5 and 10
// took 573). 2^(m - mv + 7) and its inverse stay normal for values up to the
// largest (log2 vs from -109 to 119).
constexpr float kSlackM = 8.f, kSlackV = 8.f, kLift = 7.f;
constexpr uint32_t kColO = 0, kColS = 256;         // tensor memory: O of the two tiles, then S (and w over it)

struct TlSmem {
    static constexpr uint32_t kQ = 0;                                    // [tile][hi, lo] 16 KB, K-major, 128-byte swizzle
    static constexpr uint32_t kK = kQ + 4 * kTlTile;                     // kKStages, the same layout
    static constexpr uint32_t kV = kK + kKStages * kTlTile;              // kVStages
    static constexpr uint32_t kH = kV + kVStages * kTlTile;              // V in fp16, kHStages x 32 KB, MN-major
    static constexpr uint32_t kSc = kH + kHStages * 2 * kTlTile;         // float [stage][ks 8, vs 8]
    static constexpr uint32_t kBar = kSc + kScStages * 2 * kTlBlocks * 4;
    // kfull, kempty, vfull, vempty, hfull, hempty, scfull, sfull[2], ofull[2], end
    static constexpr int kBars = 2 * (kKStages + kVStages + kHStages) + kScStages + 5;
    static constexpr uint32_t kTmem = kBar + kBars * 8;
    static constexpr uint32_t kFlag = kTmem + 4;
    static constexpr uint32_t kBytes = kFlag + 4 + 1024;  // + slack to align to 1024
    // after the walk, over the rings: 256 rows x 128 floats, then their (m, l, mv)
    static constexpr uint32_t kMl = 2 * kTlRows * kKvD * 4;
    static_assert(kMl + 2 * kTlRows * 16 <= kSc, "the merge fits in the rings");
    static_assert(kBytes <= 227 * 1024, "one CTA an SM");
};

__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, bool e5m2) {  // e5m2 or e4m3 x e4m3, both K-major, fp32 sums
    return (1u << 4) | ((uint32_t)e5m2 << 7) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_f16_bmn(int M, int N) {  // fp16 x fp16, B MN-major, fp32 sums
    return (1u << 4) | (1u << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 lanes x 32 consecutive columns: thread t of the warp gets lane base + t.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
          "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// 32 lanes x 16 consecutive columns, and the largest of each lane's 16.
__device__ __forceinline__ void tmem_ld16_max(uint32_t taddr, float* v, float& top) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    uint32_t t;
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, %16, [%17];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(t)
        : "r"(taddr));
    top = __uint_as_float(t);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// pairs of fp32, each rounded as by itself
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
// The warpgroup's registers a thread (multiples of 8): the launch's 128 are
// split into 48 for the copy, product and conversion warps and 208 for the
// softmax warps, and even again before they meet.
template <int N> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
// The meetings of m2_tile_meet.h on hardware barriers, since a look at one in
// shared memory takes some 200 cycles beside the products' own traffic.
struct TileBarriers {
    __device__ __forceinline__ void sync(int i) const { asm volatile("barrier.sync %0, 192;" ::"r"(2 + i) : "memory"); }
};
// The softmax warps give back before anyone takes: a warp that is done early
// must not take what they still wait for.
__device__ __forceinline__ void all_done() { asm volatile("barrier.sync 1, %0;" ::"n"(kTlThreads) : "memory"); }
constexpr int kRegsLaunch = 128, kRegsFew = 48, kRegsMany = 208;
static_assert(256 * kRegsFew + 256 * kRegsMany <= kTlThreads * kRegsLaunch, "the split is covered by the launch's registers");

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// The merge of a cluster's W parts of the rows that CTA wk owns, a warp a row,
// four dims a lane:
//     out = 2^(V - M - 7) sum_w 2^(mv_w - V) O_w / sum_w 2^(m_w - M) l_w
// A warp has 16 / W rows, and all of their parts are on their way together
// (a row after the other took 2 us more of a CTA's 24 with W = 2);
// lane i < 16 holds the references of a part of row i / W. A row's parts are
// taken from the CTA's own on, which needs no other's shared memory.
template <int W>
__device__ __forceinline__ void merge_rows(const PagedAttnArgs& a, uint8_t* sm, int wk, int rows, int row0, int s, int g) {
    constexpr int kWarps = kTlThreads / 32, kParts = 2 * kTlRows / kWarps;  // parts a warp
    const int lane = threadIdx.x & 31, R = a.Hq / a.c.Hkv;
    const int first = wk * (2 * kTlRows / W) + (int)(threadIdx.x >> 5);  // the warp's rows: first, first + kWarps, ...
    if (first >= rows) return;
    uint32_t from[W];
#pragma unroll
    for (int w = 1; w < W; ++w) from[w] = tc::cluster_map(tc::smem_u32(sm), (wk + w) % W);
    const int mine = min(first + kWarps * ((lane & (kParts - 1)) / W), rows - 1);
    const float4 x = ld_cluster_f32x4(tc::cluster_map(tc::smem_u32(sm), (wk + lane) % W) + TlSmem::kMl + mine * 16);
    float4 y[kParts];
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
        const int row = min(first + kWarps * (k / W), rows - 1);
        const uint32_t at = row * kKvD * 4 + (((lane + row) & 31) << 4);
        y[k] = k % W ? ld_cluster_f32x4(from[k % W] + at) : *reinterpret_cast<const float4*>(sm + at);
    }
    float M = x.x, V = x.z;
#pragma unroll
    for (int off = 1; off < W; off <<= 1) {
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        V = fmaxf(V, __shfl_xor_sync(0xffffffffu, V, off));
    }
    const float f = ex2_approx(x.z - V);
    float sum = ex2_approx(x.x - M) * x.y;
#pragma unroll
    for (int off = 1; off < W; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    const float whole = sum == 0.f ? 0.f : ex2_approx(V - M - kLift) / sum;  // a row that sees nothing: zeros
    const int rr = row0 + mine;
    const long at = ((long)s * a.T + rr / R) * a.out_stride + (long)(g * R + rr % R) * kKvD;
#pragma unroll
    for (int n = 0; n < kParts / W; ++n) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float fw = __shfl_sync(0xffffffffu, f, n * W + w);
            const float4 v = y[n * W + w];
            o.x = fmaf(fw, v.x, o.x), o.y = fmaf(fw, v.y, o.y), o.z = fmaf(fw, v.z, o.z), o.w = fmaf(fw, v.w, o.w);
        }
        const float by = __shfl_sync(0xffffffffu, whole, n * W);
        const long to = __shfl_sync(0xffffffffu, at, n * W);
        if (first + kWarps * n < rows)
            *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + to + 4 * lane) =
                make_uint2(pack_bf16x2(o.x * by, o.y * by), pack_bf16x2(o.z * by, o.w * by));
    }
}

// grid (W x Hkv x row pairs, S), a cluster of W CTAs when W > 1
__global__ void __launch_bounds__(kTlThreads, 1)
    attn_paged_tile_kernel(PagedAttnArgs a, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                           int W, bool ranked) {
    using L = TlSmem;
    extern __shared__ uint8_t tl_raw[];
    uint8_t* sm = tl_raw + ((1024u - (tc::smem_u32(tl_raw) & 1023u)) & 1023u);
    float* scales = reinterpret_cast<float*>(sm + L::kSc);
    uint64_t* kfull = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint64_t *kempty = kfull + kKStages, *vfull = kempty + kKStages, *vempty = vfull + kVStages, *hfull = vempty + kVStages,
             *hempty = hfull + kHStages, *scfull = hempty + kHStages,
             *sfull = scfull + kScStages, *ofull = sfull + 2, *endbar = ofull + 2;
    uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + L::kTmem);
    volatile uint32_t* flag = reinterpret_cast<uint32_t*>(sm + L::kFlag);
    const KvCache& c = a.c;
    const int wk = (int)blockIdx.x % W;
    int s = blockIdx.y;
    // the row pairs from the last on: under a causal limit they take longest
    const int pair = (int)(gridDim.x - 1 - blockIdx.x) / W;
    const int g = pair % c.Hkv, row0 = pair / c.Hkv * (2 * kTlRows);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int R = a.Hq / c.Hkv;

    if (tid == 32) prefetch_map(&tmk), prefetch_map(&tmv);
    if (W > 1) tc::cluster_arrive_relaxed();  // waited on before the first remote store: every CTA has started
    pdl_wait();  // the queries and the cache may come from the previous kernel
    if (ranked) {
        // More CTAs than the GPU holds at once, in the order of blockIdx: the
        // sessions by the positions that their last rows see, the most first. (At
        // most a session a thread.)
        int* key = reinterpret_cast<int*>(sm + L::kH);  // (of the values, which come later)
        int mine = -1;
        if (tid < c.S) {
            const int m = a.n_new ? min(a.n_new[tid], a.T) : a.T, L0 = a.lens[tid];
            if (m > 0 && L0 >= 0 && L0 <= c.capacity()) mine = L0 + m;
        }
        key[tid] = mine;
        __syncthreads();
        if (tid < c.S) {
            int rank = 0;
#pragma unroll 8
            for (int u = 0; u < c.S; ++u) rank += key[u] > mine || (key[u] == mine && u < tid);
            if (rank == (int)blockIdx.y) key[kTlThreads] = tid;
        }
        __syncthreads();
        s = key[kTlThreads];
    }
    int before, n;
    const bool ok = kv_extent(c, s, a.T, a.lens, a.n_new, a.causal ? c.capacity() : c.capacity() + a.T, &before, &n) &&
                    before <= c.capacity();
    if (!ok && blockIdx.x == 0 && tid == 0) record_error(c.err, ERR_ATTN_LENGTH);
    const int rows = min(n * R - row0, 2 * kTlRows);
    if (rows <= 0) return;  // the whole cluster
    // positions that the tiles' last rows see, and this CTA's run of chunks
    auto seen_by = [&](int last) { return !ok ? 0 : a.causal ? before + (row0 + last) / R + 1 : before; };
    const int total = seen_by(rows - 1);
    const int nch = (total + kTlTc - 1) / kTlTc, cpw = (nch + W - 1) / W;
    const int cb = min(wk * cpw, nch), nc = min(cpw, nch - cb);  // chunks cb .. cb + nc - 1
    const int total0 = seen_by(min(rows, kTlRows) - 1);
    const int nc0 = min(max((total0 + kTlTc - 1) / kTlTc - cb, 0), nc);  // of which tile 0 takes so many
    const int nc1 = rows > kTlRows ? nc : 0;

    if (tid == 0) {
        for (int i = 0; i < kKStages; ++i) tc::mbar_init(kfull + i, 1), tc::mbar_init(kempty + i, 1);
        for (int i = 0; i < kVStages; ++i) tc::mbar_init(vfull + i, 1), tc::mbar_init(vempty + i, 4);
        for (int i = 0; i < kHStages; ++i) tc::mbar_init(hfull + i, 4), tc::mbar_init(hempty + i, 1);
        for (int i = 0; i < kScStages; ++i) tc::mbar_init(scfull + i, 32);
        for (int i = 0; i < 2; ++i) tc::mbar_init(sfull + i, 1), tc::mbar_init(ofull + i, 1);
        tc::mbar_init(endbar, 1);
        tc::fence_mbar_init();
        *flag = 0;
    }
    if (warp == 1) {
        tc::tmem_alloc(sTmem, 512);
        tc::tmem_relinquish();
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
        record_error(c.err, ERR_MBAR_TIMEOUT_MMA);
        *flag = 1;
        return false;
    };
    // the same for a converged warp
    auto warp_ok = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait_ok(bar, parity)); };

    float m = kNone, mv = kNone, l = 0.f;  // of a softmax thread's row
    if (warp < 8) {
        regs_down<kRegsFew>();
        if (warp == 0) {
            // ------------------------------------------------------------ copies
            const int* table = c.table + (size_t)s * c.max_pages;
            const int pieces = kTlTc >> c.ps_shift;  // pages a chunk (a page holds at most a chunk)
            const uint32_t page_bytes = (uint32_t)c.ps * kKvD;
            const int last_page = (total - 1) >> c.ps_shift;
            int held = -32, page_ids = 0;  // this lane's entry of table[held .. held + 31]
            for (int j = 0; j < nc; ++j) {
                const int p0 = (cb + j) * kTlTc, first = p0 >> c.ps_shift;
                if (held < 0 || first + pieces > held + 32) {
                    held = first;
                    page_ids = first + lane <= last_page ? table[first + lane] : 0;
                    if (page_ids < 0 || page_ids >= c.n_pages) {
                        record_error(c.err, ERR_KV_PAGE);
                        page_ids = 0;  // some page of the pool: what is read is undefined
                    }
                    __syncwarp();
                }
                const int live = min(pieces, last_page - first + 1);
                const int ks = j % kKStages, vs = j % kVStages, ss = j % kScStages;
                // lane i < live copies page first + i
                const int y = (__shfl_sync(0xffffffffu, page_ids, first - held + min(lane, pieces - 1)) * c.Hkv + g) * c.ps;
                if (j >= kKStages && !warp_ok(kempty + ks, (uint32_t)(j / kKStages - 1) & 1)) break;
                if (lane == 0) tc::mbar_arrive_expect_tx(kfull + ks, live * page_bytes);
                __syncwarp();
                if (lane < live) tc::tma_load_2d(sm + L::kK + ks * kTlTile + lane * page_bytes, &tmk, 0, y, kfull + ks);
                __syncwarp();
                // The scales' ring has one stage more than the keys': the keys of chunk j waited for
                // the scores of chunk j - 3, which are issued when both tiles are done with the
                // scales of chunk j - 4.
                {
                    const int b = lane & (kTlBlocks - 1), p = p0 + b * kKvBlock;  // lanes 0 .. 7 the keys' scales, 8 .. 15 the values'
                    const int page = __shfl_sync(0xffffffffu, page_ids, min((p >> c.ps_shift) - held, 31));
                    if (lane < 2 * kTlBlocks && p < total) {
                        const size_t at = (((size_t)page * c.Hkv + g) << (c.ps_shift - 4)) + ((p & (c.ps - 1)) >> 4);
                        cp_async4(scales + ss * 2 * kTlBlocks + lane, (lane < kTlBlocks ? c.ks : c.vs) + at);
                    }
                    cp_async_arrive(scfull + ss);
                }
                if (j >= kVStages && !warp_ok(vempty + vs, (uint32_t)(j / kVStages - 1) & 1)) break;
                if (lane == 0) tc::mbar_arrive_expect_tx(vfull + vs, live * page_bytes);
                __syncwarp();
                if (lane < live) tc::tma_load_2d(sm + L::kV + vs * kTlTile + lane * page_bytes, &tmv, 0, y, vfull + vs);
                __syncwarp();
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else if (warp == 1) {
            // ---------------------------------------------------------- products
            const bool leader = tc::elect_one();
            const uint32_t sbase = tc::smem_u32(sm);
            tile_turns_meet(TileBarriers(), nc, nc0, nc1, [](int) {}, [&](int i, int j) {
                const int nci = i ? nc1 : nc0, h = (j + kHStages - 1) % kHStages, k8 = j % kKStages;
                tc::tc_fence_after();
                if (leader) {
                    if (j > 0) {  // O += w V of chunk j - 1
                        const uint64_t bd = tc::sdesc(sbase + L::kH + h * 2 * kTlTile, 2048, 128, 0);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            tc::mma_bf16_tmem_a(tm + kColO + 128 * i, tm + kColS + 128 * i + 8 * k,
                                                bd + (uint64_t)(k * 4096 >> 4), idesc_f16_bmn(kTlRows, kKvD),
                                                (j > 1 || k > 0) ? 1u : 0u);
                        // the last tile that reads this V releases it (tile 1 takes every chunk, where there is one)
                        if (i == 1 || nc1 == 0) tc::mma_commit(hempty + h);
                    }
                    if (j < nci) {  // S = q K^T of chunk j, over the weights
                        const uint64_t bd = tc::sdesc(sbase + L::kK + k8 * kTlTile, 0, 1024, 2);
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
                            const uint64_t ad = tc::sdesc(sbase + L::kQ + (2 * i + part) * kTlTile, 0, 1024, 2);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_f8(tm + kColS + 128 * i, ad + 2 * k, bd + 2 * k, idesc_f8(kTlRows, kTlTc, part == 0),
                                       (part > 0 || k > 0) ? 1u : 0u);
                        }
                        tc::mma_commit(sfull + i);
                        if (i == 1 || nc1 == 0) tc::mma_commit(kempty + k8);
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
                if (j < nc) good = good && warp_ok(kfull + j % kKStages, (uint32_t)(j / kKStages) & 1);
                if (j > 0) good = good && warp_ok(hfull + (j - 1) % kHStages, (uint32_t)((j - 1) / kHStages) & 1);
            }, [](int, int) {});
        } else if (warp >= 4) {
            // --------------------------------------------- V to fp16, four warps
            const int k7 = lane & 7;
            for (int j = 0; j < nc; ++j) {
                const int vs = j % kVStages, h = j % kHStages;
                if (!warp_ok(vfull + vs, (uint32_t)(j / kVStages) & 1)) break;
                if (j >= kHStages && !warp_ok(hempty + h, (uint32_t)(j / kHStages - 1) & 1)) break;
                const uint8_t* src = sm + L::kV + vs * kTlTile;
                uint8_t* dst = sm + L::kH + h * 2 * kTlTile;
                // positions behind the last count as zero values, and so do those of a block with a
                // scale that is not finite: the rows that see it get their NaN by the weights, and
                // the others none
                const int left = total - (cb + j) * kTlTc;
                if (!warp_ok(scfull + j % kScStages, (uint32_t)(j / kScStages) & 1)) break;
                uint32_t none = 0;  // a bit a block
                {
                    const float* sv = scales + j % kScStages * 2 * kTlBlocks + kTlBlocks;
                    const bool bad = lane < kTlBlocks && !(fabsf(sv[lane & (kTlBlocks - 1)]) < INFINITY);
                    none = __ballot_sync(0xffffffffu, bad);
                }
                // a warp's item: 8 positions (8 pg + k7) x 4 pieces of 16 dims, a piece a lane (16
                // codes, swizzled) -> two 16-byte pieces of the product's 8 x 8 blocks (MN-major);
                // the reads of four items are in flight together
#pragma unroll 1
                for (int it0 = warp - 4; it0 < kTlTc / 4; it0 += 16) {
                    uint4 w[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int it = it0 + 4 * n, sub = 4 * (it & 1) + (lane >> 3);
                        w[n] = *reinterpret_cast<const uint4*>(src + (8 * (it >> 1) + k7) * kKvD + ((sub ^ k7) << 4));
                    }
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int it = it0 + 4 * n, pg = it >> 1, sub = 4 * (it & 1) + (lane >> 3);
                        if (8 * pg + k7 >= left || (none >> (pg >> 1) & 1u)) w[n] = make_uint4(0u, 0u, 0u, 0u);
                        uint4 lo, hi;
                        lo.x = e4m3x2_to_f16x2(w[n].x & 0xFFFFu), lo.y = e4m3x2_to_f16x2(w[n].x >> 16);
                        lo.z = e4m3x2_to_f16x2(w[n].y & 0xFFFFu), lo.w = e4m3x2_to_f16x2(w[n].y >> 16);
                        hi.x = e4m3x2_to_f16x2(w[n].z & 0xFFFFu), hi.y = e4m3x2_to_f16x2(w[n].z >> 16);
                        hi.z = e4m3x2_to_f16x2(w[n].w & 0xFFFFu), hi.w = e4m3x2_to_f16x2(w[n].w >> 16);
                        uint8_t* o = dst + pg * 2048 + sub * 256 + k7 * 16;
                        *reinterpret_cast<uint4*>(o) = lo;
                        *reinterpret_cast<uint4*>(o + 128) = hi;
                    }
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(hfull + h), tc::mbar_arrive(vempty + vs);
            }
        }
        __syncwarp();
        all_done();
        regs_up<kRegsLaunch>();
    } else {
        // ------------------------------------------ softmax, one row a thread
        regs_up<kRegsMany>();
        const int i = (warp - 8) >> 2, r = tid - 256 - 128 * i, row = 128 * i + r;  // tile, row of it, row of the pair
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tm + lanes + kColS + 128 * i, tO = tm + lanes + kColO + 128 * i;
        const bool live = row < rows;
        // The warp's 32 rows of q, scaled, as hi (e5m2) + lo (e4m3), two rows at a time, 16 lanes a row
        // (a lane a row would touch 32 cache lines with every load). A row's 256 bytes come by
        // asynchronous copies to where its hi and lo will be, so that all are in flight
        // together and the loops stay short (straight-line code for all the rows cost 3 us
        // more: it runs once, as fast as instructions can be fetched). The row's factor goes
        // to the lane that owns the row.
        float cs = 0.f;
        {
            const int rr = row0 + (live ? row : 0), piece = lane & 15, up = lane >> 4;
            const long at = ((long)s * a.T + rr / R) * a.q_stride + (long)(g * R + rr % R) * kKvD;
            uint8_t* q8 = sm + L::kQ + 2 * i * kTlTile + (r & ~31) * kKvD;  // the warp's first row
#pragma unroll 4
            for (int t = 0; t < 16; ++t) {
                const long from = __shfl_sync(0xffffffffu, at, 2 * t + up);
                cp_async16(q8 + (piece >> 3) * kTlTile + (2 * t + up) * kKvD + (piece & 7) * 16,
                           reinterpret_cast<const uint16_t*>(a.q) + from + 8 * piece);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            float mine = 0.f;  // the largest magnitude of the row that this lane owns
#pragma unroll 1
            for (int t4 = 0; t4 < 16; t4 += 4) {  // eight rows side by side
                float f[4][8], top[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint4 x = *reinterpret_cast<const uint4*>(q8 + (piece >> 3) * kTlTile + (2 * (t4 + t) + up) * kKvD +
                                                                    (piece & 7) * 16);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    top[t] = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        f[t][2 * e] = __uint_as_float(w[e] << 16);
                        f[t][2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
                        top[t] = max3(top[t], fabsf(f[t][2 * e]), fabsf(f[t][2 * e + 1]));
                    }
                }
#pragma unroll
                for (int off = 1; off < 16; off <<= 1)
#pragma unroll
                    for (int t = 0; t < 4; ++t) top[t] = fmaxf(top[t], __shfl_xor_sync(0xffffffffu, top[t], off));
#pragma unroll
                for (int t = 0; t < 4; ++t) {  // (the 16 lanes have read their rows: they have exchanged the maxima)
                    const float own = __shfl_sync(0xffffffffu, top[t], (lane & 1) << 4);
                    if ((lane >> 1) == t4 + t) mine = own;
                    const float pw = row_power(top[t], kQPower), sg = a.scale < 0.f ? -pw : pw;
                    uint32_t hi[2] = {0u, 0u}, lo[2] = {0u, 0u};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y0 = f[t][2 * e] * sg, y1 = f[t][2 * e + 1] * sg;
                        const uint32_t h2 = __nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E5M2);
                        const float2 back = unpack_f16x2(e5m2x2_to_f16x2(h2));
                        const uint32_t l2 = __nv_cvt_float2_to_fp8x2(make_float2(y0 - back.x, y1 - back.y), __NV_SATFINITE, __NV_E4M3);
                        hi[e >> 1] |= h2 << (16 * (e & 1));
                        lo[e >> 1] |= l2 << (16 * (e & 1));
                    }
                    const int qr = 2 * (t4 + t) + up;
                    uint8_t* o = q8 + qr * kKvD + (((piece >> 1) ^ (qr & 7)) << 4) + 8 * (piece & 1);
                    *reinterpret_cast<uint2*>(o) = make_uint2(hi[0], hi[1]);
                    *reinterpret_cast<uint2*>(o + kTlTile) = make_uint2(lo[0], lo[1]);
                }
            }
            // a row that holds an infinity reads NaN
            cs = mine < INFINITY ? fabsf(a.scale) * kLog2e / row_power(mine, kQPower) : NAN;
            tc::fence_proxy_async_smem();
        }
        float2 l0 = make_float2(0.f, 0.f), l1 = l0;  // the row's sum, in four parts
        const int lim = !live || !ok ? -1 : a.causal ? before + (row0 + row) / R : before - 1;  // the last position seen
        const int nci = i ? nc1 : nc0;
        // the weights of chunk j from its scores
        auto softmax_chunk = [&](int j) -> bool {
            if (!warp_ok(scfull + j % kScStages, (uint32_t)(j / kScStages) & 1)) return false;
            // the chunk's scales: of the scores (with the softmax factor), and of the values
            float cxs[kTlBlocks], vss[kTlBlocks], lvs[kTlBlocks];
            {
                const float4* sk = reinterpret_cast<const float4*>(scales + j % kScStages * 2 * kTlBlocks);
#pragma unroll
                for (int b = 0; b < kTlBlocks / 4; ++b) {
                    const float4 x = sk[b], y = sk[kTlBlocks / 4 + b];
                    cxs[4 * b] = cs * x.x, cxs[4 * b + 1] = cs * x.y, cxs[4 * b + 2] = cs * x.z, cxs[4 * b + 3] = cs * x.w;
                    vss[4 * b] = y.x, vss[4 * b + 1] = y.y, vss[4 * b + 2] = y.z, vss[4 * b + 3] = y.w;
                }
#pragma unroll
                for (int b = 0; b < kTlBlocks; ++b) {
                    lvs[b] = lg2_approx(vss[b]);
                    cxs[b] = cxs[b] < FLT_MIN ? FLT_MIN : cxs[b];  // not 0: hidden scores are -inf
                }
            }
            if (!warp_ok(sfull + i, (uint32_t)j & 1)) return false;
            tc::tc_fence_after();
            const int see = lim - (cb + j) * kTlTc;  // columns 0 .. see are seen
            const bool cut = __any_sync(0xffffffffu, see < kTlTc - 1);
            float v[kTlTc], tops[kTlBlocks];  // the scores, and each block's largest
#pragma unroll
            for (int b = 0; b < kTlBlocks; ++b) tmem_ld16_max(tS + 16 * b, v + 16 * b, tops[b]);
            tc::tmem_wait_ld();
            if (cut) {  // the factors of a block that the row does not see may be anything
#pragma unroll
                for (int k = 0; k < kTlTc; ++k) v[k] = k <= see ? v[k] : -INFINITY;
#pragma unroll
                for (int b = 0; b < kTlBlocks; ++b) {
                    const float* w = v + 16 * b;
                    tops[b] = max3(max3(max3(w[0], w[1], w[2]), max3(w[3], w[4], w[5]), max3(w[6], w[7], w[8])),
                                   max3(w[9], w[10], w[11]), max3(fmaxf(w[12], w[13]), w[14], w[15]));
                    if (16 * b > see) cxs[b] = 1.f, vss[b] = 0.f, lvs[b] = -INFINITY;
                }
            }
            // the chunk's maxima: of x, and of x + log2 vs
            float mx = -INFINITY, mvx = -INFINITY;
#pragma unroll
            for (int b = 0; b < kTlBlocks; ++b) {
                const float x = tops[b] * cxs[b];
                mx = fmaxf(mx, x);
                mvx = fmaxf(mvx, x + lvs[b]);
            }
            if (mx > m + kSlackM) {
                const float f = ex2_approx(m - mx);
                l0.x *= f, l0.y *= f, l1.x *= f, l1.y *= f;
                m = mx;
            }
            const bool grow = mvx > mv + kSlackV;
            const float f = grow ? ex2_approx(mv - mvx) : 1.f;
            if (grow) mv = mvx;
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
            const float lift = fminf(ex2_approx(m - mv + kLift), FLT_MAX);  // (finite: a block of scale 0 weighs 0)
            const float2 nm = make_float2(-m, -m);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t y[16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int b = 2 * q + h;
                    const float cx = cxs[b], to = vss[b] * lift;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int at = 16 * b + 2 * k;
                        const float2 x = fma2(make_float2(v[at], v[at + 1]), make_float2(cx, cx), nm);
                        const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                        if (k & 1)
                            l1 = add2(l1, p);
                        else
                            l0 = add2(l0, p);
                        const float2 w = mul2(p, make_float2(to, to));
                        y[8 * h + k] = pack_f16x2(w.x, w.y);
                    }
                }
                tmem_st16(tS + 16 * q, y);  // over S, which is read
            }
            tc::tmem_wait_st();
            return true;
        };
        bool good = true;
        tc::tc_fence_before();
        tile_rows_meet(TileBarriers(), i, nci, [&](int j) {
            good = good && softmax_chunk(j);
            tc::tc_fence_before();
        });
        l = (l0.x + l0.y) + (l1.x + l1.y);
        __syncwarp();
        regs_down<kRegsLaunch>();
        all_done();
    }
    // ------------------------------------------------------------- the merge
    __syncwarp();
    const bool walked = warp < 8 || (warp < 12 ? nc0 : nc1) == 0 || warp_ok(ofull + (warp < 12 ? 0 : 1), 0);
    tc::tc_fence_after();
    __syncthreads();
    const bool gave_up = *flag != 0;
    if (gave_up && warp < 2 && tc::elect_one()) {
        // the copies in flight must land and every product issued must be done
        // before the tensor memory is freed and the CTA exits (all bounded)
        if (warp == 0) {
            for (int i = 0; i < kKStages; ++i)
                tc::mbar_wait(kfull + i, 0, 100000000ull), tc::mbar_wait(kfull + i, 1, 100000000ull);
            for (int i = 0; i < kVStages; ++i)
                tc::mbar_wait(vfull + i, 0, 100000000ull), tc::mbar_wait(vfull + i, 1, 100000000ull);
        } else {
            tc::mma_commit(endbar);
            tc::mbar_wait(endbar, 0, 100000000ull);
        }
    }
    __syncthreads();
    if (W > 1) tc::cluster_wait();  // (pairs with the arrival at the start)
    if (warp >= 8) {
        const int i = (warp - 8) >> 2, row = tid - 256;
        const uint32_t tO = tm + ((uint32_t)((warp & 3) * 32) << 16) + kColO + 128 * i;
        const bool some = walked && !gave_up && (i ? nc1 : nc0) > 0;  // (the same in the whole warp)
        const bool live = row < rows;
        if (!some) m = mv = kNone, l = 0.f;
        const int rr = row0 + (live ? row : 0);
        const long at = ((long)s * a.T + rr / R) * a.out_stride + (long)(g * R + rr % R) * kKvD;
        const float f = l == 0.f ? 0.f : ex2_approx(mv - m - kLift) / l;
        uint8_t* own = sm + (row & ~31) * 256;  // W == 1: the warp's rows in bf16
        // (rolled up, here and in the merge: code that runs once goes as fast as it is fetched)
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
            if (W == 1) {
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(v[k + 2 * e] * f, v[k + 2 * e + 1] * f);
                    *reinterpret_cast<uint4*>(own + lane * 256 + (((4 * q + k / 8) ^ (lane & 15)) << 4)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else if (live) {
                // 16-byte pieces rotated by the row, so that a warp's rows do not meet in one bank
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<float4*>(sm + row * kKvD * 4 + (((8 * q + k + row) & 31) << 4)) =
                        make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
            __syncwarp();
        }
        if (W == 1) {
            // two rows at a time, 16 lanes a row: whole lines go out (a lane a row took 6,000
            // cycles a CTA)
#pragma unroll 4
            for (int t = 0; t < 16; ++t) {
                const int r = 2 * t + (lane >> 4), piece = lane & 15;
                const long to = __shfl_sync(0xffffffffu, at, r);
                if ((row & ~31) + r < rows)
                    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + to + 8 * piece) =
                        *reinterpret_cast<const uint4*>(own + r * 256 + ((piece ^ (r & 15)) << 4));
            }
        }
        if (W > 1 && live) *reinterpret_cast<float4*>(sm + L::kMl + row * 16) = make_float4(m, l, mv, 0.f);
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tm, 512);
    if (W == 1) return;
    tc::cluster_arrive();  // every CTA's rows are in its shared memory ...
    tc::cluster_wait();
    // ... and each reads the rows that it owns
    if (W == 2)
        merge_rows<2>(a, sm, wk, rows, row0, s, g);
    else if (W == 4)
        merge_rows<4>(a, sm, wk, rows, row0, s, g);
    else
        merge_rows<8>(a, sm, wk, rows, row0, s, g);
    tc::cluster_arrive();  // nobody leaves while its memory is read
    tc::cluster_wait();
}

// Per device, once: the kernel's attributes, and how many clusters of 1, 2, 4
// and 8 CTAs the device holds at once.
struct TlSetup {
    bool done;
    int held[4];
};

cudaError_t tile_setup(const TlSetup** out) {
    static std::mutex mutex;
    static TlSetup per_device[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mutex);
    TlSetup& u = per_device[dev & 63];
    if (!u.done) {
        // the warps' register split draws on what the launch gives
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, attn_paged_tile_kernel);
        if (e != cudaSuccess) return e;
        if (fa.numRegs < kRegsLaunch) return cudaErrorLaunchOutOfResources;
        e = cudaFuncSetAttribute(attn_paged_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)TlSmem::kBytes);
        if (e != cudaSuccess) return e;
        u.held[0] = 152;
        for (int k = 1; k < 4; ++k) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(1u << k);
            cfg.blockDim = dim3(kTlThreads);
            cfg.dynamicSmemBytes = TlSmem::kBytes;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 1u << k;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int held = 0;
            if (cudaOccupancyMaxActiveClusters(&held, attn_paged_tile_kernel, &cfg) != cudaSuccess) held = 0;
            u.held[k] = held;
        }
        (void)cudaGetLastError();  // a refused query leaves no sticky error
        u.done = true;
    }
    *out = &u;
    return cudaSuccess;
}

}  // namespace

cudaError_t plan_attn_paged_tiles(const PagedAttnArgs& a, PagedAttnPlan* plan) {
    const TlSetup* setup = nullptr;
    const cudaError_t e = tile_setup(&setup);
    if (e != cudaSuccess) return e;
    const long groups = ((long)a.T * (a.Hq / a.c.Hkv) + 2 * kTlRows - 1) / (2 * kTlRows);
    const long pairs = (long)a.c.S * a.c.Hkv * groups, chunks = (a.c.capacity() + kTlTc - 1) / kTlTc;
    // CTAs that share a pair's positions: the least time, in chunks (of 1.45 us),
    // with 5 for a CTA's start and end and 1 for the merge. One session's CTAs
    // are all alike: rounds x a CTA's time. Several sessions are mostly shorter
    // than the table's reach: the longest, and where not all CTAs are held at
    // once, what the others take. (Over 75 calls, whose tables end with their
    // longest session, within 2.2% of the best W on average. Six sessions catching
    // up by at most 75 positions over at most 3,076, 96 pairs: 46 us with one CTA a
    // pair, 30 with two, 39 with four; by 200 over 6,200: 99, 58 and 86; 2 x 300
    // rows across to 1,500 positions: 29, 22 and 37.)
    plan->tiles = true;
    float least = 0.f;
    for (int k = 0, w = 1; k < 4 && (w == 1 || w <= chunks) && setup->held[k] > 0; ++k, w *= 2) {
        const float part = (float)pairs / (float)setup->held[k], walk = (float)((chunks + w - 1) / w);
        const float rounds = a.c.S == 1 ? ceilf(part) : fmaxf(1.f, part), ends = w > 1 ? 6.f : 5.f;
        const float cost = a.c.S == 1 ? rounds * (walk + ends)
                                      : walk + ends + (part > 1.f ? (part - 0.7f) * (0.3f * walk + ends) : 0.f);
        if (w > 1 && cost >= least) continue;
        least = cost;
        plan->W = w;
        plan->us = rounds * ((w > 1 ? 11.f : 8.f) + (a.c.S == 1 ? 1.45f : 1.1f) * walk);
    }
    return cudaSuccess;
}

cudaError_t launch_attn_paged_tiles(const PagedAttnArgs& a, int W, cudaStream_t st) {
    CUtensorMap tmk, tmv;
    cudaError_t e = make_page_map(a.c.kp, a.c, kTlTc, &tmk);
    if (e == cudaSuccess) e = make_page_map(a.c.vp, a.c, kTlTc, &tmv);
    if (e != cudaSuccess) return e;
    const long groups = ((long)a.T * (a.Hq / a.c.Hkv) + 2 * kTlRows - 1) / (2 * kTlRows);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(W * groups * a.c.Hkv), a.c.S);
    cfg.blockDim = dim3(kTlThreads);
    cfg.dynamicSmemBytes = TlSmem::kBytes;
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
    // (where a session alone fills the GPU, the order within it is enough, and
    // ranking costs 1%: 538 us for 532, 4 x 4096 positions. Twenty-four sessions
    // catching up: 52 us for 71, 20 rows of 64 sessions of up to 7,500: 210 for 260.)
    const long session = W * groups * a.c.Hkv;
    const bool ranked = a.c.S > 1 && a.c.S <= kTlThreads && session * a.c.S > 152 && session <= 152;
    return cudaLaunchKernelEx(&cfg, attn_paged_tile_kernel, a, tmk, tmv, W, ranked);
}

}  // namespace m2
