// Appending new keys and values to a paged cache held in e4m3, with the
// position rotation of keys (and queries) applied on the way.
//
// A block of 16 positions of one kv head shares one fp32 scale:
//     m = max(max |block|, 2^-100), scale = m / 448, code = e4m3(448 x / m),
// the quotient rounded once, to nearest even: the one rounding that a cached
// value gets. The positions of the block that is still open are kept in fp32 (the
// tail, rows [0, length mod 16)), so a block is always quantised from its
// exact values by its own maximum, and the cache does not depend on how the
// positions were split over calls: a prefill and single frames leave the same
// bits. The rotation of dims (a, b) of a pair at position t by the table's
// cos and sin, each product and sum rounded to fp32 by itself (no fused
// multiply-add, so that the results are those of the formula as written):
//     a' = a cos_t - b sin_t,  b' = a sin_t + b cos_t.
//
// Memory-bound: per new position and kv head 2 x 128 activations in and
// 2 x 128 bytes of codes out; per query head 128 activations in and out. The
// open block costs up to 15 fp32 rows in and out a call, which is what a
// single frame mostly moves.
//
// One CTA per (block, kv head, session): thread = (row, 8 dims) of the keys
// and of the values, so that every global access is 8 or 16 bytes wide and
// the pair (d, d + rot / 2) of the half layout sits in another lane of the
// same half-warp. The maximum goes through shuffles and shared memory. The
// queries go to CTAs of their own, 16 (position, heads) rows at a time.
// 4 x 4096 positions with 40 query heads, bf16, 446 MB: 95 us, 4.7 TB/s (70%
// of the measured copy rate; 88 us with quotients rounded twice; 34 us of that
// without the queries, where a CTA's chain of length, rows, maximum and stores
// shows: four heads in turn with the next one's rows in flight took 44). One
// frame: 2.6 us, of 64 sessions 4.0 us, mostly the launch and the chain.
#include <cuda_fp8.h>

#include "m2_common.cuh"
#include "m2_paged.h"

namespace m2 {

namespace {

constexpr int kApThreads = 256;  // 16 rows x 16 pieces of 8 dims
constexpr int kPieces = kKvD / 8;

template <typename TA>
__device__ __forceinline__ void load8(const void* base, size_t elem, float (&f)[8]) {
    Act8<TA> x;
    x.load_rw(base, elem);  // a plain load: q may be rotated in place
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = x.get(j);
}

__device__ __forceinline__ void load8_f32(const float* p, float (&f)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ void store8_f32(float* p, const float (&f)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// The rotation of dims [8 piece, 8 piece + 8) at one position: the table's
// factors, and in the half layout the lane with the pairs' other dims.
struct Turn {
    float c[8], s[8];
    int mate;
    bool on, second;  // turned at all; the pairs' second dims (half layout)

    __device__ __forceinline__ void load(const KvAppendArgs& a, int piece, int lane, int pos, bool live) {
        on = live && a.rot > 0 && 8 * piece < a.rot;
        const int half = a.rot >> 1, hp = half >> 3;  // hp: pieces of one half
        second = !a.interleaved && piece >= hp;
        mate = a.interleaved || 8 * piece >= a.rot ? lane : second ? lane - hp : lane + hp;
        if (!on) return;
        if (a.interleaved) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(a.cos + (size_t)pos * half + 4 * piece));
            const float4 y = __ldg(reinterpret_cast<const float4*>(a.sin + (size_t)pos * half + 4 * piece));
            c[0] = x.x, c[1] = x.y, c[2] = x.z, c[3] = x.w;
            s[0] = y.x, s[1] = y.y, s[2] = y.z, s[3] = y.w;
        } else {
            const size_t at = (size_t)pos * half + 8 * (second ? piece - hp : piece);
            load8_f32(a.cos + at, c);
            load8_f32(a.sin + at, s);
        }
    }
    // Every lane of the warp calls it (the half layout exchanges dims).
    __device__ __forceinline__ void apply(const KvAppendArgs& a, float (&f)[8]) const {
        if (a.rot == 0) return;
        if (a.interleaved) {
            if (!on) return;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = f[2 * j], y = f[2 * j + 1];
                f[2 * j] = __fsub_rn(__fmul_rn(x, c[j]), __fmul_rn(y, s[j]));
                f[2 * j + 1] = __fadd_rn(__fmul_rn(x, s[j]), __fmul_rn(y, c[j]));
            }
            return;
        }
        float g[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = __shfl_sync(0xffffffffu, f[j], mate);
        if (!on) return;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float u = __fmul_rn(f[j], c[j]), w = __fmul_rn(g[j], s[j]);
            f[j] = second ? __fadd_rn(w, u) : __fsub_rn(u, w);
        }
    }
};

// y, which is 448 x / m but for two units in its last place at most, is next
// to a value halfway between two codes: that value M, or its neighbour on the
// side of the exact quotient. 448 |x| = p + r exactly (r a fused
// multiply-add's), and p - M m is exact too, the two being so near.
__device__ __forceinline__ float settle(float x, float y, float m) {
    const float down = m > 1e18f ? 0x1p-20f : 1.f;  // (448 |x| stays finite)
    const float a = fabsf(x) * down, mm = m * down, t = fabsf(y) < 0x1p-6f ? fabsf(y) + 0x1p-6f : fabsf(y);
    float M = __uint_as_float(((__float_as_uint(t) + 2u - 0x80000u) & ~0xFFFFFu) + 0x80000u);
    if (fabsf(y) < 0x1p-6f) M -= 0x1p-6f;
    const float p = __fmul_rn(a, 448.f), r = __fmaf_rn(a, 448.f, -p);
    const float over = __fadd_rn(__fmaf_rn(-M, mm, p), r);
    const uint32_t bits = __float_as_uint(M) + (over > 0.f ? 1u : over < 0.f ? ~0u : 0u);
    return copysignf(__uint_as_float(bits), y);
}

// The codes e4m3(448 x / m) of 8 values, to nearest even. x (448 / m) in fp32
// is off by less than two units in its last place, which matters only next to
// a value halfway between two codes: there the exact quotient decides (bf16
// values meet such ties in one block of seven or so, where m is a multiple of
// 7; fp32 values almost never).
__device__ __forceinline__ uint2 pack_e4m3(const float (&x)[8], float m) {
    const float inv = __fdiv_rn(kE4m3Max, m);
    // e4m3 keeps three bits behind the first, so that next to halfway the other
    // 20 are next to 0x80000; below 2^-6 its step is that of [2^-6, 2^-5)
    auto off = [](float v) { return (__float_as_uint(v) + 2u - 0x80000u) & 0xFFFFFu; };
    float y[8], least = 1.f;
    uint32_t nearest = ~0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[j] = __fmul_rn(x[j], inv);
        nearest = min(nearest, off(y[j]));
        least = fminf(least, fabsf(y[j]));
    }
    if ((nearest <= 4u || least < 0x1p-6f) && m < INFINITY) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = fabsf(y[j]);
            if (off(a < 0x1p-6f ? a + 0x1p-6f : a) <= 4u) y[j] = settle(x[j], y[j], m);
        }
    }
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        h[j] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * j], y[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// grid (blocks of a session x kv heads + CTAs of its queries, sessions)
// QH: heads of the queries that a thread rotates. (bf16: five CTAs an SM, 48
// registers, 95 us above against 98 with four.)
template <typename TA, int QH>
__global__ void __launch_bounds__(kApThreads, sizeof(TA) == 2 ? 5 : 4) kv_append_kernel(KvAppendArgs a, int blocks) {
    __shared__ uint32_t smax[2][kApThreads / 32];
    const KvCache& c = a.c;
    const int s = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = tid / kPieces, piece = tid % kPieces;

    pdl_wait();  // the rows and the cache may come from the previous kernel
    pdl_trigger();
    int L, n;
    const long limit = a.rot ? min(c.capacity(), (long)a.n_pos) : c.capacity();
    if (!kv_extent(c, s, a.T, a.lens, a.n_new, limit, &L, &n)) {  // the whole session is refused
        if (blockIdx.x == 0 && tid == 0) record_error(c.err, ERR_ATTN_LENGTH);
        if ((int)blockIdx.x < c.Hkv) {  // ... and keeps its tail, whichever rows of it are open
            const size_t at = (((size_t)s * c.Hkv + blockIdx.x) * kKvBlock + row) * kKvD + 8 * piece;
            float f[8];
            if (c.kto != c.kt) load8_f32(c.kt + at, f), store8_f32(c.kto + at, f);
            if (c.vto != c.vt) load8_f32(c.vt + at, f), store8_f32(c.vto + at, f);
        }
        return;
    }
    if ((int)blockIdx.x >= blocks * c.Hkv) {
        // the queries: 16 (position, QH heads) rows; the factors are read once for the heads
        const int r = ((int)blockIdx.x - blocks * c.Hkv) * (kApThreads / kPieces) + row, parts = (a.Hq + QH - 1) / QH;
        const int t = r / parts, h0 = r % parts * QH;
        const bool live = t < n;
        Turn turn;
        turn.load(a, piece, lane, L + t, live);
        const size_t in = ((size_t)s * a.T + t) * a.q_stride + 8 * piece, to = ((size_t)s * a.T + t) * a.qo_stride + 8 * piece;
        Act8<TA> x[QH];
#pragma unroll
        for (int h = 0; h < QH; ++h)
            if (live && h0 + h < a.Hq) x[h].load_rw(a.q, in + (size_t)(h0 + h) * kKvD);
#pragma unroll
        for (int h = 0; h < QH; ++h) {
            float f[8] = {};
            const bool here = live && h0 + h < a.Hq;
            if (here) {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = x[h].get(j);
            }
            turn.apply(a, f);
            if (here) {
                const size_t o = to + (size_t)(h0 + h) * kKvD;
                if constexpr (sizeof(TA) == 2) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = (uint32_t)float_to_bf16_bits(f[2 * j]) | ((uint32_t)float_to_bf16_bits(f[2 * j + 1]) << 16);
                    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.q_out) + o) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    store8_f32(reinterpret_cast<float*>(a.q_out) + o, f);
                }
            }
        }
        return;
    }
    const int b = (int)blockIdx.x / c.Hkv, g = (int)blockIdx.x % c.Hkv;
    const int end = L + n;
    const int base = (L & ~(kKvBlock - 1)) + b * kKvBlock;
    const size_t tail = (((size_t)s * c.Hkv + g) * kKvBlock + row) * kKvD + 8 * piece;
    if (base >= end && b > 0) return;

    // position `pos` of the session, one of the new ones, in fp32 and rotated
    auto fresh = [&](int pos, bool live, float (&k)[8], float (&v)[8]) {
        if (live) {
            const size_t e = ((size_t)s * a.T + (pos - L)) * a.kv_stride + (size_t)g * kKvD + 8 * piece;
            load8<TA>(a.k, e, k);
            load8<TA>(a.v, e, v);
        }
        Turn turn;
        turn.load(a, piece, lane, pos, live);
        turn.apply(a, k);
    };
    // (n == 0 writes no block, and base may lie behind the table)
    const int page = n > 0 ? c.table[(size_t)s * c.max_pages + (base >> c.ps_shift)] : -1;
    const int pos = base + row;
    const bool old = pos < L, live = pos < end;
    float k[8] = {}, v[8] = {};
    if (old) {
        load8_f32(c.kt + tail, k);
        load8_f32(c.vt + tail, v);
    }
    fresh(pos, live && !old, k, v);  // (a row of the tail stays as it is)
    // the block's maxima, as the bits of |x|: their order is that of the
    // numbers, and a NaN is above them all
    uint32_t mk = 0, mv = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        mk = max(mk, __float_as_uint(k[j]) & 0x7FFFFFFFu);
        mv = max(mv, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    }
    mk = __reduce_max_sync(0xffffffffu, mk);
    mv = __reduce_max_sync(0xffffffffu, mv);
    if (lane == 0) {
        smax[0][warp] = mk;
        smax[1][warp] = mv;
    }
    __syncthreads();  // ... and every row of the tail has been read
#pragma unroll
    for (int w = 0; w < kApThreads / 32; ++w) {
        mk = max(mk, smax[0][w]);
        mv = max(mv, smax[1][w]);
    }
    mk = max(mk, __float_as_uint(kKvTiny));
    mv = max(mv, __float_as_uint(kKvTiny));
    if (n > 0) {
        if (page < 0 || page >= c.n_pages) {
            if (tid == 0) record_error(c.err, ERR_KV_PAGE);
        } else {
            const size_t at = ((size_t)page * c.Hkv + g) * c.ps + (base & (c.ps - 1));  // row of the block's first position
            if (live) {
                const size_t o = (at + row) * kKvD + 8 * piece;
                *reinterpret_cast<uint2*>(c.kp + o) = pack_e4m3(k, __uint_as_float(mk));
                *reinterpret_cast<uint2*>(c.vp + o) = pack_e4m3(v, __uint_as_float(mv));
            }
            if (tid == 0) {
                c.ks[at / kKvBlock] = __fdiv_rn(__uint_as_float(mk), kE4m3Max);
                c.vs[at / kKvBlock] = __fdiv_rn(__uint_as_float(mv), kE4m3Max);
            }
        }
    }
    // the tail of the block that is open afterwards, written by the CTA that
    // reads the one open before (in place, nobody else may overwrite it)
    if (b == 0) {
        const int last = end & ~(kKvBlock - 1);
        const bool stays = row < (end & (kKvBlock - 1));
        if (last != base) fresh(last + row, stays, k, v);
        if (stays) {
            store8_f32(c.kto + tail, k);
            store8_f32(c.vto + tail, v);
        }
    }
}

// QH: heads of the queries that a thread rotates.
template <typename TA, int QH>
cudaError_t launch_append(const KvAppendArgs& a, long blocks, cudaStream_t st) {
    const long rows = (long)a.T * ((a.Hq + QH - 1) / QH);
    const long qctas = (rows + kApThreads / kPieces - 1) / (kApThreads / kPieces);
    const dim3 grid((unsigned)(blocks * a.c.Hkv + qctas), (unsigned)a.c.S);
    return launch_pdl(kv_append_kernel<TA, QH>, grid, dim3(kApThreads), 0, st, a, (int)blocks);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t st) {
    const long blocks = ((long)kKvBlock - 1 + a.T + kKvBlock - 1) / kKvBlock;  // the most a session touches
    // One head a thread spreads few queries over the GPU; from two CTAs an SM
    // on, several heads a thread read the factors once and have their loads in
    // flight together (before the quotients' exact rounding, 16,384 positions
    // x 40 heads in bf16: 157 us with one, 97 with two, 88 with four, 98 with
    // eight; 1,505 x 40 in fp32, whose loads are twice as wide: 13.5 with one,
    // 11.4 with two, 11.8 with four).
    const bool many = (long)a.c.S * a.T * a.Hq / 4 >= (long)2 * 152 * (kApThreads / kPieces);
    if (a.bf16) return many ? launch_append<bf16_t, 4>(a, blocks, st) : launch_append<bf16_t, 1>(a, blocks, st);
    return many ? launch_append<float, 2>(a, blocks, st) : launch_append<float, 1>(a, blocks, st);
}

}  // namespace m2
