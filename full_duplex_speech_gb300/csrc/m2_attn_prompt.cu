// Attention of packed whole prompts over the dense caches: the rows of several
// sessions, of different lengths, one behind the other, appended to their
// caches and each attending over its session's positions up to its own.
//     a_p = scale q_t,h . k_p  (p <= before + t),  out_t,h = sum_p softmax(a)_p v_p,
//     lse_t,h = ln sum_p e^(a_p)
// with kv head g = h / R, R = Hq / Hkv. A kv head's rows are its (row, head)
// pairs, t R + r.
#include <math.h>

#include "m2_dense_dev.cuh"

namespace m2 {

namespace {

// ---------------------------------------------------------------- the append
// A warp a row: its keys and values, 16 bytes a lane at a time, to position
// before + t of its session's caches. The session by a 32-way search.
constexpr int kApThreads = 256;
__global__ void __launch_bounds__(kApThreads) prompt_append_kernel(PromptArgs a, int row_bytes) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int row = (int)((blockIdx.x * (long)kApThreads + threadIdx.x) >> 5);
    if (row >= a.rows) return;
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
    // the last session whose first row is at or before this one
    int lo = 0, size = a.S;
    while (size > 1) {
        const int step = (size + 31) >> 5, at = lo + lane * step;
        const int n = __popc(__ballot_sync(0xffffffffu, at < lo + size && a.start[min(at, a.S)] <= row));
        if (n == 0) return;  // rows ahead of the first session's
        lo += (n - 1) * step;
        size = min(step, size - (n - 1) * step);
    }
    Session x;
    if (!session_of(a, lo, &x) || !x.ok || row < x.row0 || row >= x.row0 + x.n) return;
    const size_t to = ((size_t)lo * a.Hkv * a.Tmax + x.before + (row - x.row0)) * row_bytes;
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

cudaError_t launch_append(const PromptArgs& a, cudaStream_t st) {
    const unsigned blocks = (unsigned)(((long)a.rows * 32 + kApThreads - 1) / kApThreads);
    return launch_pdl(prompt_append_kernel, dim3(blocks), dim3(kApThreads), 0, st, a, kAttnD * (a.bf16 ? 2 : 4));
}

// ------------------------------------------------- fp32 products of fp32 units
// A CTA takes up to 64 rows of one (session, kv head), whole packed rows of R
// heads, and walks the positions 64 at a time, with an online softmax.
constexpr int kPfThreads = 256, kPfRows = 64, kPfPos = 64;
constexpr int kPfPitch = kAttnD + 4;  // floats: a column of 16-byte pieces meets all banks
struct PfSmem {
    static constexpr int kQ = 0, kK = kQ + kPfRows * kPfPitch, kV = kK + kPfPos * kPfPitch, kP = kV + kPfPos * kAttnD,
                         kBad = kP + kPfRows * (kPfPos + 4), kFind = kBad + 4, kFloats = kFind + kPfThreads / 32 + 4;
};

template <typename TA> __device__ __forceinline__ float4 load4(const void* p, size_t elem) {
    if constexpr (sizeof(TA) == 2) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + elem);
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                           __uint_as_float(w.y & 0xFFFF0000u));
    } else {
        return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + elem);
    }
}

template <typename TA>
__global__ void __launch_bounds__(kPfThreads) prompt_fp32_kernel(PromptArgs a) {
    extern __shared__ __align__(16) float pf[];
    float *sQ = pf + PfSmem::kQ, *sK = pf + PfSmem::kK, *sV = pf + PfSmem::kV, *sP = pf + PfSmem::kP;
    unsigned* sBad = reinterpret_cast<unsigned*>(pf + PfSmem::kBad);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int R = a.Hq / a.Hkv, per = kPfRows / R;
    const int g = blockIdx.x % a.Hkv;
    pdl_wait();
    pdl_trigger();
    int s, tile;
    if (!find_tile(a, per, blockIdx.x / a.Hkv, reinterpret_cast<int*>(pf + PfSmem::kFind), &s, &tile)) return;
    Session x;
    session_of(a, s, &x);
    const int t0 = tile * per, rows = min(per, x.n - t0) * R;
    if (!x.ok) {
        if (tid == 0) record_error(a.err, ERR_ATTN_LENGTH);
        for (int i = tid; i < rows * kAttnD; i += kPfThreads) {
            const int row = i / kAttnD;
            store_act<TA>(a.out, (size_t)(x.row0 + t0 + row / R) * a.out_stride + (size_t)(g * R + row % R) * kAttnD + i % kAttnD, 0.f);
        }
        if (a.lse)
            for (int row = tid; row < rows; row += kPfThreads)
                a.lse[(size_t)(x.row0 + t0 + row / R) * a.Hq + g * R + row % R] = -INFINITY;
        return;
    }
    for (int i = tid; i < kPfRows * kAttnD / 4; i += kPfThreads) {
        const int row = i / (kAttnD / 4), d = i % (kAttnD / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < rows)
            v = load4<TA>(a.q, (size_t)(x.row0 + t0 + row / R) * a.q_stride + (size_t)(g * R + row % R) * kAttnD + d);
        *reinterpret_cast<float4*>(sQ + row * kPfPitch + d) = v;
    }
    const size_t cache0 = ((size_t)s * a.Hkv + g) * a.Tmax * kAttnD;
    const float sl2 = a.scale * kLog2e;
    int lim[4];  // the last position that this thread's rows see
    float m[4], l[4], o[4][8];
    bool bad[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 4 * ty + i;
        lim[i] = row < rows ? x.before + t0 + row / R : -1;
        m[i] = -FLT_MAX, l[i] = 0.f, bad[i] = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[i][e] = 0.f;
    }
    const int all = x.before + t0 + 1;         // positions that every row sees
    const int total = x.before + t0 + rows / R;  // ... and that the last one does
    for (int p0 = 0; p0 < total; p0 += kPfPos) {
        const bool cut = p0 + kPfPos > all;
        __syncthreads();  // the tiles of the positions before are read
        if (tid < 2) sBad[tid] = 0u;
        if (cut) __syncthreads();
        for (int i = tid; i < kPfPos * kAttnD / 4; i += kPfThreads) {
            const int p = i / (kAttnD / 4), d = i % (kAttnD / 4) * 4;
            float4 k = make_float4(0.f, 0.f, 0.f, 0.f), v = k;
            if (p0 + p < total) {
                k = load4<TA>(a.k_cache, cache0 + (size_t)(p0 + p) * kAttnD + d);
                v = load4<TA>(a.v_cache, cache0 + (size_t)(p0 + p) * kAttnD + d);
                // a value that is not finite must not reach the rows that do not see it: it counts as 0
                // here, and the rows that see it read NaN
                if (cut && !(fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY && fabsf(v.z) < INFINITY && fabsf(v.w) < INFINITY)) {
                    atomicOr(sBad + (p >> 5), 1u << (p & 31));
                    v = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            *reinterpret_cast<float4*>(sK + p * kPfPitch + d) = k;
            *reinterpret_cast<float4*>(sV + p * kAttnD + d) = v;
        }
        __syncthreads();
        float w[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i][j] = 0.f;
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
                    w[i][j] = fmaf(qv[i].x, kv[j].x, w[i][j]);
                    w[i][j] = fmaf(qv[i].y, kv[j].y, w[i][j]);
                    w[i][j] = fmaf(qv[i].z, kv[j].z, w[i][j]);
                    w[i][j] = fmaf(qv[i].w, kv[j].w, w[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int see = lim[i] - p0;
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[i][j] = tx + 16 * j <= see ? w[i][j] * sl2 : -INFINITY;
                top = fmaxf(top, w[i][j]);
            }
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float now = fmaxf(m[i], top), f = ex2_approx(m[i] - now);
            m[i] = now;
            l[i] *= f;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[i][e] *= f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = ex2_approx(w[i][j] - now);
                l[i] += p;
                sP[(4 * ty + i) * (kPfPos + 4) + tx + 16 * j] = p;
            }
            if (cut && see >= 0) {
                const unsigned lo = sBad[0], hi = sBad[1];
                bad[i] |= (lo & (see >= 31 ? ~0u : (2u << see) - 1u)) != 0u ||
                          (see >= 32 && (hi & (see >= 63 ? ~0u : (2u << (see - 32)) - 1u)) != 0u);
            }
        }
        __syncthreads();
#pragma unroll 2
        for (int p = 0; p < kPfPos; p += 4) {
            float4 pr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) pr[i] = *reinterpret_cast<const float4*>(sP + (4 * ty + i) * (kPfPos + 4) + p);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 va = *reinterpret_cast<const float4*>(sV + (p + q) * kAttnD + 4 * tx);
                const float4 vb = *reinterpret_cast<const float4*>(sV + (p + q) * kAttnD + 64 + 4 * tx);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float c = (&pr[i].x)[q];
                    o[i][0] = fmaf(c, va.x, o[i][0]), o[i][1] = fmaf(c, va.y, o[i][1]);
                    o[i][2] = fmaf(c, va.z, o[i][2]), o[i][3] = fmaf(c, va.w, o[i][3]);
                    o[i][4] = fmaf(c, vb.x, o[i][4]), o[i][5] = fmaf(c, vb.y, o[i][5]);
                    o[i][6] = fmaf(c, vb.z, o[i][6]), o[i][7] = fmaf(c, vb.w, o[i][7]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
        const int row = 4 * ty + i;
        if (row >= rows) continue;
        const size_t packed = x.row0 + t0 + row / R;
        const size_t at = packed * a.out_stride + (size_t)(g * R + row % R) * kAttnD;
        const float inv = bad[i] ? NAN : 1.f / l[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            store_act<TA>(a.out, at + 4 * tx + e, o[i][e] * inv);
            store_act<TA>(a.out, at + 64 + 4 * tx + e, o[i][4 + e] * inv);
        }
        if (a.lse && tx == 0) a.lse[packed * a.Hq + g * R + row % R] = m[i] * kLn2 + logf(l[i]);
    }
}

template <typename TA>
cudaError_t launch_fp32(const PromptArgs& a, cudaStream_t st) {
    constexpr int bytes = PfSmem::kFloats * 4;
    cudaError_t e = cudaFuncSetAttribute(prompt_fp32_kernel<TA>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const long tiles = most_tiles(a.S, a.rows, kPfRows / (a.Hq / a.Hkv));
    return launch_pdl(prompt_fp32_kernel<TA>, dim3((unsigned)(tiles * a.Hkv)), dim3(kPfThreads), bytes, st, a);
}

}  // namespace

cudaError_t launch_attn_prompt(const PromptArgs& a, cudaStream_t st) {
    cudaError_t e = launch_append(a, st);
    if (e != cudaSuccess) return e;
    return a.bf16 ? launch_attn_prompt_tiles(a, st) : launch_fp32<float>(a, st);
}

}  // namespace m2
