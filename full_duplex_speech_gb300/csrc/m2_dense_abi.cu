// The C ABI of the bounded dense caches (include/mamba2.h): argument, shape
// and alignment checks on the host, then the launchers of m2_dense.h and
// m2_launch.h.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mamba2.h"
#include "m2_dense.h"
#include "m2_launch.h"

namespace {

bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
size_t up(size_t b) { return (b + 255) / 256 * 256; }

bool overlap(const void* p, size_t np, const void* q, size_t nq) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + nq && b < a + np;
}

m2_status launched(cudaError_t e) {
    if (e == cudaSuccess) return M2_OK;
    m2::record_cuda_error(e);
    return M2_ECUDA;
}

// The caches' sizes (n_heads 1 x n_kv_heads where a call has no queries).
m2_status check_sizes(int S, int Hq, int Hkv, int D, int max_len, m2_dtype act) {
    if (S < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || max_len <= 0) return M2_EINVAL;
    if (act != M2_BF16 && act != M2_F32) return M2_EINVAL;
    if (D != m2::kAttnD || Hq % Hkv != 0 || Hq / Hkv > m2::kAttnMaxR) return M2_ESHAPE;
    if (S > 65535 || Hkv > 65535 || max_len > (1 << 30)) return M2_ESHAPE;  // (positions are 32-bit numbers)
    return M2_OK;
}

size_t cache_rows(int S, int Hkv, int max_len) { return (size_t)S * Hkv * max_len; }

m2_status check_rows(const void* p, long stride, long width, m2_dtype act) {
    const long size = act == M2_BF16 ? 2 : 4;
    if (!p || stride < width) return M2_EINVAL;
    if (stride >= (1L << 40) / size) return M2_ESHAPE;  // (the limit of a tensor map)
    if (!aligned(p, 16) || stride * size % 16 != 0) return M2_EALIGN;
    return M2_OK;
}

// What both calls on packed rows check.
m2_status check_packed(int S, int rows, int Hq, int Hkv, int D, int max_len, m2_dtype act, const int32_t* row_start,
                       const int32_t* lengths, const void* q, long q_stride, float scale) {
    m2_status st = check_sizes(S, Hq, Hkv, D, max_len, act);
    if (st != M2_OK) return st;
    if (rows < 0 || !isfinite(scale)) return M2_EINVAL;
    if ((long long)rows * Hkv > (1LL << 30)) return M2_ESHAPE;  // blocks of one row of every kv head, in a grid
    if (!row_start) return M2_EINVAL;
    if (!aligned(row_start, 4) || !aligned(lengths, 4)) return M2_EALIGN;
    return check_rows(q, q_stride, (long)Hq * D, act);
}

m2::PromptArgs packed(int S, int rows, int Hq, int Hkv, int max_len, m2_dtype act, const int32_t* row_start,
                      const int32_t* lengths, const void* q, long q_stride, float scale) {
    m2::PromptArgs a = {};
    a.S = S;
    a.rows = rows;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.Tmax = max_len;
    a.bf16 = act == M2_BF16;
    a.start = row_start;
    a.lens = lengths;
    a.q = q;
    a.q_stride = q_stride;
    a.scale = scale;
    a.err = m2::device_error_word();
    return a;
}

}  // namespace

extern "C" {

m2_status mamba2_attn_prompt(int n_sessions, int n_rows, int n_heads, int n_kv_heads, int head_dim, int max_len,
                             m2_dtype act, const int32_t* row_start, const int32_t* lengths, const void* q, long q_stride,
                             const void* k_new, const void* v_new, long kv_stride, void* k_cache, void* v_cache,
                             float scale, void* out, long out_stride, float* lse, void* stream) {
    m2_status st = check_packed(n_sessions, n_rows, n_heads, n_kv_heads, head_dim, max_len, act, row_start, lengths, q,
                                q_stride, scale);
    if (st == M2_OK) st = check_rows(k_new, kv_stride, (long)n_kv_heads * head_dim, act);
    if (st == M2_OK) st = check_rows(v_new, kv_stride, (long)n_kv_heads * head_dim, act);
    if (st == M2_OK) st = check_rows(out, out_stride, (long)n_heads * head_dim, act);
    if (st != M2_OK) return st;
    if (!k_cache || !v_cache || out == q || out == k_new || out == v_new || k_cache == v_cache) return M2_EINVAL;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(lse, 4)) return M2_EALIGN;
    st = m2::check_device();
    if (st != M2_OK) return st;
    if (n_sessions == 0) return M2_OK;
    m2::PromptArgs a = packed(n_sessions, n_rows, n_heads, n_kv_heads, max_len, act, row_start, lengths, q, q_stride, scale);
    a.k_new = k_new;
    a.v_new = v_new;
    a.kv_stride = kv_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.out = out;
    a.out_stride = out_stride;
    a.lse = lse;
    return launched(m2::launch_attn_prompt(a, static_cast<cudaStream_t>(stream)));
}

m2_status mamba2_attn_prompt_weights(int n_sessions, int n_rows, int n_heads, int n_kv_heads, int head_dim, int max_len,
                                     m2_dtype act, const int32_t* row_start, const int32_t* lengths, const void* q,
                                     long q_stride, const void* k_cache, float scale, const float* lse, int window,
                                     const float* acc, float* acc_out, void* stream) {
    m2_status st = check_packed(n_sessions, n_rows, n_heads, n_kv_heads, head_dim, max_len, act, row_start, lengths, q,
                                q_stride, scale);
    if (st != M2_OK) return st;
    if (!k_cache || !lse || !acc || !acc_out || window < 0) return M2_EINVAL;
    if (!aligned(k_cache, 16) || !aligned(lse, 4) || !aligned(acc, 16) || !aligned(acc_out, 16)) return M2_EALIGN;
    const size_t bytes = cache_rows(n_sessions, n_kv_heads, max_len) * 4;
    if (acc != acc_out && overlap(acc, bytes, acc_out, bytes)) return M2_EINVAL;
    st = m2::check_device();
    if (st != M2_OK) return st;
    if (n_sessions == 0) return M2_OK;
    m2::PromptArgs a = packed(n_sessions, n_rows, n_heads, n_kv_heads, max_len, act, row_start, lengths, q, q_stride, scale);
    a.k_cache = const_cast<void*>(k_cache);
    a.lse = const_cast<float*>(lse);
    m2::PromptSums w;
    w.window = window;
    w.acc = acc;
    w.acc_out = acc_out;
    return launched(m2::launch_attn_prompt_weights(a, w, static_cast<cudaStream_t>(stream)));
}

size_t mamba2_attn_decode_weights_workspace_bytes(int n_sessions, int n_heads, int n_kv_heads, int head_dim, int max_len,
                                                  m2_dtype act) {
    if (check_sizes(n_sessions, n_heads, n_kv_heads, head_dim, max_len, act) != M2_OK || n_sessions == 0) return 0;
    return up(m2::attn_workspace_bytes(n_sessions, n_heads, n_kv_heads, max_len, act == M2_BF16)) +
           m2::attn_sums_workspace_bytes(n_sessions, n_heads, n_kv_heads, max_len);
}

m2_status mamba2_attn_decode_weights(int n_sessions, int n_heads, int n_kv_heads, int head_dim, int max_len, m2_dtype act,
                                     const int32_t* lengths, const void* q, const void* k_new, const void* v_new,
                                     void* k_cache, void* v_cache, float scale, void* out, const float* acc,
                                     float* acc_out, void* workspace, size_t workspace_bytes, void* stream) {
    m2_status st = check_sizes(n_sessions, n_heads, n_kv_heads, head_dim, max_len, act);
    if (st != M2_OK) return st;
    if (!isfinite(scale) || !lengths) return M2_EINVAL;
    const void* ptrs[] = {q, k_new, v_new, k_cache, v_cache, out, acc, acc_out};
    for (const void* p : ptrs)
        if (!p) return M2_EINVAL;
    if (!aligned(lengths, 4)) return M2_EALIGN;
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return M2_EALIGN;
    const size_t bytes = cache_rows(n_sessions, n_kv_heads, max_len) * 4;
    if (acc != acc_out && overlap(acc, bytes, acc_out, bytes)) return M2_EINVAL;
    const size_t need =
        mamba2_attn_decode_weights_workspace_bytes(n_sessions, n_heads, n_kv_heads, head_dim, max_len, act);
    if (need && (!workspace || workspace_bytes < need)) return M2_EWORKSPACE;
    if (!aligned(workspace, 16)) return M2_EALIGN;
    st = m2::check_device();
    if (st != M2_OK) return st;
    if (n_sessions == 0) return M2_OK;
    m2::AttnArgs a;
    a.S = n_sessions;
    a.Hq = n_heads;
    a.Hkv = n_kv_heads;
    a.Tmax = max_len;
    a.bf16 = act == M2_BF16;
    a.lens = lengths;
    a.q = q;
    a.k_new = k_new;
    a.v_new = v_new;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.scale = scale;
    a.out = out;
    a.ws = static_cast<float*>(workspace);
    a.err = m2::device_error_word();
    a.q_ss = (long)n_heads * head_dim;
    a.kv_ss = (long)n_kv_heads * head_dim;
    a.out_ss = (long)n_heads * head_dim;
    a.len_add = 0;
    a.acc = acc;
    a.acc_out = acc_out;
    a.kept = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                      up(m2::attn_workspace_bytes(n_sessions, n_heads, n_kv_heads, max_len, a.bf16)));
    return launched(m2::launch_attn_decode(a, static_cast<cudaStream_t>(stream)));
}

m2_status mamba2_kv_evict(int n_sessions, int n_kv_heads, int head_dim, int max_len, m2_dtype act, const int32_t* lengths,
                          const void* k_cache, const void* v_cache, const float* acc, int keep, int recent,
                          int out_max_len, void* k_out, void* v_out, float* acc_out, int32_t* kept, void* stream) {
    m2_status st = check_sizes(n_sessions, n_kv_heads, n_kv_heads, head_dim, max_len, act);
    if (st != M2_OK) return st;
    if (keep <= 0 || recent < 0 || recent > keep || out_max_len <= 0 || !lengths) return M2_EINVAL;
    if (keep > out_max_len || out_max_len > (1 << 30)) return M2_ESHAPE;
    const void* ptrs[] = {k_cache, v_cache, acc, k_out, v_out, acc_out};
    for (const void* p : ptrs)
        if (!p) return M2_EINVAL;
    if (!aligned(lengths, 4) || !aligned(kept, 4)) return M2_EALIGN;
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return M2_EALIGN;
    // each array moves in place or to memory of its own
    const size_t row = (size_t)head_dim * (act == M2_BF16 ? 2 : 4);
    const size_t in = cache_rows(n_sessions, n_kv_heads, max_len), out = cache_rows(n_sessions, n_kv_heads, out_max_len);
    const bool in_place = k_out == k_cache;
    if (in_place != (v_out == v_cache)) return M2_EINVAL;
    if ((in_place || acc_out == acc) && out_max_len != max_len) return M2_EINVAL;
    const struct {
        const void* p;
        size_t bytes;
        const void* place;  // the input it may be
    } outs[] = {{k_out, out * row, k_cache},
                {v_out, out * row, v_cache},
                {acc_out, out * 4, acc},
                {kept, kept ? cache_rows(n_sessions, n_kv_heads, keep) * 4 : 0, nullptr}};
    const struct {
        const void* p;
        size_t bytes;
    } ins[] = {{k_cache, in * row}, {v_cache, in * row}, {acc, in * 4}, {lengths, (size_t)n_sessions * 4}};
    for (int i = 0; i < 4; ++i) {
        for (const auto& x : ins)
            if (!(outs[i].p == x.p && x.p == outs[i].place) && overlap(outs[i].p, outs[i].bytes, x.p, x.bytes)) return M2_EINVAL;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return M2_EINVAL;
    }
    st = m2::check_device();
    if (st != M2_OK) return st;
    if (n_sessions == 0) return M2_OK;
    m2::EvictArgs a;
    a.S = n_sessions;
    a.Hkv = n_kv_heads;
    a.Tmax = max_len;
    a.out_max = out_max_len;
    a.row_bytes = (int)row;
    a.lens = lengths;
    a.k = k_cache;
    a.v = v_cache;
    a.acc = acc;
    a.keep = keep;
    a.recent = recent;
    a.k_out = k_out;
    a.v_out = v_out;
    a.acc_out = acc_out;
    a.kept = kept;
    a.err = m2::device_error_word();
    return launched(m2::launch_kv_evict(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
