// The C ABI of the paged 8-bit cache (include/mamba2.h): argument, shape and
// alignment checks on the host, then the launchers of m2_paged.h.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mamba2.h"
#include "m2_launch.h"
#include "m2_paged.h"

namespace {

bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// The cache's sizes and T new positions a session.
m2_status check_sizes(const m2_kv_cache* c, int T) {
    if (!c) return M2_EINVAL;
    if (c->n_sessions < 0 || T < 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 || c->page_size <= 0 || c->n_pages <= 0 ||
        c->max_pages <= 0)
        return M2_EINVAL;
    if (c->act != M2_BF16 && c->act != M2_F32) return M2_EINVAL;
    if (c->head_dim != m2::kKvD) return M2_ESHAPE;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return M2_ESHAPE;
    if (c->n_sessions > 65535 || c->n_kv_heads > 65535 || T > (1 << 24)) return M2_ESHAPE;
    // positions are 32-bit numbers, and so are the pool's rows of 128 bytes
    if ((long long)c->max_pages * c->page_size > (1LL << 30)) return M2_ESHAPE;
    if ((long long)c->n_pages * c->n_kv_heads * c->page_size > (1LL << 31) - 256) return M2_ESHAPE;
    return M2_OK;
}

m2_status check_heads(const m2_kv_cache* c, int T, int n_heads) {
    if (n_heads <= 0) return M2_EINVAL;
    if (n_heads % c->n_kv_heads != 0 || (long long)T * n_heads > (1LL << 30)) return M2_ESHAPE;
    return M2_OK;
}

m2_status check_pool(const m2_kv_cache* c) {
    const void* ptrs[] = {c->k_pages, c->v_pages, c->k_scales, c->v_scales};
    if (!c->page_table) return M2_EINVAL;
    for (const void* p : ptrs)
        if (!p) return M2_EINVAL;
    if (!aligned(c->page_table, 4)) return M2_EALIGN;
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return M2_EALIGN;
    return M2_OK;
}

// Rows of `width` activations, `stride` elements apart.
m2_status check_rows(const m2_kv_cache* c, const void* p, long stride, long width) {
    if (!p || stride < width) return M2_EINVAL;
    if (!aligned(p, 16) || (stride * (c->act == M2_BF16 ? 2 : 4)) % 16 != 0) return M2_EALIGN;
    return M2_OK;
}

m2::KvCache cache_of(const m2_kv_cache* c) {
    m2::KvCache k;
    k.S = c->n_sessions;
    k.Hkv = c->n_kv_heads;
    k.ps = c->page_size;
    k.ps_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
    k.n_pages = c->n_pages;
    k.max_pages = c->max_pages;
    k.table = c->page_table;
    k.kp = c->k_pages;
    k.vp = c->v_pages;
    k.ks = c->k_scales;
    k.vs = c->v_scales;
    k.kt = c->k_tail;
    k.vt = c->v_tail;
    k.kto = c->k_tail_out;
    k.vto = c->v_tail_out;
    k.err = nullptr;
    return k;
}

m2_status launched(cudaError_t e) {
    if (e == cudaSuccess) return M2_OK;
    m2::record_cuda_error(e);
    return M2_ECUDA;
}

}  // namespace

extern "C" {

m2_status mamba2_kv_append(const m2_kv_cache* c, int T, const int32_t* lengths, const int32_t* n_new, const void* k,
                           const void* v, long kv_stride, const m2_rope* rope, int n_heads, const void* q, long q_stride,
                           void* q_out, long q_out_stride, void* stream) {
    m2_status st = check_sizes(c, T);
    if (st != M2_OK) return st;
    if (n_heads < 0) return M2_EINVAL;
    if (q || q_out) {
        st = check_heads(c, T, n_heads);
        if (st != M2_OK) return st;
    }
    const bool turns = rope && rope->rot_dim != 0;
    if (turns) {
        if (rope->rot_dim < 0 || rope->n_pos <= 0 || !rope->cos || !rope->sin) return M2_EINVAL;
        if (rope->rot_dim % 16 != 0 || rope->rot_dim > c->head_dim) return M2_ESHAPE;
        if (!aligned(rope->cos, 16) || !aligned(rope->sin, 16)) return M2_EALIGN;
    }
    st = check_pool(c);
    if (st != M2_OK) return st;
    const void* tails[] = {c->k_tail, c->v_tail, c->k_tail_out, c->v_tail_out};
    if (!lengths) return M2_EINVAL;
    for (const void* p : tails)
        if (!p) return M2_EINVAL;
    for (const void* p : tails)
        if (!aligned(p, 16)) return M2_EALIGN;
    if (!aligned(lengths, 4) || !aligned(n_new, 4)) return M2_EALIGN;
    st = check_rows(c, k, kv_stride, (long)c->n_kv_heads * c->head_dim);
    if (st == M2_OK) st = check_rows(c, v, kv_stride, (long)c->n_kv_heads * c->head_dim);
    if (st == M2_OK && (q || q_out)) {
        st = check_rows(c, q, q_stride, (long)n_heads * c->head_dim);
        if (st == M2_OK) st = check_rows(c, q_out, q_out_stride, (long)n_heads * c->head_dim);
        if (st == M2_OK && q == q_out && q_stride != q_out_stride) return M2_EINVAL;
    }
    if (st != M2_OK) return st;
    if (((long long)T / m2::kKvBlock + 2) * c->n_kv_heads > (1LL << 30)) return M2_ESHAPE;
    st = m2::check_device();
    if (st != M2_OK) return st;
    if (c->n_sessions == 0) return M2_OK;
    m2::KvAppendArgs a;
    a.c = cache_of(c);
    a.c.err = m2::device_error_word();
    a.bf16 = c->act == M2_BF16;
    a.T = T;
    a.Hq = q ? n_heads : 0;
    a.lens = lengths;
    a.n_new = n_new;
    a.k = k;
    a.v = v;
    a.q = q;
    a.q_out = q_out;
    a.kv_stride = kv_stride;
    a.q_stride = q_stride;
    a.qo_stride = q_out_stride;
    a.rot = turns ? rope->rot_dim : 0;
    a.interleaved = turns && rope->interleaved;
    a.n_pos = turns ? rope->n_pos : 0;
    a.cos = turns ? rope->cos : nullptr;
    a.sin = turns ? rope->sin : nullptr;
    return launched(m2::launch_kv_append(a, static_cast<cudaStream_t>(stream)));
}

size_t mamba2_attn_paged_workspace_bytes(const m2_kv_cache* c, int T, int n_heads) {
    (void)c, (void)T, (void)n_heads;
    return 0;  // every form merges in shared memory
}

m2_status mamba2_attn_paged(const m2_kv_cache* c, int T, int n_heads, int causal, const int32_t* lengths,
                            const int32_t* n_new, const void* q, long q_stride, float scale, void* out, long out_stride,
                            void* workspace, size_t workspace_bytes, void* stream) {
    m2_status st = check_sizes(c, T);
    if (st == M2_OK) st = check_heads(c, T, n_heads);
    if (st != M2_OK) return st;
    if (!isfinite(scale)) return M2_EINVAL;
    st = check_pool(c);
    if (st != M2_OK) return st;
    if (!lengths) return M2_EINVAL;
    if (!aligned(lengths, 4) || !aligned(n_new, 4)) return M2_EALIGN;
    st = check_rows(c, q, q_stride, (long)n_heads * c->head_dim);
    if (st == M2_OK) st = check_rows(c, out, out_stride, (long)n_heads * c->head_dim);
    if (st == M2_OK && out == q) return M2_EINVAL;
    if (st != M2_OK) return st;
    m2::PagedAttnArgs a;
    a.c = cache_of(c);
    (void)workspace_bytes;  // none is needed
    if (workspace && !aligned(workspace, 16)) return M2_EALIGN;
    st = m2::check_device();
    if (st != M2_OK) return st;
    if (c->n_sessions == 0 || T == 0) return M2_OK;
    a.c.err = m2::device_error_word();
    a.bf16 = c->act == M2_BF16;
    a.causal = causal != 0;
    a.T = T;
    a.Hq = n_heads;
    a.lens = lengths;
    a.n_new = n_new;
    a.q = q;
    a.out = out;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.scale = scale;
    return launched(m2::launch_attn_paged(a, static_cast<cudaStream_t>(stream)));
}

// How mamba2_attn_paged would run a call of these sizes, for the tests that are
// written for one form (not in the public header): the CTAs that share a set of
// rows' positions, + 256 for the form for many rows; the negative status where
// the sizes or the device are refused.
int m2_attn_paged_plan(const m2_kv_cache* c, int T, int n_heads) {
    m2_status st = check_sizes(c, T);
    if (st == M2_OK) st = check_heads(c, T, n_heads);
    if (st == M2_OK) st = m2::check_device();
    if (st != M2_OK) return -(int)st;
    m2::PagedAttnArgs a = {};
    a.c = cache_of(c);
    a.bf16 = c->act == M2_BF16;
    a.T = T;
    a.Hq = n_heads;
    m2::PagedAttnPlan plan;
    st = launched(m2::plan_attn_paged(a, &plan));
    return st == M2_OK ? plan.W + (plan.tiles ? 256 : 0) : -(int)st;
}

}  // extern "C"
