// attn_api.cu -- the C entries of include/spec_attn.h: argument checks and
// dispatch to the cache kernels (kvcache.cu) and the attention (attn.cu).

#include "attn.cuh"

#define SPEC_EXPORT extern "C" __attribute__((visibility("default")))

namespace specv {
namespace {

constexpr size_t kErrBytes = 256;  // the workspace's error word, padded

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The cache descriptor's own checks; fills the kernels' view of it.
int view_of(const spec_kv_cache *cache, CacheView *c) {
    if (!cache) return SPEC_ERR_NULL;
    if (cache->dtype != SPEC_BF16 && cache->dtype != SPEC_E4M3) return SPEC_ERR_DTYPE;
    if (cache->num_pages < 1 || cache->Hkv < 1 || cache->Hkv > 1024 ||
        (cache->D != 64 && cache->D != 128) ||
        (cache->page != 16 && cache->page != 32 && cache->page != 64 && cache->page != 128) ||
        static_cast<long long>(cache->num_pages) * cache->Hkv > INT_MAX)
        return SPEC_ERR_SHAPE;
    const bool e4m3 = cache->dtype == SPEC_E4M3;
    if (!cache->k || !cache->v || (e4m3 && (!cache->k_exp || !cache->v_exp))) return SPEC_ERR_NULL;
    if (!aligned(cache->k, 16) || !aligned(cache->v, 16) ||
        (e4m3 && (!aligned(cache->k_exp, 4) || !aligned(cache->v_exp, 4))))
        return SPEC_ERR_ALIGN;
    c->k = static_cast<uint8_t *>(cache->k);
    c->v = static_cast<uint8_t *>(cache->v);
    c->k_exp = cache->k_exp;
    c->v_exp = cache->v_exp;
    c->num_pages = cache->num_pages;
    c->Hkv = cache->Hkv;
    c->page_shift = 31 - __builtin_clz(static_cast<unsigned>(cache->page));
    c->D = cache->D;
    c->e4m3 = e4m3;
    return SPEC_OK;
}

// A token stride: 0 stands for `packed`, else at least that and whole
// 16-byte groups of bf16.
bool stride_ok(int64_t *stride, long long packed) {
    if (*stride == 0) *stride = packed;
    return *stride >= packed && *stride % 8 == 0 && *stride <= (1LL << 40);
}

bool attn_sizes_ok(int B, int N, int Hq, int Hkv, int D) {
    return B >= 0 && N >= 1 && N <= SPEC_MAX_TREE_NODES && Hkv >= 1 && Hkv <= 1024 && Hq >= Hkv &&
           Hq % Hkv == 0 && Hq <= 1 << 16 && (D == 64 || D == 128) &&
           static_cast<long long>(B) * N * Hq <= INT_MAX / 256;
}

}  // namespace
}  // namespace specv

using namespace specv;

SPEC_EXPORT int spec_kv_append(const spec_kv_cache *cache, const int32_t *page_table,
                               int table_width, const int32_t *starts, const void *k,
                               const void *v, int64_t token_stride, const int32_t *rows, int B,
                               int N, int M, int dtype, spec_stream_t stream) {
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
    AppendArgs a;
    const int rc = view_of(cache, &a.c);
    if (rc != SPEC_OK) return rc;
    if (B < 0 || N < 0 || M < 0 || table_width < 0 || (!rows && M != N) ||
        static_cast<long long>(B) * M > INT_MAX / a.c.Hkv ||
        !stride_ok(&token_stride, static_cast<long long>(a.c.Hkv) * a.c.D))
        return SPEC_ERR_SHAPE;
    if (B == 0 || M == 0 || N == 0 || table_width == 0) return SPEC_OK;
    if (!page_table || !starts || !k || !v) return SPEC_ERR_NULL;
    if (!aligned(page_table, 4) || !aligned(starts, 4) || !aligned(k, 16) || !aligned(v, 16) ||
        (rows && !aligned(rows, 4)))
        return SPEC_ERR_ALIGN;
    a.table = page_table;
    a.width = table_width;
    a.starts = starts;
    a.k = k;
    a.v = v;
    a.stride = token_stride;
    a.rows = rows;
    a.B = B;
    a.N = N;
    a.M = M;
    return launch_kv_append(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

SPEC_EXPORT int spec_kv_read(const spec_kv_cache *cache, const int32_t *page_table,
                             int table_width, const int32_t *starts, void *out_k, void *out_v,
                             int B, int M, int dtype, spec_stream_t stream) {
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
    ReadArgs a;
    const int rc = view_of(cache, &a.c);
    if (rc != SPEC_OK) return rc;
    if (B < 0 || M < 0 || table_width < 0 || static_cast<long long>(B) * M > INT_MAX / a.c.Hkv)
        return SPEC_ERR_SHAPE;
    if (B == 0 || M == 0 || (!out_k && !out_v)) return SPEC_OK;
    if ((!page_table && table_width) || !starts) return SPEC_ERR_NULL;
    if (!aligned(page_table, 4) || !aligned(starts, 4) || (out_k && !aligned(out_k, 16)) ||
        (out_v && !aligned(out_v, 16)))
        return SPEC_ERR_ALIGN;
    a.table = page_table;
    a.width = table_width;
    a.starts = starts;
    a.out_k = out_k;
    a.out_v = out_v;
    a.B = B;
    a.M = M;
    return launch_kv_read(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

SPEC_EXPORT int spec_attn_workspace_size(int B, int N, int Hq, int Hkv, int D, size_t *bytes) {
    if (!bytes) return SPEC_ERR_NULL;
    if (!attn_sizes_ok(B, N, Hq, Hkv, D)) return SPEC_ERR_SHAPE;
    *bytes = kErrBytes + attn_work_bytes(B, N, Hq, Hkv, D);
    return SPEC_OK;
}

SPEC_EXPORT int spec_attn_shared(const spec_kv_cache *cache, const int32_t *shared_table,
                                 int shared_len, const int32_t *page_table, int table_width,
                                 const int32_t *lens, const void *q, int64_t q_stride,
                                 const uint8_t *mask, const int32_t *pos, const float *slopes,
                                 int B, int N, int Hq, float scale, float cap, int window,
                                 int dtype, void *out, float *out_lse, void *workspace,
                                 size_t workspace_bytes, spec_stream_t stream) {
    if (dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
    AttnArgs a;
    const int rc = view_of(cache, &a.c);
    if (rc != SPEC_OK) return rc;
    if (!attn_sizes_ok(B, N, Hq, a.c.Hkv, a.c.D) || table_width < 0 ||
        table_width > (INT_MAX >> a.c.page_shift) || shared_len < 0 ||
        static_cast<long long>(shared_len) + (static_cast<long long>(table_width) << a.c.page_shift) >
            INT_MAX ||
        !stride_ok(&q_stride, static_cast<long long>(Hq) * a.c.D))
        return SPEC_ERR_SHAPE;
    if (!std::isfinite(scale) || !std::isfinite(cap) || cap < 0.0f || window < 0)
        return SPEC_ERR_PARAM;
    if (B == 0) return SPEC_OK;
    if ((shared_len > 0 && !shared_table) || (!page_table && table_width) || !lens || !q || !out)
        return SPEC_ERR_NULL;
    if (!aligned(shared_table, 4) || !aligned(page_table, 4) || !aligned(lens, 4) ||
        !aligned(q, 16) || (pos && !aligned(pos, 4)) || (slopes && !aligned(slopes, 4)) ||
        !aligned(out, 16) || (out_lse && !aligned(out_lse, 4)))
        return SPEC_ERR_ALIGN;
    if (!workspace || workspace_bytes < kErrBytes + attn_work_bytes(B, N, Hq, a.c.Hkv, a.c.D))
        return SPEC_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SPEC_ERR_ALIGN;
    a.shared_table = shared_table;
    a.shared_len = shared_len;
    a.table = page_table;
    a.width = table_width;
    a.lens = lens;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.q_stride = q_stride;
    a.mask = mask;
    a.pos = pos;
    a.slopes = slopes;
    a.B = B;
    a.N = N;
    a.Hq = Hq;
    a.G = Hq / a.c.Hkv;
    a.scale = scale;
    // From 2^64 on a cap is none: fp32 scores that it would change are past any
    // difference that the softmax tells, and scale / cap would leave fp32's range.
    a.cap = cap < 0x1p64f ? cap : 0.0f;
    a.window = window;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = out_lse;
    a.err = static_cast<uint32_t *>(workspace);
    a.work = static_cast<char *>(workspace) + kErrBytes;
    return launch_attn(a, reinterpret_cast<cudaStream_t>(stream));
}

SPEC_EXPORT int spec_attn_tree(const spec_kv_cache *cache, const int32_t *page_table,
                               int table_width, const int32_t *lens, const void *q,
                               int64_t q_stride, const uint8_t *mask, const int32_t *pos,
                               const float *slopes, int B, int N, int Hq, float scale, float cap,
                               int window, int dtype, void *out, float *out_lse, void *workspace,
                               size_t workspace_bytes, spec_stream_t stream) {
    return spec_attn_shared(cache, nullptr, 0, page_table, table_width, lens, q, q_stride, mask,
                            pos, slopes, B, N, Hq, scale, cap, window, dtype, out, out_lse,
                            workspace, workspace_bytes, stream);
}
