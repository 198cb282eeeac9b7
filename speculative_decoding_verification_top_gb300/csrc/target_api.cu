// target_api.cu -- the C entries of include/spec_attn.h for rotary positions and
// the latent cache: argument checks and dispatch (rope.cu, latent.cu).

#include "checks.cuh"
#include "target.cuh"
#include "wide.h"

namespace specv {
namespace {

constexpr int kMaxHead = 1024;  // elements of a head that spec_rope takes
constexpr int kRotary = 64;     // rotary elements of a latent cache's row
constexpr int kMaxRows = 1 << 30;  // query rows of a latent attention: what a 32-bit number counts with room

bool rot_ok(int rot, int D) { return rot >= 16 && rot % 16 == 0 && rot <= D; }

// Do `count` tokens from x on, each `size` elements of `bytes` and `stride` apart, share
// no element with those from y on?  Parts of one projection, of one stride, lie
// between each other.
bool apart(const void *x, long long x_stride, long long x_size, const void *y, long long y_stride, long long y_size,
           long long count, int bytes) {
    using Address = __int128;  // the largest strides and counts pass 64 bits
    const Address from_x = reinterpret_cast<uintptr_t>(x), from_y = reinterpret_cast<uintptr_t>(y), tokens = count;
    const Address to_x = from_x + ((tokens - 1) * x_stride + x_size) * bytes,
                  to_y = from_y + ((tokens - 1) * y_stride + y_size) * bytes;
    if (to_x <= from_y || to_y <= from_x) return true;
    if (x_stride != y_stride) return false;
    const Address period = Address(x_stride) * bytes, at = ((from_y - from_x) % period + period) % period;
    return at >= x_size * bytes && at + y_size * bytes <= period;
}

// The turn's arguments; `first` + rot within the head is the caller's check.
int turn_of(const uint64_t *freqs, int rot, float amplitude, int layout, Turn *t) {
    if (layout != SPEC_ROPE_HALF && layout != SPEC_ROPE_INTERLEAVED) return SPEC_ERR_MODE;
    if (!std::isfinite(amplitude)) return SPEC_ERR_PARAM;
    t->freqs = reinterpret_cast<const unsigned long long *>(freqs);
    t->rot = rot;
    t->first = 0;
    t->amplitude = amplitude;
    t->interleaved = layout == SPEC_ROPE_INTERLEAVED;
    t->inverse = 0;
    return SPEC_OK;
}

int latent_view(const spec_latent_cache *cache, LatentView *c) {
    if (!cache) return SPEC_ERR_NULL;
    if (cache->num_pages < 1 || (cache->C != 128 && cache->C != 256 && cache->C != 512) || cache->R != kRotary ||
        (cache->page != 16 && cache->page != 32 && cache->page != 64 && cache->page != 128))
        return SPEC_ERR_SHAPE;
    if (!cache->data) return SPEC_ERR_NULL;
    if (!aligned(cache->data, 16)) return SPEC_ERR_ALIGN;
    c->data = static_cast<__nv_bfloat16 *>(cache->data);
    c->num_pages = cache->num_pages;
    c->page_shift = 31 - __builtin_clz(static_cast<unsigned>(cache->page));
    c->C = cache->C;
    c->R = cache->R;
    return SPEC_OK;
}

bool latent_sizes_ok(int B, int N, int H, int C) {
    return B >= 0 && N >= 1 && N <= SPEC_MAX_TREE_NODES && H >= 1 && H <= 1024 && (C == 128 || C == 256 || C == 512) &&
           static_cast<long long>(B) * N * H <= kMaxRows;
}

}  // namespace
}  // namespace specv

using namespace specv;

SPEC_EXPORT int spec_rope_freqs(int rot, double base, int scaling, double factor, double original, double low,
                                double high, uint64_t *freqs) {
    if (!freqs) return SPEC_ERR_NULL;
    if (!rot_ok(rot, kMaxHead)) return SPEC_ERR_SHAPE;
    if (scaling < SPEC_ROPE_PLAIN || scaling > SPEC_ROPE_INDEX) return SPEC_ERR_MODE;
    const double most = 1e30, pi = 3.14159265358979323846;
    const bool parts = scaling == SPEC_ROPE_TURNS || scaling == SPEC_ROPE_INDEX;
    if (!(base > 1.0 && base <= most) || (scaling != SPEC_ROPE_PLAIN && !(factor >= 1.0 && factor <= most)) ||
        (parts && !(original >= 1.0 && original <= most && low > 0.0 && low < high && high <= most)))
        return SPEC_ERR_PARAM;
    double a = 0.0, b = 0.0;
    if (scaling == SPEC_ROPE_INDEX) {
        auto at = [&](double turns) { return rot * std::log(original / (2.0 * pi * turns)) / (2.0 * std::log(base)); };
        a = std::fmax(0.0, std::floor(at(high)));
        b = std::fmin(rot - 1.0, std::ceil(at(low)));
    }
    // In two doubles: a frequency has up to 62 bits, and what it is off by grows with
    // the position.
    const Wide one = wide(1.0), per_turn = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / (2 pi)
    const Wide step = one / root(base, rot / 2);
    Wide plain = one;  // base^(-2 i / rot)
    for (int i = 0; i < rot / 2; ++i, plain = plain * step) {
        Wide theta = plain, w = wide(0.0);
        if (scaling == SPEC_ROPE_TURNS) w = share(wide(original) * theta * per_turn - wide(low), wide(high) - wide(low));
        if (scaling == SPEC_ROPE_INDEX) w = one - share(wide(i - a), wide(std::fmax(b - a, 1e-3)));
        if (scaling != SPEC_ROPE_PLAIN) theta = theta * (w + (one - w) / wide(factor));
        // theta <= 1: under a sixth of a turn, so the product is below 2^62
        freqs[i] = nearest(theta * per_turn * wide(0x1p64));
    }
    return SPEC_OK;
}

SPEC_EXPORT int spec_rope(const void *x, int64_t x_stride, void *out, int64_t out_stride, const uint64_t *freqs, int rot,
                          int first, float amplitude, int layout, int inverse, const int32_t *pos, int B, int N, int H,
                          int D, int dtype, spec_stream_t stream) {
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
    RopeArgs a;
    const int rc = turn_of(freqs, rot, amplitude, layout, &a.t);
    if (rc != SPEC_OK) return rc;
    if (B < 0 || N < 0 || H < 1 || D < 16 || D > kMaxHead || D % 16 || !rot_ok(rot, D) || first < 0 || first % 16 ||
        first > D - rot || H > 1 << 20 || static_cast<long long>(B) * N > INT_MAX / (static_cast<long long>(H) * (D / 16)) ||
        !stride_ok(&x_stride, static_cast<long long>(H) * D) || !stride_ok(&out_stride, static_cast<long long>(H) * D) ||
        (x == out && x_stride != out_stride))
        return SPEC_ERR_SHAPE;
    if (B == 0 || N == 0) return SPEC_OK;
    if (!x || !out || !freqs || !pos) return SPEC_ERR_NULL;
    if (!aligned(x, 16) || !aligned(out, 16) || !aligned(freqs, 16) || !aligned(pos, 4)) return SPEC_ERR_ALIGN;
    const long long size = static_cast<long long>(H) * D, count = static_cast<long long>(B) * N;
    if (x != out && !apart(x, x_stride, size, out, out_stride, size, count, dtype == SPEC_F32 ? 4 : 2)) return SPEC_ERR_SHAPE;
    a.x = x;
    a.out = out;
    a.x_stride = x_stride;
    a.out_stride = out_stride;
    a.pos = pos;
    a.tokens = B * N;
    a.H = H;
    a.D = D;
    a.t.first = first;
    a.t.inverse = inverse != 0;
    return launch_rope(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

SPEC_EXPORT int spec_kv_append_rope(const spec_kv_cache *cache, const int32_t *page_table, int table_width,
                                    const int32_t *starts, const void *k, const void *v, int64_t token_stride,
                                    const int32_t *rows, const int32_t *pos, const uint64_t *freqs, int rot,
                                    float amplitude, int layout, const void *q, int64_t q_stride, void *out_q,
                                    int64_t out_q_stride, int B, int N, int M, int Hq, int dtype, spec_stream_t stream) {
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
    AppendRopeArgs a = {};
    int rc = view_of(cache, &a.a.c);
    if (rc != SPEC_OK) return rc;
    rc = turn_of(freqs, rot, amplitude, layout, &a.t);
    if (rc != SPEC_OK) return rc;
    const CacheView &c = a.a.c;
    const bool queries = q || out_q;
    const long long units = c.D / 16;
    if (B < 0 || N < 0 || M < 0 || table_width < 0 || (!rows && M != N) || !rot_ok(rot, c.D) ||
        static_cast<long long>(B) * M > INT_MAX / 2 / (c.Hkv * units) ||
        !stride_ok(&token_stride, static_cast<long long>(c.Hkv) * c.D) ||
        (queries && (Hq < 1 || Hq > 1 << 16 || static_cast<long long>(B) * N > INT_MAX / 2 / (Hq * units) ||
                     !stride_ok(&q_stride, static_cast<long long>(Hq) * c.D) ||
                     !stride_ok(&out_q_stride, static_cast<long long>(Hq) * c.D) || (q == out_q && q_stride != out_q_stride))))
        return SPEC_ERR_SHAPE;
    if (queries && rows) return SPEC_ERR_PARAM;
    if (B == 0 || M == 0 || N == 0 || (table_width == 0 && !queries)) return SPEC_OK;
    if ((!page_table && table_width) || !starts || !k || !v || !freqs || (queries && (!q || !out_q))) return SPEC_ERR_NULL;
    if (!aligned(page_table, 4) || !aligned(starts, 4) || !aligned(k, 16) || !aligned(v, 16) || !aligned(rows, 4) ||
        !aligned(pos, 4) || !aligned(freqs, 16) || !aligned(q, 16) || !aligned(out_q, 16))
        return SPEC_ERR_ALIGN;
    if (queries) {
        const long long size = static_cast<long long>(Hq) * c.D, kv = static_cast<long long>(c.Hkv) * c.D;
        const long long count = static_cast<long long>(B) * N;
        const int bytes = dtype == SPEC_F32 ? 4 : 2;
        if ((q != out_q && !apart(q, q_stride, size, out_q, out_q_stride, size, count, bytes)) ||
            !apart(k, token_stride, kv, out_q, out_q_stride, size, count, bytes) ||
            !apart(v, token_stride, kv, out_q, out_q_stride, size, count, bytes))
            return SPEC_ERR_SHAPE;
    }
    a.a.table = page_table;
    a.a.width = table_width;
    a.a.starts = starts;
    a.a.k = k;
    a.a.v = v;
    a.a.stride = token_stride;
    a.a.rows = rows;
    a.a.B = B;
    a.a.N = N;
    a.a.M = M;
    a.pos = pos;
    a.q = q;
    a.out_q = out_q;
    a.q_stride = q_stride;
    a.out_q_stride = out_q_stride;
    a.Hq = queries ? Hq : 0;
    return launch_kv_append_rope(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

SPEC_EXPORT int spec_latent_append(const spec_latent_cache *cache, const int32_t *page_table, int table_width,
                                   const int32_t *starts, const void *c, int64_t c_stride, const void *r, int64_t r_stride,
                                   const int32_t *rows, const int32_t *pos, const uint64_t *freqs, float amplitude,
                                   int layout, int B, int N, int M, int dtype, spec_stream_t stream) {
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_DTYPE;
    LatentAppendArgs a = {};
    int rc = latent_view(cache, &a.c);
    if (rc != SPEC_OK) return rc;
    rc = turn_of(freqs, freqs ? a.c.R : 0, amplitude, layout, &a.t);
    if (rc != SPEC_OK) return rc;
    if (B < 0 || N < 0 || M < 0 || table_width < 0 || (!rows && M != N) ||
        static_cast<long long>(B) * M > INT_MAX / ((a.c.C + a.c.R) / 16) || !stride_ok(&c_stride, a.c.C) ||
        !stride_ok(&r_stride, a.c.R))
        return SPEC_ERR_SHAPE;
    if (B == 0 || M == 0 || N == 0 || table_width == 0) return SPEC_OK;
    if (!page_table || !starts || !c || !r) return SPEC_ERR_NULL;
    if (!aligned(page_table, 4) || !aligned(starts, 4) || !aligned(c, 16) || !aligned(r, 16) || !aligned(rows, 4) ||
        !aligned(pos, 4) || !aligned(freqs, 16))
        return SPEC_ERR_ALIGN;
    a.table = page_table;
    a.width = table_width;
    a.starts = starts;
    a.x = c;
    a.r = r;
    a.x_stride = c_stride;
    a.r_stride = r_stride;
    a.rows = rows;
    a.pos = pos;
    a.B = B;
    a.N = N;
    a.M = M;
    return launch_latent_append(a, dtype, reinterpret_cast<cudaStream_t>(stream));
}

SPEC_EXPORT int spec_latent_workspace_size(int B, int N, int H, int C, size_t *bytes) {
    if (!bytes) return SPEC_ERR_NULL;
    if (!latent_sizes_ok(B, N, H, C)) return SPEC_ERR_SHAPE;
    *bytes = kErrBytes + latent_work_bytes(B, N, H, C);
    return SPEC_OK;
}

SPEC_EXPORT int spec_latent_attn(const spec_latent_cache *cache, const int32_t *page_table, int table_width,
                                 const int32_t *lens, const void *q, int64_t q_stride, const uint8_t *mask, int B, int N,
                                 int H, float scale, void *out, float *out_lse, void *workspace, size_t workspace_bytes,
                                 spec_stream_t stream) {
    LatentArgs a = {};
    const int rc = latent_view(cache, &a.c);
    if (rc != SPEC_OK) return rc;
    if (!latent_sizes_ok(B, N, H, a.c.C) || table_width < 0 || table_width > (INT_MAX >> a.c.page_shift) ||
        !stride_ok(&q_stride, static_cast<long long>(H) * (a.c.C + a.c.R)))
        return SPEC_ERR_SHAPE;
    if (!std::isfinite(scale)) return SPEC_ERR_PARAM;
    if (B == 0) return SPEC_OK;
    if ((!page_table && table_width) || !lens || !q || !out) return SPEC_ERR_NULL;
    if (!aligned(page_table, 4) || !aligned(lens, 4) || !aligned(q, 16) || !aligned(out, 16) || !aligned(out_lse, 4))
        return SPEC_ERR_ALIGN;
    if (!workspace || workspace_bytes < kErrBytes + latent_work_bytes(B, N, H, a.c.C)) return SPEC_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return SPEC_ERR_ALIGN;
    a.table = page_table;
    a.width = table_width;
    a.lens = lens;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.q_stride = q_stride;
    a.mask = mask;
    a.B = B;
    a.N = N;
    a.H = H;
    a.scale = scale;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = out_lse;
    a.err = static_cast<uint32_t *>(workspace);
    a.work = static_cast<char *>(workspace) + kErrBytes;
    return launch_latent(a, reinterpret_cast<cudaStream_t>(stream));
}
