// attn.cu -- attention of a target pass's new tokens to the paged cache.
//
// For one query row (token i, query head h) over the positions j it sees:
//   t_j = log2(e) * score_j;  m = max t_j;  l = sum 2^(t_j - m);
//   out = sum 2^(t_j - m) v_j / l.
// One pass over the cache.  m, l and the output's accumulator are running
// values; two partial results (m, l, O) of the same row join as
//   M = max m;  L = sum 2^(m - M) l;  out = sum 2^(m - M) O / L.
//
// attn_kernel   persistent, one CTA per SM.  A unit of work is one key/value
//               head of one sequence (or of the shared prefix) and up to 256
//               query rows: the N G rows (new token, query head of the group)
//               that share the head's keys.  All units' tiles of 128
//               positions, laid end to end, are cut into equal shares, one
//               per CTA; a share's piece of a unit is a segment, and leaves
//               one partial result per row.
//                 warp 8      loads key and value tiles page by page (TMA)
//                             into a ring of slots
//                 warp 9      issues the products (tcgen05): S = Q K^T into
//                             TMEM, then O += P V with P in TMEM
//                 warps 0-3, 4-7   two softmax groups, a thread per row: S
//                             from TMEM, 2^(t - m), P back into TMEM
//                 warp 10     the e4m3 cache's exponents, as factors
//                 warp 11     the query tiles (two, so mostly a segment ahead)
//               A unit of up to 128 rows alternates its tiles between the
//               two groups, each with its own S and O (TMEM: 2 x 128 + 2 x D
//               columns), so that one group's softmax runs under the other's
//               products.  A larger unit gives each group 128 rows of its
//               own and both work on every tile.
// join_kernel   a programmatic dependent: joins each row's partial results.
//
// e4m3 cache: keys and values go to the tensor cores as the bytes they are.
// The bf16 query, scaled per row by a power of two, splits exactly into two
// e4m3 terms (4 + 4 significant bits; what falls under 2^-10 of the scaled
// unit is at most 2^-18 of the row's maximum), and S = Q1 K^T + Q2 K^T at the
// e4m3 rate costs what one bf16 product does.  The weights split into two
// terms likewise (2^-8 relative at worst).  A key's exponent multiplies its
// column of S; a value's exponent is added to t_j, so that the weight carries
// it, and taken back in l.

#include "attn.cuh"
#include "tensor.cuh"

namespace specv {
namespace {

constexpr int kTile = 128;        // positions a tile
constexpr int kGroupRows = 128;   // query rows a softmax group
constexpr int kAttnThreads = 384;
constexpr int kMaxSlots = 16;
constexpr int kScaleRing = 4;
constexpr int kMaxGrid = 152;
constexpr int kSmemMax = 232448;  // bytes a CTA may have
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kStalled = SPEC_DATA_STALL;

// How the units are numbered and cut; the same arithmetic in both kernels.
struct Plan {
    int B, N, G, Hkv, width, page_shift;
    int R, rt, ru;        // rows, 128-row tiles and units a (sequence, head)
    int Ls;               // shared prefix
    int sR, srt, sru, sT; // the same for the prefix (rows of all sequences), and its tiles
    int sT0;              // first tile of the prefix (0: windows do not trim it)
    int rc, src;          // rows a partial result holds (own, shared)
    int parts, sparts;    // partial results a slot: 2 where units pass 128 rows
    int grid;
    const int32_t *lens, *pos;
    int window;
    long long *base;      // [B + 2] first cost of each sequence's units; the total; a CTA's share
    float4 *o, *so;       // [slots, parts, D / 4, rc] partial O
    float2 *ml, *sml;     // [slots, parts, rc] partial (m, l)
};

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// A sequence's tiles [t0, t1): those a row may see.
struct Span {
    int len, t0, t1;
};

__device__ __forceinline__ Span span_of(const Plan &p, int b) {
    Span s;
    s.len = p.lens[b];
    if (s.len < 0 || s.len > (p.width << p.page_shift)) s.len = 0;  // the join fails it
    s.t1 = (s.len + kTile - 1) / kTile;
    s.t0 = 0;
    if (p.window > 0) {
        // pos_i - pos_j < window for some row: j >= min pos_i - window + 1 among the context;
        // the new tokens themselves are kept whatever their positions say.
        long long least = static_cast<long long>(p.Ls) + s.len - p.N;
        if (p.pos) {
            int m = INT_MAX;
            for (int n = 0; n < p.N; ++n) m = min(m, p.pos[static_cast<long long>(b) * p.N + n]);
            least = m;
        }
        long long j = least - p.window + 1 - p.Ls;
        j = min(j, static_cast<long long>(s.len) - p.N);
        if (j > 0) s.t0 = min(static_cast<int>(j / kTile), s.t1);
    }
    return s;
}

// One unit and this CTA's tiles [t0, t1) of it.
struct Segment {
    bool shared, dual;
    int b, h, row0, rows;  // rows [row0, row0 + rows) of the unit's (sequence, head)
    int t0, t1, len, slot;
};

// Walks a CTA's share [x, end) of the cost line.  A tile of a unit costs its
// row tiles (1 or 2): the products' work.  Every warp walks it by itself.
struct Walk {
    long long ubase, x, end;
    int b, h, u;          // next unit; b = -1: the shared prefix
    Span s;
    const Plan &p;

    __device__ Walk(const Plan &plan, long long from, long long to, int b0, long long base0)
        : ubase(0), x(from), end(to), b(b0), h(0), u(0), s(), p(plan) {
        if (x >= end) {
            ubase = end;
            return;
        }
        const bool sh = b < 0;
        if (!sh) s = span_of(p, b);
        const int T = sh ? p.sT : s.t1 - s.t0, rt = sh ? p.srt : p.rt;
        const long long in = x - base0, head = static_cast<long long>(T) * rt;
        if (head == 0) return;
        h = static_cast<int>(in / head);
        u = static_cast<int>((in - h * head) / (2ll * T));
        ubase = base0 + h * head + u * 2ll * T;
    }

    __device__ bool next(Segment *g) {
        while (ubase < end && b < p.B) {
            const bool sh = b < 0;
            const int T = sh ? p.sT : s.t1 - s.t0;
            if (T == 0) {  // a sequence without tiles
                advance_sequence();
                continue;
            }
            const int R = sh ? p.sR : p.R, ru = sh ? p.sru : p.ru;
            g->shared = sh;
            g->b = b;
            g->h = h;
            g->row0 = u * 2 * kGroupRows;
            g->rows = min(R - g->row0, 2 * kGroupRows);
            g->dual = g->rows > kGroupRows;
            const int c = g->dual ? 2 : 1;
            const int first = sh ? p.sT0 : s.t0;
            g->t0 = x > ubase ? static_cast<int>((x - ubase + c - 1) / c) : 0;
            g->t1 = static_cast<int>(min(static_cast<long long>(T), (end - ubase + c - 1) / c));
            g->len = sh ? p.Ls : s.len;
            g->slot = ((sh ? 0 : b) * p.Hkv + h) * ru + u + static_cast<int>(blockIdx.x);
            const bool some = g->t0 < g->t1;
            g->t0 += first;
            g->t1 += first;
            ubase += static_cast<long long>(T) * c;
            if (++u == ru) {
                u = 0;
                if (++h == p.Hkv) {
                    h = 0;
                    if (sh) {
                        b = 0;
                        s = span_of(p, 0);
                    } else {
                        advance_sequence();
                    }
                }
            }
            if (some) return true;
        }
        return false;
    }

    __device__ void advance_sequence() {
        ++b;
        if (b < p.B) s = span_of(p, b);
    }
};

struct Barriers {
    unsigned long long full[kMaxSlots], empty[kMaxSlots];
    unsigned long long scale_full[kScaleRing], scale_empty[kScaleRing];
    unsigned long long q_full[2], q_empty[2], o_full, s_full[2], p_full[2], fold, drained;
};

struct Shared {
    Barriers bar;
    long long scan[kAttnThreads / 32 + 1];
    long long total, from, to, base0;
    int b0;
    float2 ml[8][32];  // per softmax warp and lane: (m, l), for the fold
    uint32_t tmem;
    int dead;          // a wait ran out: everyone leaves
    int fail[16];      // per segment (mod 16): a page id out of range
    int odd[16];       // per segment (mod 16): a cleaned tile held values that are not finite
};

template <int D, bool E4M3>
struct Shape {
    static constexpr int kRow = E4M3 ? D : 128;              // bytes of a shared-memory matrix row
    static constexpr int kHalves = E4M3 ? 1 : D / 64;        // 64-column blocks of a bf16 matrix
    static constexpr int kMat = kTile * kRow;                // bytes of one block
    static constexpr int kSlot = kMat * kHalves;             // a key or value tile
    static constexpr int kQ = E4M3 ? 2 * kMat : kSlot;       // a group's query tile
    static constexpr int kScale = E4M3 ? (kScaleRing * 3 * kTile + 2 * kGroupRows) * 4 : 0;  // and query factors
    static constexpr int kFixed = kScale + static_cast<int>((sizeof(Shared) + 127) / 128 * 128);
    static constexpr int kRoom = (kSmemMax - kFixed - 2 * kQ) / kSlot;
    static constexpr int kSlots = kRoom < kMaxSlots ? kRoom : kMaxSlots;
    static constexpr int kBytes = kFixed + 2 * kQ + kSlots * kSlot;
};

struct KernelArgs {
    AttnArgs a;
    Plan p;
};

// Whether row (own row r of sequence b, its token's position pos_i) sees own
// position j; *pos_j gets the position's index.
__device__ __forceinline__ bool sees(const AttnArgs &a, int b, int n, int pos_i, int first, int len,
                                     int j, int *pos_j) {
    *pos_j = a.shared_len + j;
    if (j >= len) return false;
    const int c = j - first;
    if (c >= 0) {
        const long long bn = static_cast<long long>(b) * a.N;
        if (a.pos) *pos_j = a.pos[bn + c];
        if (a.mask ? a.mask[(bn + n) * a.N + c] == 0 : c > n) return false;
    }
    return a.window == 0 || static_cast<long long>(pos_i) - *pos_j < a.window;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 e4m3_values(uint32_t pair) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(pair), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Few query rows are repeated over a group's 128 lanes.
__device__ __forceinline__ int copies_of(bool dual, int rows) { return dual || rows > 64 ? 1 : rows > 32 ? 2 : 4; }

// Query row -> rows row, row + span, ... of the group's tile in shared memory
// (zeros without a query), and its factor 2^e (see the top of the file).
template <int D, bool E4M3>
__device__ __forceinline__ void stage_query(const __nv_bfloat16 *q, uint8_t *tile, int row, int span, bool neg,
                                            float *factor) {
    using S = Shape<D, E4M3>;
    uint4 u[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
        u[i] = q ? __ldg(reinterpret_cast<const uint4 *>(q) + i) : make_uint4(0, 0, 0, 0);
    const uint32_t flip = neg ? 0x80008000u : 0u;
    if (!E4M3) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            uint4 w = u[i];
            w.x ^= flip, w.y ^= flip, w.z ^= flip, w.w ^= flip;
            for (int r = row; r < kGroupRows; r += span)
                *reinterpret_cast<uint4 *>(tile + (i / 8) * S::kMat + swizzled<S::kRow>(r, (i % 8) * 16)) = w;
        }
        return;
    }
    uint32_t top = 0;  // bf16 bits of max |q|
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7fffu, w[k] >> 16 & 0x7fffu));
    }
    // e: max |q| <= 448 * 2^e
    int e = static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);
    e = max(-120, min(120, e));
    const float f = exp2i(-e);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint4 v = u[2 * i + k / 2];
            const uint32_t a = (k & 1 ? v.z : v.x) ^ flip, b = (k & 1 ? v.w : v.y) ^ flip;
            const float x0 = __uint_as_float(a << 16) * f, x1 = __uint_as_float(a & 0xffff0000u) * f;
            const float x2 = __uint_as_float(b << 16) * f, x3 = __uint_as_float(b & 0xffff0000u) * f;
            const uint32_t p = e4m3_pair(x0, x1), r = e4m3_pair(x2, x3);
            const float2 y = e4m3_values(p), z = e4m3_values(r);
            hi[k] = p | r << 16;
            lo[k] = e4m3_pair(x0 - y.x, x1 - y.y) | e4m3_pair(x2 - z.x, x3 - z.y) << 16;
        }
        for (int r = row; r < kGroupRows; r += span) {
            const uint32_t o = swizzled<S::kRow>(r, i * 16);
            *reinterpret_cast<uint4 *>(tile + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(tile + S::kMat + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
    for (int r = row; r < kGroupRows; r += span) factor[r] = exp2i(e);
}

// Row `row` of a value tile whose positions some rows do not see: zeros where
// the position is not held (the slot has whatever was there), and zeros for
// elements that are not finite, so that an unseen one does not reach a row
// through 0 * inf.  Returns whether a held element was not finite.
template <int D, bool E4M3>
__device__ __forceinline__ bool clean_values(uint8_t *tile, int row, bool held) {
    using S = Shape<D, E4M3>;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < D * (E4M3 ? 1 : 2) / 16; ++i) {
        uint4 *at = reinterpret_cast<uint4 *>(tile + (i * 16 / S::kRow) * S::kMat +
                                              swizzled<S::kRow>(row, i * 16 % S::kRow));
        if (!held) {
            *at = make_uint4(0, 0, 0, 0);
            continue;
        }
        uint4 u = *at;
        uint32_t w[4] = {u.x, u.y, u.z, u.w};
        bool here = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t keep;
            if (E4M3) {
                // 0x80 in each byte that is 0x7f or 0xff
                const uint32_t nan = ((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                keep = ~((nan >> 7) * 0xffu);
            } else {
                keep = ((w[k] & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) |
                       ((w[k] & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u);
            }
            here |= keep != 0xffffffffu;
            w[k] &= keep;
        }
        if (here) *at = make_uint4(w[0], w[1], w[2], w[3]);
        odd |= here;
    }
    return odd;
}

// Growth of t over the reference maximum that is let stand: a weight stays
// under 2^8 (bf16), or 2^5 * 2^3.75 < 448 (e4m3, whose weights are scaled by
// 2^5 so that small ones keep their second term).
constexpr float kSlackBf16 = 8.0f, kSlackE4M3 = 3.75f, kLiftE4M3 = 5.0f;

// What a softmax thread holds of its row.
struct Row {
    int b, n, tok;           // sequence, new token, token of the batch
    int first, pos_i;        // own position of token 0, the token's position index
    bool has;
    float rs, slope;         // score factor (the log2 e and the query's own in it), slope * log2 e
    float m, l;              // reference maximum and sum
};

// t of 32 columns from column `col` of a tile, from the raw products v in place.
template <bool E4M3, bool EXTRA>
__device__ __forceinline__ float scores32(const AttnArgs &a, const Segment &g, const Row &x, int j0, int col,
                                          bool whole, const float *fa, float (&v)[32]) {
    // Columns of positions some rows do not see: a row's set depends on its
    // token alone, so the warp finds the sets of its tokens one by one, a
    // lane a column.
    uint32_t seen = 0xffffffffu;
    int pos_col = 0;  // position index of this lane's column
    if (!whole) {
        const int lane = threadIdx.x & 31, j = j0 + col + lane, c = j - x.first;
        const bool held = j < g.len, node = !g.shared && c >= 0;
        pos_col = (g.shared ? 0 : a.shared_len) + j;
        if (node && held && a.pos) pos_col = a.pos[static_cast<long long>(x.b) * a.N + c];
        uint32_t todo = __ballot_sync(0xffffffffu, x.has);
        seen = 0;
        while (todo) {
            const int from = __ffs(todo) - 1;
            const int tok = __shfl_sync(0xffffffffu, x.tok, from), n = __shfl_sync(0xffffffffu, x.n, from);
            const int pos_i = __shfl_sync(0xffffffffu, x.pos_i, from);
            bool y = held;
            if (node && held) y = a.mask ? a.mask[static_cast<long long>(tok) * a.N + c] != 0 : c <= n;
            y = y && (a.window == 0 || static_cast<long long>(pos_i) - pos_col < a.window);
            const uint32_t word = __ballot_sync(0xffffffffu, y);
            const bool me = x.has && x.tok == tok;
            if (me) seen = word;
            todo &= ~__ballot_sync(0xffffffffu, me);
        }
    }
    const float far0 =
        EXTRA ? static_cast<float>((g.shared ? 0 : a.shared_len) + j0 + col - x.pos_i) : 0.0f;
    const float capl = a.cap * kLog2e;
    float top[2] = {kNegInf, kNegInf};
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
        float4 k4 = {}, b4 = {};
        if (E4M3) {
            k4 = *reinterpret_cast<const float4 *>(fa + col + c);
            b4 = *reinterpret_cast<const float4 *>(fa + kTile + col + c);
        }
        const float fk[4] = {k4.x, k4.y, k4.z, k4.w}, fb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float y = v[c + k];
            if (E4M3) y *= fk[k];
            if (EXTRA && a.cap > 0.0f) {
                // cap tanh(y) log2 e, tanh(y) = 1 - 2 / (1 + e^2y)
                const float e = ex2(y * x.rs * (2.0f * kLog2e));
                y = capl - __fdividef(2.0f * capl, 1.0f + e);
            } else if (!E4M3 || EXTRA) {
                y *= x.rs;
            }
            if (EXTRA) {
                float far = far0 + static_cast<float>(c + k);
                if (!whole && a.pos) far = static_cast<float>(__shfl_sync(0xffffffffu, pos_col, c + k) - x.pos_i);
                y = fmaf(x.slope, far, y);
                if (E4M3) y += fb[k];
            } else if (E4M3) {
                y = fmaf(y, x.rs, fb[k]);
            }
            if (!whole && !(seen >> (c + k) & 1u)) y = kNegInf;
            v[c + k] = y;
            top[k & 1] = fmaxf(top[k & 1], y);
        }
    }
    return fmaxf(top[0], top[1]);
}

// Weights 2^(t - ref) of 32 columns into TMEM as the product's operand: 16
// columns of bf16 pairs, or 8 of first and 8 of second e4m3 terms.
template <bool E4M3>
__device__ __forceinline__ float weights32(uint32_t dst, float ref, const float *fc, const float (&t)[32]) {
    float sum[4] = {};
    uint32_t pk[16];
    if (E4M3) {
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
            const float4 f4 = *reinterpret_cast<const float4 *>(fc + c);
            const float x0 = ex2(t[c] - ref), x1 = ex2(t[c + 1] - ref);
            const float x2 = ex2(t[c + 2] - ref), x3 = ex2(t[c + 3] - ref);
            sum[0] = fmaf(x0, f4.x, sum[0]);
            sum[1] = fmaf(x1, f4.y, sum[1]);
            sum[2] = fmaf(x2, f4.z, sum[2]);
            sum[3] = fmaf(x3, f4.w, sum[3]);
            const uint32_t u = e4m3_pair(x0, x1), v = e4m3_pair(x2, x3);
            const float2 y = e4m3_values(u), z = e4m3_values(v);
            pk[c / 4] = u | v << 16;
            pk[8 + c / 4] = e4m3_pair(x0 - y.x, x1 - y.y) | e4m3_pair(x2 - z.x, x3 - z.y) << 16;
        }
    } else {
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
            const float x0 = ex2(t[c] - ref), x1 = ex2(t[c + 1] - ref);
            sum[c & 2] += x0;
            sum[(c & 2) + 1] += x1;
            pk[c / 2] = bf16_pair(x0, x1);
        }
    }
    tmem_store16(dst, pk);
    return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

// Moves the row's reference maximum up to `top` where that is needed,
// rescaling the sum and, if there is one, the accumulator in TMEM.
template <int D, bool E4M3>
__device__ __forceinline__ void grow(Row &x, float top, bool wrote, uint32_t ot) {
    const bool up = top > x.m + (E4M3 ? kSlackE4M3 : kSlackBf16);
    if (!__any_sync(0xffffffffu, up)) return;
    const float keep = up ? ex2(x.m - top) : 1.0f;
    if (up) x.m = top;
    x.l *= keep;
    if (!wrote) return;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        float o[32];
        tmem_load32(ot + c, o);
        tmem_load_wait();
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] *= keep;
        tmem_store32(ot + c, reinterpret_cast<const uint32_t *>(o));
    }
}

// One tile of one row: this copy's NC chunks of 32 columns; the other
// copies' columns get weight zero.
template <int D, bool E4M3, bool EXTRA, int NC>
__device__ __forceinline__ void softmax_tile(const AttnArgs &a, const Segment &g, Row &x, int j0, bool whole,
                                             bool wrote, int copy, uint32_t st, uint32_t ot, const float *fa) {
    if constexpr (NC < 4) {
        float t[NC][32], top = kNegInf;
        const int c0 = copy * NC;
#pragma unroll
        for (int c = 0; c < NC; ++c) tmem_load32(st + (c0 + c) * 32, t[c]);
        tmem_load_wait();
#pragma unroll
        for (int c = 0; c < NC; ++c)
            top = fmaxf(top, scores32<E4M3, EXTRA>(a, g, x, j0, (c0 + c) * 32, whole, fa, t[c]));
        grow<D, E4M3>(x, top, wrote, ot);
        const float ref = x.m == kNegInf ? 0.0f : x.m - (E4M3 ? kLiftE4M3 : 0.0f);
        const uint32_t zero[16] = {};
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c < c0 || c >= c0 + NC) tmem_store16(st + c * 16, zero);
#pragma unroll
        for (int c = 0; c < NC; ++c)
            x.l += weights32<E4M3>(st + (c0 + c) * 16, ref, fa + 2 * kTile + (c0 + c) * 32, t[c]);
    } else {
        // Twice over the tile, so that 32 values are held at a time: t back
        // into TMEM with the maximum, then the weights.
        float top = kNegInf;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float t[32];
            tmem_load32(st + c * 32, t);
            tmem_load_wait();
            top = fmaxf(top, scores32<E4M3, EXTRA>(a, g, x, j0, c * 32, whole, fa, t));
            tmem_store32(st + c * 32, reinterpret_cast<const uint32_t *>(t));
        }
        grow<D, E4M3>(x, top, wrote, ot);
        tmem_store_wait();
        const float ref = x.m == kNegInf ? 0.0f : x.m - (E4M3 ? kLiftE4M3 : 0.0f);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float t[32];
            tmem_load32(st + c * 32, t);
            tmem_load_wait();
            x.l += weights32<E4M3>(st + c * 16, ref, fa + 2 * kTile + c * 32, t);
        }
    }
    tmem_store_wait();
}

// Adds to `cols` output columns from `col` on, at dst[(k / 4) s4 + k % 4], what
// the products left out: values that are not finite, of the positions the row
// sees in the segment's cleaned tiles.  (In a tile that was not cleaned they
// are in the sum already, and adding them again changes nothing.)
template <int D, bool E4M3>
__device__ __noinline__ void add_odd_values(const AttnArgs &a, const Segment g, const Row x, int col, int cols,
                                            float *dst, int s4) {
    const int32_t *table = g.shared ? a.shared_table : a.table + static_cast<long long>(g.b) * a.width;
    for (int t = g.t0; t < g.t1; ++t) {
        for (int j = t * kTile; j < min(g.len, (t + 1) * kTile); ++j) {
            int pj, slot;
            if (g.shared ? a.window > 0 && static_cast<long long>(x.pos_i) - j >= a.window
                         : !sees(a, x.b, x.n, x.pos_i, x.first, g.len, j, &pj))
                continue;
            const int page = page_of(a.c, table, INT_MAX, j, &slot);
            if (page < 0) continue;
            const long long at = cache_row(a.c, page, g.h, slot) * D + col;
            for (int k = 0; k < cols; ++k) {
                float y;
                if (E4M3)
                    y = (a.c.v[at + k] & 0x7f) == 0x7f ? NAN : 0.0f;
                else
                    y = __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(a.c.v)[at + k]);
                if (!isfinite(y)) dst[(k / 4) * s4 + k % 4] += y;
            }
        }
    }
}

template <int D, bool E4M3, bool EXTRA>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_kernel(const __grid_constant__ KernelArgs ka, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
    using S = Shape<D, E4M3>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const AttnArgs &a = ka.a;
    const Plan &p = ka.p;
    uint8_t *qt = smem, *ring = qt + 2 * S::kQ;
    float *scales = reinterpret_cast<float *>(ring + S::kSlots * S::kSlot);
    Shared &sh = *reinterpret_cast<Shared *>(reinterpret_cast<uint8_t *>(scales) + S::kScale);
    Barriers &bar = sh.bar;
    float *q_factor = scales + kScaleRing * 3 * kTile;  // [2][kGroupRows], e4m3
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;");

    // The cost line: the prefix's units, then each sequence's.  Thread i sums
    // a contiguous share of the sequences; a scan places them.
    const int each = ceil_div(p.B, kAttnThreads);
    const int bf = min(p.B, tid * each), bt = min(p.B, bf + each);
    const long long per = static_cast<long long>(p.Hkv) * p.rt;
    long long mine = 0;
    for (int b = bf; b < bt; ++b) {
        const Span s = span_of(p, b);
        mine += (s.t1 - s.t0) * per;
    }
    long long incl = mine;
    for (int o = 1; o < 32; o *= 2) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sh.scan[warp] = incl;
    if (tid == 0) {
        for (int i = 0; i < S::kSlots; ++i) {
            bar_init(smem_addr(&bar.full[i]), 1);
            bar_init(smem_addr(&bar.empty[i]), 1);
        }
        for (int i = 0; i < kScaleRing; ++i) {
            bar_init(smem_addr(&bar.scale_full[i]), 1);
            bar_init(smem_addr(&bar.scale_empty[i]), 8);
        }
        bar_init(smem_addr(&bar.o_full), 1);
        bar_init(smem_addr(&bar.fold), 8);
        bar_init(smem_addr(&bar.drained), 1);
        for (int w = 0; w < 2; ++w) {
            bar_init(smem_addr(&bar.q_full[w]), 1);
            bar_init(smem_addr(&bar.q_empty[w]), 9);
            bar_init(smem_addr(&bar.s_full[w]), 1);
            bar_init(smem_addr(&bar.p_full[w]), 4);
        }
        sh.dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_proxy();
    }
    if (warp == 9) tmem_alloc(smem_addr(&sh.tmem), 512);
    __syncthreads();
    const long long prefix_cost = static_cast<long long>(p.Hkv) * p.srt * p.sT;
    long long before = prefix_cost, total = prefix_cost;
    for (int w = 0; w < kAttnThreads / 32; ++w) {
        if (w < warp) before += sh.scan[w];
        total += sh.scan[w];
    }
    before += incl - mine;
    const long long share = (total + gridDim.x - 1) / gridDim.x;
    const long long from = min(total, share * blockIdx.x), to = min(total, from + share);
    if (tid == 0) {
        sh.b0 = -1;
        sh.base0 = 0;
    }
    __syncthreads();
    if (from >= prefix_cost && before <= from && from < before + mine) {
        long long at = before;
        for (int b = bf; b < bt; ++b) {
            const Span s = span_of(p, b);
            const long long c = (s.t1 - s.t0) * per;
            if (from < at + c) {
                sh.b0 = b;
                sh.base0 = at;
                break;
            }
            at += c;
        }
    }
    if (blockIdx.x == 0) {
        long long at = before;
        for (int b = bf; b < bt; ++b) {
            const Span s = span_of(p, b);
            p.base[b] = at;
            at += (s.t1 - s.t0) * per;
        }
        if (tid == 0) {
            p.base[p.B] = total;
            p.base[p.B + 1] = share;
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = sh.tmem;
    volatile int *dead = &sh.dead;
    Walk walk(p, from, to, sh.b0, sh.base0);
    Segment g;

    if (warp == 8) {
        // ---- loads: tiles in the order the products take them
        uint32_t slot = 0, phase = 1, n = 0;
        int seg = 0;
        bool live = true;
        while (live && walk.next(&g)) {
            if (lane == 0) sh.fail[seg & 15] = sh.odd[seg & 15] = 0;
            __syncwarp();
            const int32_t *table = g.shared ? a.shared_table : a.table + static_cast<long long>(g.b) * a.width;
            const int shift = a.c.page_shift, per_tile = kTile >> shift, n_tiles = g.t1 - g.t0;
            // Alternating tiles: K0 K1 V0 K2 V1 ...; both groups on each tile: K0 V0 K1 V1 ...
            int kt = 0, vt = 0;
            for (int i = 0; i < 2 * n_tiles; ++i) {
                const bool key = kt < n_tiles && (kt == vt || (!g.dual && kt == vt + 1));
                const int t = g.t0 + (key ? kt++ : vt++);
                const int pages = min(per_tile, ((g.len - t * kTile) + (1 << shift) - 1) >> shift);
                int id = -1;
                if (lane < pages) {
                    id = table[t * per_tile + lane];
                    if (id < 0 || id >= a.c.num_pages) {
                        id = -1;
                        sh.fail[seg & 15] = 1;
                        atomicOr(a.err, static_cast<uint32_t>(SPEC_DATA_PAGE_RANGE));
                    }
                }
                const int good = __popc(__ballot_sync(0xffffffffu, id >= 0));
                live = bar_wait(smem_addr(&bar.empty[slot]), phase, dead);
                live = __all_sync(0xffffffffu, live);
                if (!live) break;
                const uint32_t full = smem_addr(&bar.full[slot]);
                if (lane == 0) bar_arrive_tx(full, static_cast<uint32_t>(good * (S::kSlot >> 7) << shift));
                __syncwarp();
                if (id >= 0) {
                    const CUtensorMap *map = key ? &kmap : &vmap;
                    const uint32_t dst = smem_addr(ring + slot * S::kSlot) + ((lane << shift) * S::kRow);
#pragma unroll
                    for (int x = 0; x < S::kHalves; ++x)
                        tma_load(dst + x * S::kMat, map, full, x * 64, 0, id * a.c.Hkv + g.h);
                }
                ++n;
                if (++slot == static_cast<uint32_t>(S::kSlots)) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            ++seg;
        }
        if (!live) {  // the copies in flight land before the CTA's memory goes
            for (uint32_t i = n > static_cast<uint32_t>(S::kSlots) ? n - S::kSlots : 0; i < n; ++i)
                bar_drain(smem_addr(&bar.full[i % S::kSlots]), (i / S::kSlots) & 1);
        }
    } else if (warp == 9) {
        // ---- products
        if (lane == 0) {
            constexpr uint32_t kQk = mma_desc(E4M3, kTile, false), kPv = mma_desc(E4M3, D, true);
            constexpr uint32_t kHi = kMatrixHi<S::kRow>;
            uint32_t qn = 0, pn[2] = {0, 0};
            uint32_t slot = 0, phase = 0;  // the ring, in the order it is filled
            bool live = true;
            const uint32_t q0 = matrix_lo(smem_addr(qt), 0), k0 = matrix_lo(smem_addr(ring), 0);
            const uint32_t v0 = matrix_lo(smem_addr(ring), S::kMat);
            const uint32_t full0 = smem_addr(&bar.full[0]), empty0 = smem_addr(&bar.empty[0]);
            const uint32_t s_full = smem_addr(&bar.s_full[0]), p_full = smem_addr(&bar.p_full[0]);
            auto advance = [&] {
                if (++slot == static_cast<uint32_t>(S::kSlots)) {
                    slot = 0;
                    phase ^= 1;
                }
            };
            // S of group w from the query tile qi and the key tile in slot s
            auto scores = [&](uint32_t w, uint32_t qi, uint32_t s) {
                const uint32_t q = q0 + qi * (S::kQ >> 4), k = k0 + s * (S::kSlot >> 4), d = tmem + w * kTile;
                if (E4M3) {
#pragma unroll
                    for (int i = 0; i < 2 * (D / 32); ++i) {
                        const uint32_t half = i / (D / 32), j = i % (D / 32);
                        mma_ss<true>(d, q + ((half * S::kMat + j * 32) >> 4), kHi, k + (j * 32 >> 4), kHi, kQk, i > 0);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        const uint32_t o = ((i / 4) * S::kMat + (i % 4) * 32) >> 4;
                        mma_ss<false>(d, q + o, kHi, k + o, kHi, kQk, i > 0);
                    }
                }
            };
            // O += P V of group w with the value tile in slot s
            auto values = [&](uint32_t w, uint32_t s, bool first) {
                const uint32_t v = v0 + s * (S::kSlot >> 4), d = tmem + 2 * kTile + w * D, pt = tmem + w * kTile;
                if (E4M3) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t j = i % 4;
                        mma_ts<true>(d, pt + j * 16 + (i / 4) * 8, v + (j * 32 * S::kRow >> 4), kHi, kPv, i > 0 || !first);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mma_ts<false>(d, pt + i * 8, v + (i * 16 * S::kRow >> 4), kHi, kPv, i > 0 || !first);
                }
            };
            while (live && walk.next(&g)) {
                const int T = g.t1 - g.t0, lead = g.dual ? 1 : min(2, T);
                uint32_t qi[2];  // the groups' query tiles
                qi[0] = qi[1] = qn & 1;
                live = bar_wait(smem_addr(&bar.q_full[qn & 1]), (qn >> 1) & 1, dead);
                ++qn;
                if (g.dual) {
                    qi[1] = qn & 1;
                    live = live && bar_wait(smem_addr(&bar.q_full[qn & 1]), (qn >> 1) & 1, dead);
                    ++qn;
                }
                for (int t = 0; live && t < lead; ++t) {  // scores of each group's first tile
                    if (!(live = bar_wait(full0 + 8 * slot, phase, dead))) break;
                    fence_after_sync();
                    if (g.dual) {
                        scores(0, qi[0], slot);
                        mma_commit(s_full);
                        scores(1, qi[1], slot);
                        mma_commit(s_full + 8);
                    } else {
                        scores(t, qi[0], slot);
                        mma_commit(s_full + 8 * t);
                    }
                    mma_commit(empty0 + 8 * slot);
                    advance();
                }
                for (int t = 0; live && t < T; ++t) {
                    const uint32_t vs = slot, vp = phase;
                    advance();
                    const bool more = t + lead < T;
                    const uint32_t ks = slot, kp = phase;
                    if (more) advance();
                    if (!(live = bar_wait(full0 + 8 * vs, vp, dead))) break;
                    const uint32_t w0 = g.dual ? 0 : t & 1, w1 = g.dual ? 1 : t & 1;
                    for (uint32_t w = w0; w <= w1; ++w) {
                        if (!(live = bar_wait(p_full + 8 * w, pn[w]++ & 1, dead))) break;
                        fence_after_sync();
                        values(w, vs, g.dual ? t == 0 : t < 2);
                        if (w == w1) mma_commit(empty0 + 8 * vs);
                        if (!more) continue;
                        if (!(live = bar_wait(full0 + 8 * ks, kp, dead))) break;
                        scores(w, qi[w], ks);
                        mma_commit(s_full + 8 * w);
                        if (w == w1) mma_commit(empty0 + 8 * ks);
                    }
                }
                if (live) {
                    mma_commit(smem_addr(&bar.o_full));
                    mma_commit(smem_addr(&bar.q_empty[qi[0]]));
                    if (g.dual) mma_commit(smem_addr(&bar.q_empty[qi[1]]));
                }
            }
            if (!live) {  // products in flight end before TMEM is freed
                mma_commit(smem_addr(&bar.drained));
                bar_drain(smem_addr(&bar.drained), 0);
            }
        }
        __syncwarp();
    } else if (warp == 11) {
        // ---- query tiles, a segment ahead where the ring of two has room
        uint32_t qn = 0;
        bool live = true;
        while (live && walk.next(&g)) {
            for (int w = 0; live && w < (g.dual ? 2 : 1); ++w, ++qn) {
                const int row0 = g.row0 + w * kGroupRows, rows = min(kGroupRows, g.rows - w * kGroupRows);
                const int span = kGroupRows / copies_of(g.dual, rows);
                live = bar_wait(smem_addr(&bar.q_empty[qn & 1]), ((qn >> 1) & 1) ^ 1, dead);
                live = __all_sync(0xffffffffu, live);
                if (!live) break;
#pragma unroll 1
                for (int row = lane; row < span; row += 32) {
                    const __nv_bfloat16 *q = nullptr;
                    if (row < rows) {
                        const int r = row0 + row;
                        const long long tok = (g.shared ? 0 : static_cast<long long>(g.b) * a.N) + r / a.G;
                        q = a.q + tok * a.q_stride + static_cast<long long>(g.h * a.G + r % a.G) * D;
                    }
                    stage_query<D, E4M3>(q, qt + (qn & 1) * S::kQ, row, span, a.scale < 0.0f, q_factor + (qn & 1) * kGroupRows);
                }
                fence_async_proxy();
                __syncwarp();
                if (lane == 0) bar_arrive(smem_addr(&bar.q_full[qn & 1]));
            }
        }
    } else if (warp == 10) {
        // ---- the e4m3 exponents as factors: 2^ek, ev, 2^-ev of every position
        if (E4M3) {
            uint32_t n = 0;
            bool live = true;
            while (live && walk.next(&g)) {
                const int32_t *table = g.shared ? a.shared_table : a.table + static_cast<long long>(g.b) * a.width;
                for (int t = g.t0; t < g.t1; ++t, ++n) {
                    const int j = t * kTile + lane * 4;
                    int slot = 0;
                    const int page = j < g.len ? page_of(a.c, table, INT_MAX, j, &slot) : -1;
                    uint32_t ek = 0, ev = 0;
                    if (page >= 0) {
                        const long long row = cache_row(a.c, page, g.h, slot);
                        ek = __ldg(reinterpret_cast<const uint32_t *>(a.c.k_exp + row));
                        ev = __ldg(reinterpret_cast<const uint32_t *>(a.c.v_exp + row));
                    }
                    const uint32_t s = n % kScaleRing;
                    live = bar_wait(smem_addr(&bar.scale_empty[s]), ((n / kScaleRing) & 1) ^ 1, dead);
                    live = __all_sync(0xffffffffu, live);
                    if (!live) break;
                    float *f = scales + s * 3 * kTile + lane * 4;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int x = max(-120, min(120, static_cast<int>(static_cast<int8_t>(ek >> 8 * i))));
                        const int y = max(-120, min(120, static_cast<int>(static_cast<int8_t>(ev >> 8 * i))));
                        f[i] = exp2i(x);
                        f[kTile + i] = static_cast<float>(y);
                        f[2 * kTile + i] = exp2i(-y);
                    }
                    __syncwarp();
                    if (lane == 0) bar_arrive(smem_addr(&bar.scale_full[s]));
                }
            }
        }
    } else {
        // ---- softmax groups
        const int w = warp >> 2, quad = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(quad) << 21;  // this warp's TMEM lanes
        const uint32_t st = tmem + lanes + w * kTile, ot = tmem + lanes + 2 * kTile + w * D;
        const float mul = (a.cap > 0.0f ? fabsf(a.scale) / a.cap : fabsf(a.scale) * kLog2e);
        uint32_t segs = 0, qn = 0, sn = 0, n_ring = 0, n_scale = 0, fn = 0;
        bool live = true;
        // All eight softmax warps meet (bounded, unlike a hardware barrier).
        auto meet = [&] {
            __syncwarp();
            if (lane == 0) bar_arrive(smem_addr(&bar.fold));
            live = bar_wait(smem_addr(&bar.fold), fn++ & 1, dead);
            live = __all_sync(0xffffffffu, live);
            return live;
        };
        while (live && walk.next(&g)) {
            const int T = g.t1 - g.t0, row0 = g.row0 + (g.dual ? w * kGroupRows : 0);
            const int rows = min(kGroupRows, g.rows - (g.dual ? w * kGroupRows : 0));
            // Few rows are repeated over the 128 lanes, and each copy takes its
            // share of a tile's columns.
            const int copies = copies_of(g.dual, rows), span = kGroupRows / copies;
            const int copy = quad / (4 / copies), row = (quad * 32 + lane) & (span - 1);
            const bool has = row < rows, active = (quad * 32 & (span - 1)) < rows;
            const int r = row0 + row, tok_in = has ? r / a.G : 0, head = g.h * a.G + (has ? r % a.G : 0);
            const long long tok = g.shared ? tok_in : static_cast<long long>(g.b) * a.N + tok_in;
            const int b = g.shared ? (has ? static_cast<int>(tok / a.N) : 0) : g.b;
            const int n = has ? static_cast<int>(tok - static_cast<long long>(b) * a.N) : 0;
            Row x;
            x.b = b;
            x.n = n;
            x.tok = static_cast<int>(tok);
            const int seq_len = g.shared ? (has ? a.lens[b] : 0) : g.len;
            x.first = seq_len - a.N;
            x.pos_i = !has ? 0 : a.pos ? a.pos[tok] : a.shared_len + x.first + n;
            x.has = has;
            const uint32_t qi = (qn + (g.dual ? w : 0)) & 1, q_other = qi ^ 1;
            if (E4M3) {
                live = bar_wait(smem_addr(&bar.q_full[qi]), ((qn + (g.dual ? w : 0)) >> 1) & 1, dead);
                live = __all_sync(0xffffffffu, live);
                if (!live) break;
            }
            x.rs = mul * (E4M3 ? q_factor[qi * kGroupRows + quad * 32 + lane] : 1.0f);
            x.slope = EXTRA && a.slopes && has ? a.slopes[head] * kLog2e : 0.0f;
            x.m = kNegInf;
            x.l = 0.0f;
            const int ctx = g.shared ? g.len : max(0, x.first);  // positions every row sees (no window)
            // The unit's largest position index: every warp finds it from all the
            // unit's rows, so that both groups treat a tile alike.
            int far_most = INT_MIN;
            if (a.window > 0) {
                for (int i = lane; i < g.rows; i += 32) {
                    const long long tk = (g.row0 + i) / a.G + (g.shared ? 0 : static_cast<long long>(g.b) * a.N);
                    const int tb = static_cast<int>(tk / a.N);
                    far_most = max(far_most, a.pos ? a.pos[tk] : a.shared_len + a.lens[tb] - a.N + static_cast<int>(tk % a.N));
                }
                far_most = __reduce_max_sync(0xffffffffu, far_most);
            }
            bool wrote = false;
            for (int t = g.t0; t < g.t1; ++t) {
                const int idx = t - g.t0;
                if (!g.dual && (idx & 1) != w) continue;
                const int j0 = t * kTile;
                // Does every row see the whole tile?
                bool whole = j0 + kTile <= ctx;
                if (a.window > 0)
                    whole = whole && static_cast<long long>(far_most) - (g.shared ? 0 : a.shared_len) - j0 < a.window;
                live = bar_wait(smem_addr(&bar.s_full[w]), sn++ & 1, dead);
                const float *fa = nullptr;
                if (E4M3) {
                    const uint32_t s = (n_scale + idx) % kScaleRing;
                    live = live && bar_wait(smem_addr(&bar.scale_full[s]), ((n_scale + idx) / kScaleRing) & 1, dead);
                    fa = scales + s * 3 * kTile;
                }
                // the tile's values: slot index as the loads number them
                const uint32_t vi = n_ring + (g.dual ? 2 * idx + 1 : idx == T - 1 ? 2 * idx + 1 : 2 * idx + 2);
                if (!whole) live = live && bar_wait(smem_addr(&bar.full[vi % S::kSlots]), (vi / S::kSlots) & 1, dead);
                live = __all_sync(0xffffffffu, live);
                if (!live) break;
                fence_after_sync();
                if (active) {
                    if (copies == 4)
                        softmax_tile<D, E4M3, EXTRA, 1>(a, g, x, j0, whole, wrote, copy, st, ot, fa);
                    else if (copies == 2)
                        softmax_tile<D, E4M3, EXTRA, 2>(a, g, x, j0, whole, wrote, copy, st, ot, fa);
                    else
                        softmax_tile<D, E4M3, EXTRA, 4>(a, g, x, j0, whole, wrote, 0, st, ot, fa);
                }
                wrote = true;
                if (!whole) {
                    const int at = quad * 32 + lane;
                    if (clean_values<D, E4M3>(ring + vi % S::kSlots * S::kSlot, at, j0 + at < g.len)) sh.odd[segs & 15] = 1;
                    fence_async_proxy();
                }
                fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(smem_addr(&bar.p_full[w]));
                    if (E4M3) bar_arrive(smem_addr(&bar.scale_empty[(n_scale + idx) % kScaleRing]), g.dual ? 1 : 2);
                }
            }
            if (!live) break;
            live = bar_wait(smem_addr(&bar.o_full), segs & 1, dead);
            live = __all_sync(0xffffffffu, live);
            if (!live) break;
            fence_after_sync();
            // ---- the segment's partial result
            const int rc = g.shared ? p.src : p.rc;
            const long long part = static_cast<long long>(g.slot) * (g.shared ? p.sparts : p.parts) + (g.dual ? w : 0);
            float2 *ml = (g.shared ? p.sml : p.ml) + part * rc;
            float4 *o = (g.shared ? p.so : p.o) + part * (D / 4) * rc;
            const bool failed = reinterpret_cast<volatile int *>(sh.fail)[segs & 15] != 0;
            const bool odd = reinterpret_cast<volatile int *>(sh.odd)[segs & 15] != 0;
            const bool some = active && wrote;
            const float lift = x.m == kNegInf ? kNegInf : x.m - (E4M3 ? kLiftE4M3 : 0.0f);
            if (g.dual) {
                if (has) ml[row] = make_float2(lift, failed ? NAN : x.l);
                if (some) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float v[32];
                        tmem_load32(ot + c, v);
                        tmem_load_wait();
                        if (has) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                o[(c / 4 + k) * rc + row] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                            if (odd)
                                add_odd_values<D, E4M3>(a, g, x, c, 32, reinterpret_cast<float *>(o + (c / 4) * rc + row), 4 * rc);
                        }
                    }
                }
            } else {
                // Fold the copies and the two groups into one.  The groups' accumulators
                // of a row lie in one lane: each group joins both for half of the
                // columns; the copies meet in the query tile's memory (its products
                // are done).
                constexpr int kCols = S::kQ >= 32768 ? 32 : 16;
                float4 *buf = reinterpret_cast<float4 *>(qt + qi * S::kQ) + w * (kCols / 4) * kGroupRows;
                sh.ml[warp][lane] = make_float2(has && wrote ? lift : kNegInf, has && wrote ? x.l : 0.0f);
                if (!meet()) break;
                const int per = 4 / copies, in = quad % per;  // warps a copy, this one's place
                float M = kNegInf, L = 0.0f;
                for (int i = 0; i < 2 * copies; ++i)
                    M = fmaxf(M, sh.ml[(i / copies) * 4 + (i % copies) * per + in][lane].x);
                for (int i = 0; i < 2 * copies; ++i) {
                    const float2 y = sh.ml[(i / copies) * 4 + (i % copies) * per + in][lane];
                    L += (y.x == kNegInf ? 0.0f : ex2(y.x - M)) * y.y;
                }
                // this lane's two accumulators and their factors
                const float m0 = sh.ml[quad][lane].x, m1 = sh.ml[4 + quad][lane].x;
                const float f0 = m0 == kNegInf ? 0.0f : ex2(m0 - M), f1 = m1 == kNegInf ? 0.0f : ex2(m1 - M);
                if (w == 0 && copy == 0 && has) ml[row] = make_float2(M, failed ? NAN : L);
                const uint32_t o0 = tmem + lanes + 2 * kTile, o1 = o0 + D;
#pragma unroll 1
                for (int c = w * (D / 2); c < (w + 1) * (D / 2); c += kCols) {
                    float v[kCols], u[kCols];
                    if constexpr (kCols == 32) {
                        tmem_load32(o0 + c, v);
                        tmem_load32(o1 + c, u);
                    } else {
                        tmem_load16(o0 + c, v);
                        tmem_load16(o1 + c, u);
                    }
                    tmem_load_wait();
#pragma unroll
                    for (int k = 0; k < kCols; ++k)  // an accumulator that was not written may hold anything
                        v[k] = (f0 > 0.0f ? v[k] * f0 : 0.0f) + (f1 > 0.0f ? u[k] * f1 : 0.0f);
                    if (copies == 1) {
                        if (!has) continue;
#pragma unroll
                        for (int k = 0; k < kCols / 4; ++k)
                            o[(c / 4 + k) * rc + row] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                        if (odd)
                            add_odd_values<D, E4M3>(a, g, x, c, kCols, reinterpret_cast<float *>(o + (c / 4) * rc + row), 4 * rc);
                        continue;
                    }
#pragma unroll
                    for (int k = 0; k < kCols / 4; ++k)
                        buf[k * kGroupRows + quad * 32 + lane] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                    if (!meet()) break;
                    for (int i = quad * 32 + lane; i < span * (kCols / 4); i += kGroupRows) {
                        const int ri = i & (span - 1), k = i / span;
                        if (ri >= rows) continue;
                        float4 y = buf[k * kGroupRows + ri];
                        for (int e = 1; e < copies; ++e) {
                            const float4 z = buf[k * kGroupRows + e * span + ri];
                            y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
                        }
                        o[(c / 4 + k) * rc + ri] = y;
                    }
                    if (odd) {
                        __threadfence_block();
                        if (!meet()) break;
                        if (has && copy == 0)
                            add_odd_values<D, E4M3>(a, g, x, c, kCols, reinterpret_cast<float *>(o + (c / 4) * rc + row), 4 * rc);
                    }
                    if (!meet()) break;
                }
                if (!live) break;
            }
            if (lane == 0) {
                bar_arrive(smem_addr(&bar.q_empty[qi]));
                if (g.dual) bar_arrive(smem_addr(&bar.q_empty[q_other]));
            }
            qn += g.dual ? 2 : 1;
            fence_before_sync();
            ++segs;
            n_ring += 2 * T;
            n_scale += T;
        }
        if (!live && tid == 0) atomicOr(a.err, kStalled);
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 9) tmem_free(tmem, 512);
}

// ------------------------------------------------------------------ join

// A row's partial results of one unit, kBatch at a time: f(slots, half, row,
// count) with a slot of -1 where a share holds no whole tile of the unit.
constexpr int kBatchParts = 4;

template <typename F>
__device__ __forceinline__ void each_part(long long share, long long ubase, int T, int unit, int rows, int row, F f) {
    const bool dual = rows > kGroupRows;
    const int c = dual ? 2 : 1;
    const long long uend = ubase + static_cast<long long>(T) * c;
    int lo, hi;
    if (uend < INT_MAX) {
        lo = static_cast<int>(ubase) / static_cast<int>(share);
        hi = static_cast<int>(uend - 1) / static_cast<int>(share);
    } else {
        lo = static_cast<int>(ubase / share);
        hi = static_cast<int>((uend - 1) / share);
    }
    for (int i = lo; i <= hi; i += kBatchParts) {
        int slots[kBatchParts];
#pragma unroll
        for (int k = 0; k < kBatchParts; ++k) {
            const long long from = (i + k) * share, to = from + share;
            const long long t0 = from > ubase ? (from - ubase + c - 1) / c : 0;
            const long long t1 = min(static_cast<long long>(T), (to - ubase + c - 1) / c);
            slots[k] = i + k <= hi && t0 < t1 ? unit + i + k : -1;
        }
        f(slots, dual ? row / kGroupRows : 0, dual ? row % kGroupRows : row);
    }
}

constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ KernelArgs ka) {
    constexpr int kV = D / 32;  // float4 a thread: its warp's eighth of a row
    const AttnArgs &a = ka.a;
    const Plan &p = ka.p;
    const int chunks = ceil_div(p.R, 32);
    const int chunk = blockIdx.x % chunks, bh = blockIdx.x / chunks, b = bh / p.Hkv, h = bh % p.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = chunk * 32 + lane;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (r >= p.R) return;
    const long long share = p.base[p.B + 1];
    const int len = p.lens[b];
    const bool bad = len < 0 || len > (p.width << p.page_shift);
    const Span s = span_of(p, b);
    float M = kNegInf, L = 0.0f;
    float4 acc[kV] = {};
    auto add = [&](const float2 *ml, const float4 *o, int parts, int rc, const int *slots, int half, int row) {
        float2 x[kBatchParts];
        float4 y[kBatchParts][kV];
#pragma unroll
        for (int i = 0; i < kBatchParts; ++i) {
            const long long part = static_cast<long long>(max(slots[i], 0)) * parts + half;
            x[i] = slots[i] >= 0 ? ml[part * rc + row] : make_float2(kNegInf, 0.0f);
#pragma unroll
            for (int k = 0; k < kV; ++k)
                y[i][k] = slots[i] >= 0 ? o[(part * (D / 4) + warp * kV + k) * rc + row] : float4{};
        }
        float top = M;
#pragma unroll
        for (int i = 0; i < kBatchParts; ++i) {
            top = fmaxf(top, x[i].x);
            if (isnan(x[i].y)) L = NAN;
        }
        if (top == kNegInf) return;
        const float keep = ex2(M - top);
        M = top;
        L *= keep;
#pragma unroll
        for (int k = 0; k < kV; ++k) acc[k].x *= keep, acc[k].y *= keep, acc[k].z *= keep, acc[k].w *= keep;
#pragma unroll
        for (int i = 0; i < kBatchParts; ++i) {
            if (x[i].x == kNegInf) continue;  // nothing seen: its accumulator was not written
            const float f = ex2(x[i].x - top);
            L = fmaf(f, x[i].y, L);
#pragma unroll
            for (int k = 0; k < kV; ++k) {
                acc[k].x = fmaf(f, y[i][k].x, acc[k].x);
                acc[k].y = fmaf(f, y[i][k].y, acc[k].y);
                acc[k].z = fmaf(f, y[i][k].z, acc[k].z);
                acc[k].w = fmaf(f, y[i][k].w, acc[k].w);
            }
        }
    };
    if (p.sT > 0) {
        const int g = b * p.R + r, u = g / (2 * kGroupRows), rows = min(p.sR - u * 2 * kGroupRows, 2 * kGroupRows);
        each_part(share, static_cast<long long>(h) * p.srt * p.sT + u * 2ll * p.sT, p.sT, h * p.sru + u, rows,
                  g % (2 * kGroupRows),
                  [&](const int *slots, int half, int row) { add(p.sml, p.so, p.sparts, p.src, slots, half, row); });
    }
    if (s.t1 > s.t0) {
        const int T = s.t1 - s.t0, u = r / (2 * kGroupRows), rows = min(p.R - u * 2 * kGroupRows, 2 * kGroupRows);
        each_part(share, p.base[b] + static_cast<long long>(h) * p.rt * T + u * 2ll * T, T, bh * p.ru + u, rows,
                  r % (2 * kGroupRows),
                  [&](const int *slots, int half, int row) { add(p.ml, p.o, p.parts, p.rc, slots, half, row); });
    }
    if (bad) {
        L = NAN;
        if (lane == 0 && warp == 0) atomicOr(a.err, static_cast<uint32_t>(SPEC_DATA_PAGE_RANGE));
    }
    const int tok = b * p.N + r / p.G, head = h * p.G + r % p.G;
    const long long row = static_cast<long long>(tok) * a.Hq + head;
    // Nothing seen: L = 0 and every accumulator 0.
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    __nv_bfloat16 *out = a.out + row * D + warp * kV * 4;
#pragma unroll
    for (int k = 0; k < kV; ++k)
        reinterpret_cast<uint2 *>(out)[k] = make_uint2(bf16_pair(acc[k].x * inv, acc[k].y * inv),
                                                       bf16_pair(acc[k].z * inv, acc[k].w * inv));
    if (a.lse && warp == 0) a.lse[row] = L == 0.0f ? kNegInf : (M + log2f(L)) / kLog2e;
}

// ------------------------------------------------------------------ host

int round8(int n) { return (n + 7) / 8 * 8; }

// Fills the plan's sizes and carves its arrays; returns the bytes needed.
size_t carve_plan(Plan *p, int D, char *work) {
    p->R = p->N * p->G;
    p->rt = ceil_div(p->R, kGroupRows);
    p->ru = ceil_div(p->R, 2 * kGroupRows);
    p->sR = p->B * p->R;
    p->srt = ceil_div(p->sR, kGroupRows);
    p->sru = ceil_div(p->sR, 2 * kGroupRows);
    p->rc = min(kGroupRows, round8(p->R));
    p->src = min(kGroupRows, round8(p->sR));
    p->parts = p->R > kGroupRows ? 2 : 1;
    p->sparts = p->sR > kGroupRows ? 2 : 1;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) / 256 * 256;
        return work + at;
    };
    const size_t slots = static_cast<size_t>(p->B) * p->Hkv * p->ru + kMaxGrid;
    const size_t sslots = static_cast<size_t>(p->Hkv) * p->sru + kMaxGrid;
    p->base = reinterpret_cast<long long *>(take((p->B + 2) * sizeof(long long)));
    p->ml = reinterpret_cast<float2 *>(take(slots * p->parts * p->rc * sizeof(float2)));
    p->o = reinterpret_cast<float4 *>(take(slots * p->parts * p->rc * D * sizeof(float)));
    p->sml = reinterpret_cast<float2 *>(take(sslots * p->sparts * p->src * sizeof(float2)));
    p->so = reinterpret_cast<float4 *>(take(sslots * p->sparts * p->src * D * sizeof(float)));
    return off;
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// The cache as [num_pages * Hkv][page][D]; a box is one page's head, in
// columns of one shared-memory row.
bool make_map(CUtensorMap *map, void *data, const CacheView &c) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t esz = c.e4m3 ? 1 : 2, page = 1ull << c.page_shift, D = c.D;
    const cuuint64_t dims[3] = {D, page, static_cast<cuuint64_t>(c.num_pages) * c.Hkv};
    const cuuint64_t strides[2] = {D * esz, D * esz * page};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(c.e4m3 ? D : 64), static_cast<cuuint32_t>(page), 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    return fn(map, c.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, data, dims, strides,
              box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              c.e4m3 && c.D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool E4M3, bool EXTRA>
int launch_shape(KernelArgs &ka, cudaStream_t st) {
    using S = Shape<D, E4M3>;
    constexpr int kMaxDev = 64;
    static int done[kMaxDev];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return SPEC_ERR_CUDA;
    auto kernel = attn_kernel<D, E4M3, EXTRA>;
    if (!__atomic_load_n(&done[dev], __ATOMIC_RELAXED)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess)
            return SPEC_ERR_CUDA;
        __atomic_store_n(&done[dev], 1, __ATOMIC_RELAXED);
    }
    CUtensorMap kmap, vmap;
    if (!make_map(&kmap, ka.a.c.k, ka.a.c) || !make_map(&vmap, ka.a.c.v, ka.a.c)) return SPEC_ERR_CUDA;
    Plan &p = ka.p;
    p.grid = min(sms, kMaxGrid);
    kernel<<<p.grid, kAttnThreads, S::kBytes, st>>>(ka, kmap, vmap);
    if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.B * p.Hkv * ceil_div(p.R, 32)));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<D>, ka) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

size_t attn_work_bytes(int B, int N, int Hq, int Hkv, int D) {
    Plan p = {};
    p.B = B;
    p.N = N;
    p.G = Hq / Hkv;
    p.Hkv = Hkv;
    return carve_plan(&p, D, nullptr);
}

int launch_attn(const AttnArgs &a, cudaStream_t st) {
    KernelArgs ka = {};
    ka.a = a;
    Plan &p = ka.p;
    p.B = a.B;
    p.N = a.N;
    p.G = a.G;
    p.Hkv = a.c.Hkv;
    p.width = a.width;
    p.page_shift = a.c.page_shift;
    p.Ls = a.shared_len;
    p.lens = a.lens;
    p.pos = a.pos;
    p.window = a.window;
    carve_plan(&p, a.c.D, a.work);
    p.sT = (a.shared_len + kTile - 1) / kTile;
    const bool extra = a.cap > 0.0f || a.slopes, wide = a.c.D == 128;
    if (a.c.e4m3)
        return extra ? (wide ? launch_shape<128, true, true>(ka, st) : launch_shape<64, true, true>(ka, st))
                     : (wide ? launch_shape<128, true, false>(ka, st) : launch_shape<64, true, false>(ka, st));
    return extra ? (wide ? launch_shape<128, false, true>(ka, st) : launch_shape<64, false, true>(ka, st))
                 : (wide ? launch_shape<128, false, false>(ka, st) : launch_shape<64, false, false>(ka, st));
}

}  // namespace specv
