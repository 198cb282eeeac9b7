// attn_plan.cuh -- what the attention kernels (attn_wide.cu, attn_few.cu) and
// the host side (attn.cu) share: how the work is numbered and cut, and the
// steps both kernels take.  Not a public header.
#pragma once

#include "attn.cuh"
#include "tensor.cuh"

namespace specv {

constexpr int kTile = 128;        // positions a tile
constexpr int kGroupRows = 128;   // query rows a softmax group of the wide kernel
constexpr int kFewRows = 64;      // units of at most this many rows go to the few-row kernel
constexpr int kAttnThreads = 384;
constexpr int kMaxSlots = 16;
constexpr int kMaxGrid = 152;
constexpr int kSmemMax = 232448;  // bytes a CTA may have
constexpr float kLog2e = 1.4426950408889634f;

// Growth of t over the reference maximum that is let stand: a weight stays
// under 2^8.
constexpr float kSlack = 8.0f;

// The units of one kind (the prefix's, or the sequences' own).
struct Units {
    int rows;             // query rows a (sequence, head); of all sequences for the prefix
    int units;            // of 256 rows, the last of fewer
    int cost, last, head; // a tile's cost in a unit of over 128 rows, in the last unit, in all units
    int rc, few;          // rows a partial result holds; handled by the few-row kernel
    int start;            // what beginning a unit costs, in tiles
    float *o;             // [slots, 2, rc, D] partial O
    float2 *ml;           // [slots, 2, rc] partial (m, l)
};

// How the work is numbered and cut; the same arithmetic in all kernels.
struct Plan {
    int B, N, G, Hkv, width, page_shift;
    int Ls, sT;           // shared prefix: length, tiles
    Units own, shared;
    int do_own, do_shared;  // which of them this launch works on
    const int32_t *lens, *pos;
    int window;
    long long *base;      // [B] first cost of each sequence's units
    long long *share;     // [3] a CTA's share of the launch that did the own, the prefix's units; prefix_first
};

struct KernelArgs {
    AttnArgs a;
    Plan p;
    int beside;  // launched beside the tail of this call's other kernel
};

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// A sequence's tiles [t0, t1): those a row may see.
struct Tiles {
    int len, t0, t1;
};

__device__ __forceinline__ Tiles tiles_of(const Plan &p, int b) {
    Tiles s;
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

// A unit's place on the cost line: `start` tiles' worth for beginning it, then
// its tiles, each at cost c.  The share [from, to) of the line holds the
// tiles [*t0, *t1) of the unit at ubase, possibly none.
__device__ __forceinline__ void tiles_in(long long from, long long to, long long ubase, int T, int start, int c, int *t0,
                                         int *t1) {
    *t0 = from > ubase ? max(0, static_cast<int>((from - ubase + c - 1) / c) - start) : 0;
    *t1 = max(0, static_cast<int>(min(static_cast<long long>(T), (to - ubase + c - 1) / c - start)));
}

// One unit and this CTA's tiles [t0, t1) of it.
struct Segment {
    bool shared, dual;
    int b, h, row0, rows;  // rows [row0, row0 + rows) of the unit's (sequence, head)
    int t0, t1, len, slot;
};

// Walks a CTA's share [x, end) of the cost line.  A tile of a unit has
// a cost by its row tiles (1 or 2); so does the unit's start, `start` times.
// Every warp walks it by itself.
struct Walk {
    long long ubase, x, end;
    int b, h, u;          // next unit; b = -1: the shared prefix
    int prefix_first;     // the prefix's first tile that a row may see
    Tiles s;
    const Plan &p;

    __device__ Walk(const Plan &plan, long long from, long long to, int b0, long long base0, int first)
        : ubase(0), x(from), end(to), b(b0), h(0), u(0), prefix_first(first), s(), p(plan) {
        if (x >= end) {
            ubase = end;
            return;
        }
        const bool sh = b < 0;
        if (!sh) s = tiles_of(p, b);
        const Units &k = sh ? p.shared : p.own;
        const int T = (sh ? p.sT - prefix_first : s.t1 - s.t0) + k.start;
        const long long in = x - base0, head = static_cast<long long>(T) * k.head;
        if (in < INT_MAX && head < INT_MAX) {
            h = static_cast<int>(in) / static_cast<int>(head);
            u = (static_cast<int>(in) - h * static_cast<int>(head)) / (k.cost * T);
        } else {
            h = static_cast<int>(in / head);
            u = static_cast<int>((in - h * head) / (static_cast<long long>(k.cost) * T));
        }
        ubase = base0 + h * head + static_cast<long long>(u) * k.cost * T;
    }

    __device__ bool next(Segment *g) {
        while (ubase < end && b < p.B) {
            const bool sh = b < 0;
            const int T = sh ? p.sT - prefix_first : s.t1 - s.t0;
            if (T == 0) {  // a sequence, or a prefix, without tiles
                advance_sequence();
                continue;
            }
            const Units &k = sh ? p.shared : p.own;
            g->shared = sh;
            g->b = b;
            g->h = h;
            g->row0 = u * 2 * kGroupRows;
            g->rows = min(k.rows - g->row0, 2 * kGroupRows);
            g->dual = g->rows > kGroupRows;
            const int c = u + 1 == k.units ? k.last : k.cost;
            const int first = sh ? prefix_first : s.t0;
            tiles_in(x, end, ubase, T, k.start, c, &g->t0, &g->t1);
            g->len = sh ? p.Ls : s.len;
            g->slot = ((sh ? 0 : b) * p.Hkv + h) * k.units + u + static_cast<int>(blockIdx.x);
            const bool some = g->t0 < g->t1;
            g->t0 += first;
            g->t1 += first;
            ubase += static_cast<long long>(T + k.start) * c;
            if (++u == k.units) {
                u = 0;
                if (++h == p.Hkv) {
                    h = 0;
                    if (sh) {
                        b = 0;
                        s = tiles_of(p, 0);
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
        if (b < p.B) s = tiles_of(p, b);
    }
};

// Tiles a sequence's unit counts for; nothing without tiles.
__device__ __forceinline__ int cost_of(const Units &u, const Tiles &s) {
    return s.t1 > s.t0 ? s.t1 - s.t0 + u.start : 0;
}

// The start of a CTA's share, found by all its threads together.
struct Start {
    long long scan[kAttnThreads / 32];
    int least[kAttnThreads / 32];
    long long base0;
    int b0;
};

// The least position index among this thread's part of all rows, for the
// prefix's window.  A sequence whose length is out of range has none.
__device__ __forceinline__ int least_position(const Plan &p) {
    int least = INT_MAX;
    if (p.pos) {
        const int n = p.B * p.N;
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += kAttnThreads) least = min(least, p.pos[i]);
    } else {
        for (int b = threadIdx.x; b < p.B; b += kAttnThreads) {
            const int len = p.lens[b];
            if (len >= 0 && len <= (p.width << p.page_shift)) least = min(least, p.Ls + len - p.N);
        }
    }
    return least;
}

// The cost line: the prefix's units, then each sequence's.  Thread i sums a
// contiguous run of the sequences; a scan places them.  Leaves this CTA's share
// in *from, *to and where it starts in sh; CTA 0 writes the line down for the
// join.  Returns the prefix's first tile that some row's window reaches.
// Contains block barriers; `sh` may be read after the next one.
__device__ __forceinline__ int find_share(const Plan &p, Start &sh, long long *from, long long *to) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int each = p.do_own ? ceil_div(p.B, kAttnThreads) : 0;
    const int bf = min(p.B, tid * each), bt = min(p.B, bf + each);
    const long long per = static_cast<long long>(p.Hkv) * p.own.head;
    long long mine = 0;
    for (int b = bf; b < bt; ++b) {
        const Tiles s = tiles_of(p, b);
        mine += cost_of(p.own, s) * per;
    }
    long long incl = mine;
    for (int o = 1; o < 32; o *= 2) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sh.scan[warp] = incl;
    const bool trim = p.do_shared && p.window > 0;
    if (trim) {
        const int least = __reduce_min_sync(0xffffffffu, least_position(p));
        if (lane == 0) sh.least[warp] = least;
    }
    if (tid == 0) {
        sh.b0 = -1;
        sh.base0 = 0;
    }
    __syncthreads();
    int first = 0;
    if (trim) {
        int least = sh.least[0];
        for (int w = 1; w < kAttnThreads / 32; ++w) least = min(least, sh.least[w]);
        first = static_cast<int>(max(0ll, min(static_cast<long long>(p.sT), (static_cast<long long>(least) - p.window + 1) / kTile)));
    }
    const long long prefix = p.do_shared && first < p.sT
                                 ? static_cast<long long>(p.Hkv) * p.shared.head * (p.sT - first + p.shared.start)
                                 : 0;
    long long before = prefix, total = prefix;
    for (int w = 0; w < kAttnThreads / 32; ++w) {
        if (w < warp) before += sh.scan[w];
        total += sh.scan[w];
    }
    before += incl - mine;
    const int grid = static_cast<int>(gridDim.x);
    const long long share =
        total < INT_MAX - grid ? (static_cast<int>(total) + grid - 1) / grid : (total + grid - 1) / grid;
    const long long x = min(total, share * blockIdx.x);
    *from = x;
    *to = min(total, x + share);
    const bool here = x >= prefix && before <= x && x < before + mine;
    if (here || blockIdx.x == 0) {
        long long at = before;
        for (int b = bf; b < bt; ++b) {
            const Tiles s = tiles_of(p, b);
            const long long c = cost_of(p.own, s) * per;
            if (here && x >= at && x < at + c) {
                sh.b0 = b;
                sh.base0 = at;
            }
            if (blockIdx.x == 0) p.base[b] = at;
            at += c;
        }
    }
    if (blockIdx.x == 0 && tid == 0) {
        if (p.do_own) p.share[0] = share;
        if (p.do_shared) {
            p.share[1] = share;
            p.share[2] = first;
        }
    }
    return first;
}

// Bytes of the shared-memory matrices: keys, values and queries lie as rows of
// 128 bytes (64 for e4m3 heads of 64), a wider row in blocks of 64 columns.
template <int D, bool E4M3>
struct Shape {
    static constexpr int kRow = E4M3 ? D : 128;              // bytes of a matrix row
    static constexpr int kHalves = E4M3 ? 1 : D / 64;        // 64-column blocks of a bf16 matrix
    static constexpr int kMat = kTile * kRow;                // bytes of one block
    static constexpr int kSlot = kMat * kHalves;             // a key or value tile
};

// Whether token n of sequence b, at position index pos_i, sees own position j;
// *pos_j gets the position's index.
__device__ __forceinline__ bool sees(const AttnArgs &a, int b, int n, int pos_i, int first, int len, int j, int *pos_j) {
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

// The largest position index of a unit's rows: every warp finds it from all of
// them, so that both groups treat a tile alike.
__device__ __forceinline__ int last_position(const AttnArgs &a, const Segment &g) {
    int most = INT_MIN;
    for (int i = threadIdx.x & 31; i < g.rows; i += 32) {
        const long long tk = (g.row0 + i) / a.G + (g.shared ? 0 : static_cast<long long>(g.b) * a.N);
        const int tb = static_cast<int>(tk / a.N);
        most = max(most, a.pos ? a.pos[tk] : a.shared_len + a.lens[tb] - a.N + static_cast<int>(tk % a.N));
    }
    return __reduce_max_sync(0xffffffffu, most);
}

// Does every row of the unit see the whole tile from position j0 on?
__device__ __forceinline__ bool sees_whole(const AttnArgs &a, const Segment &g, int j0, int last_pos) {
    if (j0 + kTile > (g.shared ? g.len : max(0, g.len - a.N))) return false;
    return a.window == 0 || static_cast<long long>(last_pos) - (g.shared ? 0 : a.shared_len) - j0 < a.window;
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

// Two fp32 operations an instruction (sm_100 and later).
struct F2 {
    unsigned long long v;
};

__device__ __forceinline__ F2 pair_of(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ float2 parts_of(F2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
    return r;
}

__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// cap tanh(y) log2 e of n scores in place, capl = cap log2 e.  tanh(y) = 1 - 2 /
// (1 + e^2y) is good to a rounding of the cap, 2^-22 of capl: under 2^-11 for caps
// up to 1000, where weights are rounded to 2^-9.  Above, arguments under 1/4 go by
// the series y - y^3 / 3 + 2 y^5 / 15 - 17 y^7 / 315 (its next term is under 2^-21
// of y), with which 128 chains of 4 tokens take 153 us, with the plain form 121.
constexpr float kPlainCap = 1000.0f;

template <int n>
__device__ __forceinline__ void cap_scores(float *y, float cap) {
    const float capl = cap * kLog2e;
    if (cap <= kPlainCap) {
#pragma unroll
        for (int i = 0; i < n; ++i) y[i] = capl - __fdividef(2.0f * capl, 1.0f + ex2(y[i] * (2.0f * kLog2e)));
        return;
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
        const float x = y[i], x2 = x * x, far = capl - __fdividef(2.0f * capl, 1.0f + ex2(x * (2.0f * kLog2e)));
        const float near = capl * x * fmaf(x2, fmaf(x2, fmaf(x2, -17.0f / 315.0f, 2.0f / 15.0f), -1.0f / 3.0f), 1.0f);
        y[i] = fabsf(x) < 0.25f ? near : far;
    }
}

// Stages the query rows [row0, row0 + rows) of a unit as the rows of a matrix
// of `tile_rows` rows (zeros past `rows`), kQMat bytes a block, and for e4m3
// their factors 2^e: the bf16 row times 2^-e, at most 448, splits exactly into
// two e4m3 terms (4 + 4 significant bits; what falls under 2^-10 is at most
// 2^-18 of the row's maximum), the first in block 0, the second in block 1.
// `threads` threads, whole warps, call it, this one as number `me`; D / 16
// lanes share a row.
template <int D, bool E4M3>
__device__ __forceinline__ void stage_queries(const AttnArgs &a, const Segment &g, int row0, int rows, int tile_rows,
                                              uint8_t *tile, float *factor, int me, int threads) {
    constexpr int kRow = Shape<D, E4M3>::kRow, kParts = D / 16;
    constexpr int kAtOnce = 4;  // rows a thread has in flight
    const int block = tile_rows * kRow, step = threads / kParts;
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
    const int part = me % kParts;
    for (int first = me / kParts; first < tile_rows; first += kAtOnce * step) {
        uint4 u[kAtOnce][2] = {};
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int row = first + i * step;
            if (row >= min(rows, tile_rows)) continue;
            const int r = row0 + row, n = r / a.G;
            const long long tok = (g.shared ? 0 : static_cast<long long>(g.b) * a.N) + n;
            const uint4 *q = reinterpret_cast<const uint4 *>(
                a.q + tok * a.q_stride + static_cast<long long>(g.h * a.G + r - n * a.G) * D + part * 16);
            u[i][0] = __ldg(q);
            u[i][1] = __ldg(q + 1);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int row = first + i * step;
            if (row >= tile_rows) break;  // whole warps alike
            uint32_t w[8] = {u[i][0].x, u[i][0].y, u[i][0].z, u[i][0].w, u[i][1].x, u[i][1].y, u[i][1].z, u[i][1].w};
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] ^= flip;
            if (!E4M3) {
                uint8_t *at = tile + (part / 4) * block;
                *reinterpret_cast<uint4 *>(at + swizzled<kRow>(row, part % 4 * 32)) = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4 *>(at + swizzled<kRow>(row, part % 4 * 32 + 16)) =
                    make_uint4(w[4], w[5], w[6], w[7]);
                continue;
            }
            uint32_t top = 0;  // bf16 bits of max |q|
#pragma unroll
            for (int k = 0; k < 8; ++k) top = max(top, max(w[k] & 0x7fffu, w[k] >> 16 & 0x7fffu));
#pragma unroll
            for (int s = kParts / 2; s > 0; s /= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, s));
            // e: max |q| <= 448 * 2^e
            int e = static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);
            e = max(-120, min(120, e));
            const float f = exp2i(-e);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float x0 = __uint_as_float(w[2 * k] << 16) * f, x1 = __uint_as_float(w[2 * k] & 0xffff0000u) * f;
                const float x2 = __uint_as_float(w[2 * k + 1] << 16) * f,
                            x3 = __uint_as_float(w[2 * k + 1] & 0xffff0000u) * f;
                const uint32_t p = e4m3_pair(x0, x1), r = e4m3_pair(x2, x3);
                const float2 y = e4m3_values(p), z = e4m3_values(r);
                hi[k] = p | r << 16;
                lo[k] = e4m3_pair(x0 - y.x, x1 - y.y) | e4m3_pair(x2 - z.x, x3 - z.y) << 16;
            }
            const uint32_t o = swizzled<kRow>(row, part * 16);
            *reinterpret_cast<uint4 *>(tile + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(tile + block + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            // The conversion makes an infinite element a finite one: its row is NaN.
            if (part == 0) factor[row] = top >= 0x7f80u ? NAN : exp2i(e);
        }
    }
}

// Row `row` of a bf16 value tile whose positions some rows do not see: zeros where
// the position is not held (the slot has whatever was there), and zeros for
// elements that are not finite, so that an unseen one does not reach a row
// through 0 * inf.  Returns whether a held element was not finite.
template <int D>
__device__ __forceinline__ bool clean_values(uint8_t *tile, int row, bool held) {
    using S = Shape<D, false>;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        uint4 *at = reinterpret_cast<uint4 *>(tile + (i / 8) * S::kMat + swizzled<S::kRow>(row, i % 8 * 16));
        if (!held) {
            *at = make_uint4(0, 0, 0, 0);
            continue;
        }
        uint4 u = *at;
        uint32_t w[4] = {u.x, u.y, u.z, u.w};
        bool here = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t keep = ((w[k] & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) |
                                  ((w[k] & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u);
            here |= keep != 0xffffffffu;
            w[k] &= keep;
        }
        if (here) *at = make_uint4(w[0], w[1], w[2], w[3]);
        odd |= here;
    }
    return odd;
}

// Row `row` of an e4m3 value tile as bf16 values times f, a power of two, into a
// bf16 tile: exact.  (With the weights in two e4m3 terms instead, as the other
// operand of a product of bytes, those under 2^-15 of the largest were lost.)
// CLEAN: some query rows do not see all positions; as above.  AT_ONCE pieces of 16
// columns are worked on together: 4, unrolled, in the few-row kernel, whose softmax
// groups do it (64 chains of 6: 200 us, 2 in a loop 213); 2 in a loop for the wide
// kernel's helper warps, whose code then stays in the instruction cache (16 trees
// of 85 nodes: 243 us, 4 unrolled 262).
template <int D, int AT_ONCE, bool CLEAN>
__device__ __forceinline__ bool widen_row(const uint8_t *from, uint8_t *to, int row, float f, bool held) {
    using S = Shape<D, true>;
    using T = Shape<D, false>;
    constexpr int kUnroll = AT_ONCE == 4 ? D / 64 : 1;
    const F2 f2 = pair_of(f, f);
    bool odd = false;
#pragma unroll kUnroll
    for (int i0 = 0; i0 < D / 16; i0 += AT_ONCE) {
        uint4 u[AT_ONCE];
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i)
            u[i] = *reinterpret_cast<const uint4 *>(from + swizzled<S::kRow>(row, (i0 + i) * 16));
#pragma unroll
        for (int i = 0; i < AT_ONCE; ++i) {
            uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w}, y[8];
            if (CLEAN) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // 0x80 in each byte that is 0x7f or 0xff
                    const uint32_t nan = ((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                    odd |= held && nan != 0;
                    w[k] = held ? w[k] & ~((nan >> 7) * 0xffu) : 0u;
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float2 v = e4m3_values(w[k / 2] >> (k % 2 * 16) & 0xffffu);
                const float2 x = parts_of(mul2(pair_of(v.x, v.y), f2));
                y[k] = bf16_pair(x.x, x.y);
            }
            uint8_t *at = to + ((i0 + i) / 4) * T::kMat;
            *reinterpret_cast<uint4 *>(at + swizzled<T::kRow>(row, (i0 + i) % 4 * 32)) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4 *>(at + swizzled<T::kRow>(row, (i0 + i) % 4 * 32 + 16)) = make_uint4(y[4], y[5], y[6], y[7]);
        }
    }
    return odd;
}

template <int D>
__device__ __noinline__ bool widen_clean(const uint8_t *from, uint8_t *to, int row, float f, bool held) {
    return widen_row<D, 1, true>(from, to, row, f, held);
}

template <int D, int AT_ONCE>
__device__ __forceinline__ bool widen_values(const uint8_t *from, uint8_t *to, int row, float f, bool held, bool clean) {
    if (!clean) return widen_row<D, AT_ONCE, false>(from, to, row, f, true);
    // A tile in ten and fewer; a call would cost the few-row kernel registers.
    return AT_ONCE == 4 ? widen_row<D, 1, true>(from, to, row, f, held) : widen_clean<D>(from, to, row, f, held);
}

// Element `at` of the cached values where it is not finite, else anything finite.
template <bool E4M3>
__device__ __forceinline__ float odd_value(const CacheView &c, long long at) {
    if (E4M3) return (c.v[at] & 0x7f) == 0x7f ? NAN : 0.0f;
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(c.v)[at]);
}

// 2^e of a cached exponent, kept in the range the cache is written with.
__device__ __forceinline__ float power_of(int e) { return exp2i(max(-120, min(120, e))); }

__device__ __forceinline__ const int32_t *pages_of(const AttnArgs &a, const Segment &g) {
    return g.shared ? a.shared_table : a.table + static_cast<long long>(g.b) * a.width;
}

// A warp's view of the page tables for one run of tiles in order: ids are read
// 32 at a time, a lane each, with 32 more on their way, so that a tile waits
// for a table entry once a segment.
struct PageIds {
    int block, ids, ids_next;

    __device__ int entries(const AttnArgs &a, const Segment &g, int first) const {
        const int i = first + (threadIdx.x & 31), shift = a.c.page_shift;
        return i < (g.len + (1 << shift) - 1) >> shift ? pages_of(a, g)[i] : -1;
    }

    __device__ void begin(const AttnArgs &a, const Segment &g) {
        block = (g.t0 * (kTile >> a.c.page_shift)) >> 5;
        ids = entries(a, g, block * 32);
        ids_next = entries(a, g, block * 32 + 32);
    }

    // Makes the block of page `first` (a tile's first: its pages lie in one
    // block) the one held.
    __device__ void turn(const AttnArgs &a, const Segment &g, int first) {
        if (first >> 5 == block) return;
        block = first >> 5;
        ids = ids_next;
        ids_next = entries(a, g, block * 32 + 32);
    }
};

// The loads of one CTA into a ring of slots, by one warp, in the order the
// products take the tiles.
template <int D, bool E4M3, int kSlots>
struct Loader {
    using S = Shape<D, E4M3>;
    uint32_t slot = 0, phase = 1, n = 0;

    // Tile t of segment g (keys or values) into the next slot, once `empty` (if
    // given) has completed its last use: in the ring's own phase.  False when a
    // wait ran out.  *fail is set where a page id is out of range (that page's
    // rows keep what the slot had; the segment's results are failed).  `exps`, if
    // given: the ring of the tiles' key and value exponents, 2 kTile bytes a slot,
    // whose copies arrive at the same barrier (one arrival a lane).
    __device__ bool tile(const AttnArgs &a, const Segment &g, PageIds &from, int t, const CUtensorMap *map, uint32_t ring,
                         unsigned long long *full_bar, uint32_t empty, volatile int *dead, int *fail, uint32_t exps = 0) {
        const int lane = threadIdx.x & 31, shift = a.c.page_shift, first = t * (kTile >> shift);
        const int pages = min(kTile >> shift, ((g.len - t * kTile) + (1 << shift) - 1) >> shift);
        from.turn(a, g, first);
        int id = __shfl_sync(0xffffffffu, from.ids, (first + lane) & 31);
        if (lane >= pages) {
            id = -1;
        } else if (id < 0 || id >= a.c.num_pages) {
            id = -1;
            if (fail) *fail = 1;
            atomicOr(a.err, static_cast<uint32_t>(SPEC_DATA_PAGE_RANGE));
        }
        const int good = __popc(__ballot_sync(0xffffffffu, id >= 0));
        const bool live = empty == 0 || bar_wait(empty, phase, dead);
        if (!__all_sync(0xffffffffu, live)) return false;
        const uint32_t full = smem_addr(full_bar + slot);
        if (lane == 0) bar_arrive_tx(full, static_cast<uint32_t>(good * (S::kSlot >> 7) << shift));
        __syncwarp();
        if (id >= 0) {
            const uint32_t dst = ring + slot * S::kSlot + ((lane << shift) * S::kRow);
#pragma unroll
            for (int x = 0; x < S::kHalves; ++x)
                tma_load(dst + x * S::kMat, map, full, x * 64, 0, id * a.c.Hkv + g.h);
        }
        if (exps) {  // four positions a lane
            const int page = __shfl_sync(0xffffffffu, id, lane * 4 >> shift);
            const long long at = cache_row(a.c, max(page, 0), g.h, lane * 4 & ((1 << shift) - 1));
            const uint32_t dst = exps + slot * 2 * kTile + lane * 4;
            copy4(dst, a.c.k_exp + at, page >= 0);
            copy4(dst + kTile, a.c.v_exp + at, page >= 0);
            copies_arrive(full);
        }
        ++n;
        if (++slot == kSlots) {
            slot = 0;
            phase ^= 1;
        }
        return true;
    }

    // The copies in flight land before the CTA's memory goes.
    __device__ void drain(unsigned long long *full_bar) const {
        for (uint32_t i = n > kSlots ? n - kSlots : 0; i < n; ++i)
            bar_drain(smem_addr(full_bar + i % kSlots), (i / kSlots) & 1);
    }
};

int launch_wide(KernelArgs &ka, int grid, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st);
int launch_few(KernelArgs &ka, int grid, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st);

// A launch that may start before the kernel ahead of it in the stream has ended
// (each kernel here waits for that itself before it touches memory).
template <typename... Params, typename... Args>
bool launch_early(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

// Raises the kernel's shared-memory limit, once per kernel and device (`done`
// is the kernel's own).
template <typename Kernel>
bool allow_smem(Kernel kernel, int bytes, int (&done)[64]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (__atomic_load_n(&done[dev], __ATOMIC_RELAXED)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    __atomic_store_n(&done[dev], 1, __ATOMIC_RELAXED);
    return true;
}

}  // namespace specv
