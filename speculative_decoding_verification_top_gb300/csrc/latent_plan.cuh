// latent_plan.cuh -- how the work of the latent attention (latent.cu) is numbered
// and cut.  Not a public header.
#pragma once

#include "target.cuh"
#include "tensor.cuh"
#include "util.cuh"

namespace specv {

constexpr int kTile = 64;             // positions a tile
constexpr int kRows = 64;             // query rows a unit
constexpr int kBlock = 64 * 128;      // bytes of 64 rows of 64 columns
constexpr int kMaxThreads = 512;
constexpr int kMaxSlots = 16, kMaxRopes = 8;
constexpr int kAhead = 32;            // segments that the loads may be ahead, and more

// A unit's part of a CTA that holds its beginning but not its end: the others are
// the next groups' CTAs.
struct Head {
    int b, row0, rows, parts;  // parts: CTAs that hold some of it; 0: no such unit
};

struct LatentPlan {
    int B, N, rows, units;     // query rows and units a sequence
    int width, bands, groups;  // units taken together, bands of so many, CTA groups
    int start;                 // what beginning a band costs, in tiles
    int rc;                    // rows a partial result holds
    const int32_t *lens;
    int most;                  // positions that a table covers
    Head *head;                // [grid]
    float2 *ml;                // [grid, 2, rc] partial (m, l): of a unit begun before, of one that goes on
    float *o;                  // [grid, 2, rc, C] partial O
};

struct LatentKernelArgs {
    LatentArgs a;
    LatentPlan p;
};

// A sequence's tiles; none for a length out of range (the join fails it).
__device__ __forceinline__ int length_of(const LatentPlan &p, int b) {
    const int len = p.lens[b];
    return len < 0 || len > p.most ? 0 : len;
}

__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// A sequence's cost on the line.
__device__ __forceinline__ long long cost_of(const LatentPlan &p, int len) {
    return len == 0 ? 0 : static_cast<long long>(p.bands) * (tiles_of(len) + p.start);
}

// Where a CTA's share begins, found by all its threads together.
struct Begin {
    long long scan[kMaxThreads / 32];
    long long base, share;
    int b;
};

// Contains block barriers; `at` may be read after the next one.
template <int kThreads>
__device__ __forceinline__ void find_begin(const LatentPlan &p, Begin &at, long long *from, long long *to) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int each = (p.B + kThreads - 1) / kThreads;
    const int bf = min(p.B, tid * each), bt = min(p.B, bf + each);
    long long mine = 0;
    for (int b = bf; b < bt; ++b) mine += cost_of(p, length_of(p, b));
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) at.scan[warp] = incl;
    if (tid == 0) {
        at.b = p.B;
        at.base = 0;
    }
    __syncthreads();
    long long before = incl - mine, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += at.scan[w];
        total += at.scan[w];
    }
    const long long share = (total + p.groups - 1) / p.groups;
    const long long x = min(total, share * (blockIdx.x / static_cast<unsigned>(p.width)));
    *from = x;
    *to = min(total, x + share);
    if (tid == 0) at.share = share;
    if (before <= x && x < before + mine) {
        for (int b = bf; b < bt; ++b) {
            const long long c = cost_of(p, length_of(p, b));
            if (x >= before && x < before + c) {
                at.b = b;
                at.base = before;
            }
            before += c;
        }
    }
}

// One unit and this CTA's tiles [t0, t1) of its `tiles`.
struct Segment {
    int b, row0, rows;
    int t0, t1, tiles, len;
    int parts;  // CTAs from this one on that hold some of the unit
};

// Walks a CTA's share of the line; every warp by itself.
struct Walk {
    const LatentPlan &p;
    long long from, to, base, share;
    int b, band, len;

    __device__ Walk(const LatentPlan &plan, long long f, long long t, const Begin &at)
        : p(plan), from(f), to(t), base(at.base), share(at.share), b(at.b), band(0), len(0) {
        if (b >= p.B) return;
        len = length_of(p, b);
        const long long each = tiles_of(len) + p.start;
        band = static_cast<int>((from - base) / each);
        base += band * each;
    }

    __device__ bool next(Segment *g) {
        while (b < p.B && base < to) {
            const int T = tiles_of(len), unit = band * p.width + static_cast<int>(blockIdx.x % static_cast<unsigned>(p.width));
            const long long first = base + p.start, end = first + T;
            g->b = b;
            g->row0 = unit * kRows;
            g->rows = min(kRows, p.rows - g->row0);
            g->tiles = T;
            g->len = len;
            g->t0 = static_cast<int>(max(0ll, from - first));
            g->t1 = static_cast<int>(max(0ll, min(static_cast<long long>(T), to - first)));
            g->parts = end <= to ? 1 : 1 + static_cast<int>((end - to + share - 1) / share);
            base = end;
            if (++band == p.bands) {
                band = 0;
                do {
                    len = ++b < p.B ? length_of(p, b) : 0;
                } while (b < p.B && len == 0);
            }
            if (unit < p.units && g->t0 < g->t1) return true;
        }
        return false;
    }
};

// Do all rows of the segment see the whole tile from position j0 on?
__device__ __forceinline__ bool sees_whole(const LatentArgs &a, const Segment &g, int j0) {
    return j0 + kTile <= g.len - a.N;
}

}  // namespace specv
