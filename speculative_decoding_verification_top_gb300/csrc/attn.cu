// attn.cu -- attention of a target pass's new tokens to the paged cache: the
// join of partial results, and the host side.  The work itself is in
// attn_few.cu and attn_wide.cu.
//
// For one query row (token i, query head h) over the positions j it sees:
//   t_j = log2(e) * score_j;  m = max t_j;  l = sum 2^(t_j - m);
//   out = sum 2^(t_j - m) v_j / l.
// One pass over the cache.  m, l and the output's accumulator O are running
// values; partial results (m, l, O) of the same row join as
//   M = max m;  L = sum 2^(m - M) l;  out = sum 2^(m - M) O / L.
//
// A unit of work is one key/value head of one sequence (or of the shared
// prefix) and up to 256 query rows: the N G rows (new token, query head of the
// group) that share the head's keys.  All units' tiles of 128 positions, laid
// end to end, are cut into equal shares, one per CTA of a persistent grid (the
// lengths are read on the device, so a captured call follows them).  A share's
// piece of a unit is a segment, and leaves one partial result per softmax group
// and row; the join adds them in a fixed order.

#include "attn_plan.cuh"

namespace specv {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

// The shares that a unit of `cost` from ubase on touches.
__device__ __forceinline__ void shares_of(long long share, long long ubase, long long cost, int *lo, int *hi) {
    if (ubase + cost < INT_MAX) {
        *lo = static_cast<int>(ubase) / static_cast<int>(share);
        *hi = static_cast<int>(ubase + cost - 1) / static_cast<int>(share);
    } else {
        *lo = static_cast<int>(ubase / share);
        *hi = static_cast<int>((ubase + cost - 1) / share);
    }
}

// Joins the rows of one (sequence, key/value head).  SPLIT: a block takes one
// row, its warps the shares in turn, for units cut into many shares (a long
// cache of few sequences).  Else a warp takes four rows together, so that their
// loads are in flight at once: it is bound by the latency of the chain lens,
// line, (m, l) and O.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ KernelArgs ka) {
    constexpr int kJoinRows = SPLIT ? 1 : 4;                              // rows a warp
    constexpr int kBlockRows = SPLIT ? 1 : kJoinRows * kJoinWarps;
    constexpr int kV = D / 32;  // elements a lane: a warp holds a row
    struct alignas(4 * kV) Vec {
        float x[kV];
    };
    const AttnArgs &a = ka.a;
    const Plan &p = ka.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunks = ceil_div(p.own.rows, kBlockRows);
    const int bh = blockIdx.x / chunks, b = bh / p.Hkv, h = bh - b * p.Hkv;
    const int r0 = (blockIdx.x - bh * chunks) * kBlockRows + (SPLIT ? 0 : warp * kJoinRows);
    if (r0 >= p.own.rows) return;
    const int n = min(kJoinRows, p.own.rows - r0);
    const int len = p.lens[b];  // an input: there before the grids this one follows
    const bool bad = len < 0 || len > (p.width << p.page_shift);
    const Tiles s = tiles_of(p, b);
    float M[kJoinRows], L[kJoinRows];
    Vec acc[kJoinRows] = {};
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) {
        M[i] = kNegInf;
        L[i] = 0.0f;
    }
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // Adds the rows' results of one slot: two groups, both of these rows, or each
    // of its own 128 rows.
    auto add = [&](const Units &u, int slot, const int (&row)[kJoinRows], const bool (&dual)[kJoinRows],
                   const bool (&here)[kJoinRows]) {
        float2 x[kJoinRows][2];
        Vec y[kJoinRows][2];
#pragma unroll
        for (int i = 0; i < kJoinRows; ++i)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const bool some = here[i] && (!dual[i] || w == row[i] / kGroupRows);
                const long long k = (slot * 2ll + w) * u.rc + (dual[i] ? row[i] % kGroupRows : row[i]);
                x[i][w] = some ? u.ml[k] : make_float2(kNegInf, 0.0f);
                y[i][w] = some ? *reinterpret_cast<const Vec *>(u.o + k * D + lane * kV) : Vec{};
            }
#pragma unroll
        for (int i = 0; i < kJoinRows; ++i) {
            const float top = fmaxf(M[i], fmaxf(x[i][0].x, x[i][1].x));
            if (isnan(x[i][0].y) || isnan(x[i][1].y)) L[i] = NAN;
            if (top == kNegInf) continue;
            const float keep = ex2(M[i] - top);
            M[i] = top;
            L[i] *= keep;
#pragma unroll
            for (int k = 0; k < kV; ++k) acc[i].x[k] *= keep;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (x[i][w].x == kNegInf) continue;  // nothing seen: its accumulator was not written
                const float f = ex2(x[i][w].x - top);
                L[i] = fmaf(f, x[i][w].y, L[i]);
#pragma unroll
                for (int k = 0; k < kV; ++k) acc[i].x[k] = fmaf(f, y[i][w].x[k], acc[i].x[k]);
            }
        }
    };
    // The units of `u` that hold rows first.. (of a unit line that starts at
    // line, units of T tiles): they may straddle two units.
    auto join = [&](const Units &u, long long share, long long line, int T, int slot0, int first) {
        int row[kJoinRows], unit[kJoinRows];
        bool dual[kJoinRows];
#pragma unroll
        for (int i = 0; i < kJoinRows; ++i) {
            unit[i] = (first + min(i, n - 1)) / (2 * kGroupRows);
            row[i] = (first + min(i, n - 1)) % (2 * kGroupRows);
            dual[i] = u.rows - unit[i] * 2 * kGroupRows > kGroupRows;
        }
        for (int k = unit[0]; k <= unit[kJoinRows - 1]; ++k) {
            const int c = k + 1 == u.units ? u.last : u.cost;
            const long long ubase = line + static_cast<long long>(k) * u.cost * (T + u.start);
            int lo, hi;
            shares_of(share, ubase, static_cast<long long>(T + u.start) * c, &lo, &hi);
#pragma unroll 2
            for (int i = lo + (SPLIT ? warp : 0); i <= hi; i += SPLIT ? kJoinWarps : 1) {
                int t0, t1;  // a share that holds no whole tile of the unit wrote nothing
                tiles_in(i * share, i * share + share, ubase, T, u.start, c, &t0, &t1);
                const bool written = t0 < t1;
                bool here[kJoinRows];
#pragma unroll
                for (int q = 0; q < kJoinRows; ++q) here[q] = written && unit[q] == k;
                add(u, slot0 + k + i, row, dual, here);
            }
        }
    };
    const int prefix = p.sT > 0 ? p.sT - static_cast<int>(p.share[2]) : 0;
    if (prefix > 0)
        join(p.shared, p.share[1], static_cast<long long>(h) * p.shared.head * (prefix + p.shared.start), prefix,
             h * p.shared.units, b * p.own.rows + r0);
    if (s.t1 > s.t0)
        join(p.own, p.share[0], p.base[b] + static_cast<long long>(h) * p.own.head * (s.t1 - s.t0 + p.own.start), s.t1 - s.t0,
             bh * p.own.units, r0);
    if constexpr (SPLIT) {
        __shared__ float2 ml[kJoinWarps];
        __shared__ Vec part[kJoinWarps][32];
        if (lane == 0) ml[warp] = make_float2(M[0], L[0]);
        part[warp][lane] = acc[0];
        __syncthreads();
        if (warp > 0) return;
        for (int w = 0; w < kJoinWarps; ++w) M[0] = fmaxf(M[0], ml[w].x);
        L[0] = 0.0f;
        acc[0] = Vec{};
        for (int w = 0; w < kJoinWarps; ++w) {
            const float2 x = ml[w];
            const float f = x.x == kNegInf ? 0.0f : ex2(x.x - M[0]);
            L[0] = isnan(x.y) ? NAN : fmaf(f, x.y, L[0]);
#pragma unroll
            for (int k = 0; k < kV; ++k) acc[0].x[k] = fmaf(f, part[w][lane].x[k], acc[0].x[k]);
        }
    }
    if (bad && lane == 0) atomicOr(a.err, static_cast<uint32_t>(SPEC_DATA_PAGE_RANGE));
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) {
        if (i >= n) break;
        const int r = r0 + i;
        const long long at = static_cast<long long>(b * p.N + r / p.G) * a.Hq + h * p.G + r % p.G;
        if (bad) L[i] = NAN;
        // Nothing seen: L = 0 and every accumulator 0.
        const float inv = L[i] == 0.0f ? 0.0f : 1.0f / L[i];
        uint32_t *out = reinterpret_cast<uint32_t *>(a.out + at * D) + lane * (kV / 2);
        if constexpr (kV == 4)
            *reinterpret_cast<uint2 *>(out) = make_uint2(bf16_pair(acc[i].x[0] * inv, acc[i].x[1] * inv),
                                                         bf16_pair(acc[i].x[2] * inv, acc[i].x[3] * inv));
        else
            *out = bf16_pair(acc[i].x[0] * inv, acc[i].x[1] * inv);
        if (a.lse && lane == 0) a.lse[at] = L[i] == 0.0f ? kNegInf : (M[i] + log2f(L[i])) / kLog2e;
    }
}

// ------------------------------------------------------------------ host

// What beginning a unit costs, in tiles: staging its queries, a first tile that
// waits for them, masked tiles, the partial result.  Few rows: 3 to 12 are
// within 2 %.  Many rows (16 trees of 85 nodes under a prefix of 8190 / 16 trees
// over caches of up to 7001): 5 takes 251 / 213 us, 8 224 / 212, 11 231 / 216.
// A prefix has one masked tile at most: 3 takes 218 us for 64 chains of 6 under
// 16001, 8 226.
constexpr int kStartFew = 5, kStartWide = 8, kStartPrefix = 3;

// A tile's cost in a unit of two row tiles and of one.  In bf16 one row tile is
// held up by its loads (64 KB a tile) and by one chain of softmax and products
// a group, and takes 0.9 of what two take: 4 to 3 gives 212 and 224 us on the
// trees above, 2 to 1 217 and 240.  In e4m3 3 to 2 gives 247 and 286 us on the
// trees over their own caches and under a prefix and 202 for 64 chains under one,
// 2 to 1 254, 302 and 203, 4 to 3 247, 287 and 206.
constexpr int kDualBf16 = 4, kSingleBf16 = 3, kDualE4M3 = 3, kSingleE4M3 = 2;

// Fills the plan's sizes and carves its arrays; returns the bytes needed.
size_t carve_plan(Plan *p, int D, bool e4m3, char *work) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) / 256 * 256;
        return work + at;
    };
    auto kind = [&](Units *u, int rows, int heads, bool own) {
        u->rows = rows;
        u->units = ceil_div(rows, 2 * kGroupRows);
        u->rc = min(kGroupRows, (rows + 7) / 8 * 8);
        u->few = rows <= kFewRows;
        u->cost = e4m3 ? kDualE4M3 : kDualBf16;
        const bool dual = rows - (u->units - 1) * 2 * kGroupRows > kGroupRows;
        u->last = u->few ? 1 : dual ? u->cost : e4m3 ? kSingleE4M3 : kSingleBf16;
        u->head = (u->units - 1) * u->cost + u->last;
        u->start = u->few ? kStartFew : own ? kStartWide : kStartPrefix;
        const size_t parts = (static_cast<size_t>(heads) * u->units + kMaxGrid) * 2 * u->rc;
        u->ml = reinterpret_cast<float2 *>(take(parts * sizeof(float2)));
        u->o = reinterpret_cast<float *>(take(parts * D * sizeof(float)));
    };
    kind(&p->own, p->N * p->G, p->B * p->Hkv, true);
    kind(&p->shared, p->B * p->N * p->G, p->Hkv, false);
    p->base = reinterpret_cast<long long *>(take(p->B * sizeof(long long)));
    p->share = reinterpret_cast<long long *>(take(3 * sizeof(long long)));
    return off;
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

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

template <int D>
int launch_join(const KernelArgs &ka, int grid, cudaStream_t st) {
    // Units that reach over four shares or more: 12 us with SPLIT against 25 for
    // one sequence over 131077 positions; without, 23 us against 57 for 16
    // sequences of 85 nodes (two to three shares a unit).
    const Plan &p = ka.p;
    const bool split = 4ll * p.B * p.Hkv * p.own.units <= grid && p.sT == 0;
    const dim3 blocks(static_cast<unsigned>(p.B * p.Hkv * ceil_div(p.own.rows, split ? 1 : 4 * kJoinWarps)));
    return launch_early(split ? attn_join_kernel<D, true> : attn_join_kernel<D, false>, blocks, dim3(kJoinThreads), 0, st, ka)
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}

}  // namespace

// The current device's multiprocessors, asked for once a device.
static int multiprocessors() {
    static int known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if ((n = __atomic_load_n(&known[dev], __ATOMIC_RELAXED)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    __atomic_store_n(&known[dev], n, __ATOMIC_RELAXED);
    return n;
}

size_t attn_work_bytes(int B, int N, int Hq, int Hkv, int D) {
    Plan p = {};
    p.B = B;
    p.N = N;
    p.G = Hq / Hkv;
    p.Hkv = Hkv;
    return carve_plan(&p, D, false, nullptr);
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
    p.sT = (a.shared_len + kTile - 1) / kTile;
    p.lens = a.lens;
    p.pos = a.pos;
    p.window = a.window;
    carve_plan(&p, a.c.D, a.c.e4m3, a.work);
    CUtensorMap kmap, vmap;
    const int sms = multiprocessors();
    if (sms <= 0 || !make_map(&kmap, a.c.k, a.c) || !make_map(&vmap, a.c.v, a.c)) return SPEC_ERR_CUDA;
    const int grid = min(sms, kMaxGrid);
    // One launch where both kinds of units (or the only one) go to one kernel;
    // else the prefix's wide one and, beside its tail, the sequences' few-row one.
    p.do_shared = p.sT > 0;
    p.do_own = !p.do_shared || p.shared.few == p.own.few;
    const bool few = p.do_shared ? p.shared.few : p.own.few;
    int rc = few ? launch_few(ka, grid, kmap, vmap, st) : launch_wide(ka, grid, kmap, vmap, st);
    if (rc != SPEC_OK) return rc;
    if (!p.do_own) {
        p.do_shared = 0;
        p.do_own = 1;
        ka.beside = 1;
        rc = launch_few(ka, grid, kmap, vmap, st);
        if (rc != SPEC_OK) return rc;
    }
    return a.c.D == 128 ? launch_join<128>(ka, grid, st) : launch_join<64>(ka, grid, st);
}

}  // namespace specv
