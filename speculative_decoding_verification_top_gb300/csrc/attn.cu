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

// A row's partial results of one unit, kBatch at a time: f(slots, row) with a
// slot of -1 where a share holds no whole tile of the unit.
constexpr int kBatch = 4;

template <typename F>
__device__ __forceinline__ void each_slot(long long share, long long ubase, int T, bool dual, int unit, F f) {
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
    for (int i = lo; i <= hi; i += kBatch) {
        int slots[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const long long from = (i + k) * share, to = from + share;
            const long long t0 = from > ubase ? (from - ubase + c - 1) / c : 0;
            const long long t1 = min(static_cast<long long>(T), (to - ubase + c - 1) / c);
            slots[k] = i + k <= hi && t0 < t1 ? unit + i + k : -1;
        }
        f(slots);
    }
}

constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ KernelArgs ka) {
    constexpr int kV = D / 32;  // elements a lane: a warp holds a row
    struct alignas(4 * kV) Vec {
        float x[kV];
    };
    const AttnArgs &a = ka.a;
    const Plan &p = ka.p;
    const int lane = threadIdx.x & 31;
    const long long at = static_cast<long long>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
    if (at >= static_cast<long long>(p.B) * p.N * a.Hq) return;
    const int head = static_cast<int>(at % a.Hq), tok = static_cast<int>(at / a.Hq);
    const int b = tok / p.N, h = head / p.G, r = (tok - b * p.N) * p.G + head % p.G;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int len = p.lens[b];
    const bool bad = len < 0 || len > (p.width << p.page_shift);
    const Tiles s = tiles_of(p, b);
    float M = kNegInf, L = 0.0f;
    Vec acc = {};
    auto add = [&](const Units &u, int slot0, int slot1, int slot2, int slot3, bool dual, int row) {
        // Two groups' results a slot: both of this row, or each of its own 128 rows.
        const int slots[kBatch] = {slot0, slot1, slot2, slot3};
        float2 x[kBatch][2];
        Vec y[kBatch][2];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const bool here = slots[i] >= 0 && (!dual || w == row / kGroupRows);
                const long long k = (max(slots[i], 0) * 2ll + w) * u.rc + (dual ? row % kGroupRows : row);
                x[i][w] = here ? u.ml[k] : make_float2(kNegInf, 0.0f);
                y[i][w] = here ? *reinterpret_cast<const Vec *>(u.o + k * D + lane * kV) : Vec{};
            }
        float top = M;
#pragma unroll
        for (int i = 0; i < 2 * kBatch; ++i) {
            top = fmaxf(top, x[i / 2][i % 2].x);
            if (isnan(x[i / 2][i % 2].y)) L = NAN;
        }
        if (top == kNegInf) return;
        const float keep = ex2(M - top);
        M = top;
        L *= keep;
#pragma unroll
        for (int k = 0; k < kV; ++k) acc.x[k] *= keep;
#pragma unroll
        for (int i = 0; i < 2 * kBatch; ++i) {
            const float2 ml = x[i / 2][i % 2];
            if (ml.x == kNegInf) continue;  // nothing seen: its accumulator was not written
            const float f = ex2(ml.x - top);
            L = fmaf(f, ml.y, L);
#pragma unroll
            for (int k = 0; k < kV; ++k) acc.x[k] = fmaf(f, y[i / 2][i % 2].x[k], acc.x[k]);
        }
    };
    if (p.sT > 0) {
        const int g = b * p.own.rows + r, u = g / (2 * kGroupRows), row = g % (2 * kGroupRows);
        const bool dual = p.shared.rows - u * 2 * kGroupRows > kGroupRows;
        each_slot(p.share[1], static_cast<long long>(h) * p.shared.row_tiles * p.sT + u * 2ll * p.sT, p.sT, dual,
                  h * p.shared.units + u,
                  [&](const int *k) { add(p.shared, k[0], k[1], k[2], k[3], dual, row); });
    }
    if (s.t1 > s.t0) {
        const int T = s.t1 - s.t0, u = r / (2 * kGroupRows), row = r % (2 * kGroupRows);
        const bool dual = p.own.rows - u * 2 * kGroupRows > kGroupRows;
        each_slot(p.share[0], p.base[b] + static_cast<long long>(h) * p.own.row_tiles * T + u * 2ll * T, T, dual,
                  (b * p.Hkv + h) * p.own.units + u,
                  [&](const int *k) { add(p.own, k[0], k[1], k[2], k[3], dual, row); });
    }
    if (bad) {
        L = NAN;
        if (lane == 0) atomicOr(a.err, static_cast<uint32_t>(SPEC_DATA_PAGE_RANGE));
    }
    // Nothing seen: L = 0 and every accumulator 0.
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    uint32_t *out = reinterpret_cast<uint32_t *>(a.out + at * D) + lane * (kV / 2);
    if constexpr (kV == 4)
        *reinterpret_cast<uint2 *>(out) =
            make_uint2(bf16_pair(acc.x[0] * inv, acc.x[1] * inv), bf16_pair(acc.x[2] * inv, acc.x[3] * inv));
    else
        *out = bf16_pair(acc.x[0] * inv, acc.x[1] * inv);
    if (a.lse && lane == 0) a.lse[at] = L == 0.0f ? kNegInf : (M + log2f(L)) / kLog2e;
}

// ------------------------------------------------------------------ host

// Fills the plan's sizes and carves its arrays; returns the bytes needed.
size_t carve_plan(Plan *p, int D, char *work) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) / 256 * 256;
        return work + at;
    };
    auto kind = [&](Units *u, int rows, int heads) {
        u->rows = rows;
        u->row_tiles = ceil_div(rows, kGroupRows);
        u->units = ceil_div(rows, 2 * kGroupRows);
        u->rc = min(kGroupRows, (rows + 7) / 8 * 8);
        u->few = rows <= kFewRows;
        const size_t parts = (static_cast<size_t>(heads) * u->units + kMaxGrid) * 2 * u->rc;
        u->ml = reinterpret_cast<float2 *>(take(parts * sizeof(float2)));
        u->o = reinterpret_cast<float *>(take(parts * D * sizeof(float)));
    };
    kind(&p->own, p->N * p->G, p->B * p->Hkv);
    kind(&p->shared, p->B * p->N * p->G, p->Hkv);
    p->base = reinterpret_cast<long long *>(take(p->B * sizeof(long long)));
    p->share = reinterpret_cast<long long *>(take(2 * sizeof(long long)));
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
int launch_join(const KernelArgs &ka, cudaStream_t st) {
    const long long rows = static_cast<long long>(ka.p.B) * ka.p.N * ka.a.Hq;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32)));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<D>, ka) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
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
    p.sT = (a.shared_len + kTile - 1) / kTile;
    p.lens = a.lens;
    p.pos = a.pos;
    p.window = a.window;
    carve_plan(&p, a.c.D, a.work);
    CUtensorMap kmap, vmap;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        !make_map(&kmap, a.c.k, a.c) || !make_map(&vmap, a.c.v, a.c))
        return SPEC_ERR_CUDA;
    const int grid = min(sms, kMaxGrid);
    // One launch where both kinds of units (or the only one) go to one kernel;
    // else the prefix's wide one and, beside its tail, the sequences' few-row one.
    p.do_shared = p.sT > 0;
    p.do_own = !p.do_shared || p.shared.few == p.own.few;
    const bool few = p.do_shared ? p.shared.few : p.own.few;
    int rc = few ? launch_few(ka, grid, kmap, vmap, false, st) : launch_wide(ka, grid, kmap, vmap, st);
    if (rc != SPEC_OK) return rc;
    if (!p.do_own) {
        p.do_shared = 0;
        p.do_own = 1;
        rc = launch_few(ka, grid, kmap, vmap, true, st);
        if (rc != SPEC_OK) return rc;
    }
    return a.c.D == 128 ? launch_join<128>(ka, st) : launch_join<64>(ka, st);
}

}  // namespace specv
