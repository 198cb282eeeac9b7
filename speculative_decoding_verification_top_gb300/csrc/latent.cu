// latent.cu -- attention of a target pass's new tokens to a latent cache.
//
// For one query row (token i, head h) over the positions j it sees:
//   t_j = log2(e) scale q . (c_j, r_j);  m = max t_j;  l = sum 2^(t_j - m);
//   out = sum 2^(t_j - m) c_j / l.
// All heads read the same rows (c_j, r_j), and c_j is key and value at once: a
// tile of 64 positions is loaded once for both products.
//
// A unit is 64 of a sequence's N H query rows; its keys are up to 72 KB a tile and
// its accumulator 64 x C in fp32.  The products are laid out so that both fit:
//   S = Q K^T     M = 64 rows, N = 64 positions; Q in shared memory, for C = 512
//                 its first 256 columns in TMEM, which leaves room for 2.5 tiles
//   O^T += C^T P^T   M = 128 elements of the latent, N = 64 rows: the tile's own
//                 bytes are the first operand, its positions their rows, and an
//                 accumulator of 512 x 64 is 256 columns of TMEM
// latent_kernel      persistent, one CTA per SM; its share of the tiles segment by
//                    segment
//   4 or 8 warps     softmax, a thread per row and half a tile's positions (an
//                    accumulator of 64 rows fills 16 of a warp's 32 lanes; the
//                    load gives the other lanes its second half); the query tile;
//                    the results
//   2 warps          issue the products, S and O: each as soon as its operands are
//                    there.  (One warp for both has O wait for the loads of the S
//                    ahead of it: 3600 cycles a tile, of 2040 that the products take.)
//   3 or 5 warps     load tiles page by page (TMA), in slots of 128 columns, and the
//                    rotary part: a thread's wait, arrival and copy take 300 cycles
//                    whatever the copy's size, and one thread's nine copies a tile
//                    would be the bound
// latent_join_kernel joins the partial results of units cut between CTAs
//
// The work: a sequence's units are taken `width` at a time, by as many CTAs that go
// through its tiles together, so that a tile comes from memory once for them.  All
// (sequence, band of `width` units) lie on one line, a cost of one a tile and
// `start` for beginning; it is cut into equal shares, one per group of CTAs.  A
// unit that one share holds whole is written out at once, the others' parts (m, l,
// O) are joined in the line's order: results do not depend on timing.
//
// What bounds it.  The products of 64 query rows: 36 x 34.5 + 16 x 50 = 2040 cycles a
// tile for C = 512, 1090 for 256, 614 for 128 (64 x 64 and 128 x 64 of depth 16, both
// near what shared memory delivers).  Calls of two lengths take 1.06 to 1.13, 0.63 and
// 0.43 us a tile, 2050 to 2190, 1220 and 840 cycles, and 27, 23 and 16 us beside the
// tiles: 2.3 segments a CTA with their beginnings and ends, and the launch.  Every
// operand's bytes at 128 a cycle, 112 + 96 KiB for S and O and 80 that loads and weights
// write (C = 512), would be 2304 (1408, 832): some are read less often than that.
// For C = 128 a softmax group's own chain is as long, 1680 cycles for every second tile.
// 64 x 6 tokens of 32 heads over up to 8200 positions, 174 to 178 us (0.49 of the measured
// product rate); 16 trees of 85 nodes, 16 heads, 7001 positions, 272 to 277 us (0.49); one
// token each of 64 sequences, 16 heads, 89 us (0.75 of the copy rate).  The chains with
// C = 256 104 us (0.44), 128 72 us (0.35; one group: 128).
// Not taken: a cluster's CTAs loading a tile once for all of them (chains 312 us: a slot
// is free only when the last of them is done).  Not built: pairs of CTAs on one product.

#include "latent_plan.cuh"

namespace specv {
namespace {

struct Barriers {
    unsigned long long full[kMaxSlots], empty[kMaxSlots];     // the latent's slots
    unsigned long long r_full[kMaxRopes], r_empty[kMaxRopes]; // the rotary part's
    unsigned long long q_full, s_full[2], s_empty[2], p_full[2], pv_done[2], drained[2];
};

struct Shared {
    Barriers bar;
    Begin begin;
    uint32_t tmem;
    int dead;               // a wait ran out: nobody waits any more
    int fail[kAhead];       // per segment (mod kAhead): a page id out of range
    int odd[2];             // of the segment, by group: cleaned elements that were not finite
    float2 ml[2][kRows];    // a group's maxima and sums
    alignas(16) float row[2][kRows];  // its factors of the rows: of a rescaling, or for the results
};

template <int C>
struct Layout {
    static constexpr int kPairs = C / 128;                       // slots a tile, and accumulators of 128 elements
    static constexpr int kInTmem = C == 512 ? 4 : 0;             // 64-column blocks of Q in TMEM
    static constexpr int kInSmem = C / 64 + 1 - kInTmem;         // and in shared memory, the rotary one last
    static constexpr int kRopes = C == 512 ? 1 : C == 256 ? 4 : 7;
    static constexpr int kFixed = (kInSmem + 2 + kRopes) * kBlock + static_cast<int>((sizeof(Shared) + 127) / 128 * 128);
    static constexpr int kRoom = (kSmemMax - kFixed) / (2 * kBlock);
    static constexpr int kSlots = kRoom < kMaxSlots ? kRoom : kMaxSlots;
    static constexpr int kBytes = kFixed + kSlots * 2 * kBlock;
    // Softmax groups: each takes every kGroups-th tile, with an O^T of its own.  Under
    // 512 elements there is room for two, and the chain scores, weights, products
    // (1400 cycles a tile) is the bound with one.
    static constexpr int kGroups = C == 512 ? 1 : 2;
    static constexpr int kSoftmax = 128 * kGroups;               // their threads
    // Warps: softmax, the two that issue products, the slots' loaders, the rotary part's
    static constexpr int kScores = 4 * kGroups, kValues = kScores + 1, kLoaders = kScores + 2;
    static constexpr int kSlotLoaders = C == 512 ? 4 : 2;
    static constexpr int kThreads = 32 * (kLoaders + kSlotLoaders + 1);
    // TMEM columns: O^T from 0, two S, Q
    static constexpr int kS = 256, kQ = 384;
    static_assert(kSlots >= 2 * kPairs && kRopes <= kMaxRopes, "S of a tile is made before O of the one before");
};

constexpr int kRotary = 64;  // rotary elements of a row
constexpr int kBoxes = 4;    // pages of a tile, at most
constexpr int kGroup = 128;  // threads of a softmax group
constexpr float kLowest = -FLT_MAX;

// Hardware barriers: of a group's votes and rows (the next one of either is the
// second group's), and of all groups.
constexpr int kVoteBarrier = 1, kRowBarrier = 3, kAllBarrier = 5;

template <int kThreads>
__device__ __forceinline__ void meet(int id) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "n"(kThreads) : "memory");
}

// 32 columns of 16 lanes for lanes 0-15, and the 32 columns from `kSecond` on of
// the same 16 for lanes 16-31.
template <int kSecond>
__device__ __forceinline__ void tmem_load_halves(uint32_t addr, float *v) {
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32], %33;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr), "n"(kSecond)
        : "memory");
}

template <int kSecond>
__device__ __forceinline__ void tmem_store_halves(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x32bx2.x32.b32 [%0], %33, "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "n"(kSecond)
        : "memory");
}

// Instruction descriptor with M = 64 rows (tensor.cuh's has 128).
__host__ __device__ constexpr uint32_t mma_desc64(int n) {
    return (mma_desc(false, n, false, false) & ~(0x1fu << 24)) | (64u >> 4) << 24;
}

// Where the query row `row` of a segment lies; null past its rows.
__device__ __forceinline__ const uint4 *query_row(const LatentArgs &a, const Segment &g, int row) {
    if (row >= g.rows) return nullptr;
    const int r = g.row0 + row, n = r / a.H;
    return reinterpret_cast<const uint4 *>(a.q + (static_cast<long long>(g.b) * a.N + n) * a.q_stride +
                                           static_cast<long long>(r - n * a.H) * (a.c.C + a.c.R));
}

// The segment's query tile, zeros past its rows; the scale's sign goes into it.  A
// group lays it down, a warp 16 rows, all of its loads on their way at once (through
// registers, 20 vectors a lane in four turns, a segment's queries took 6500 cycles).
template <int C>
__device__ __forceinline__ void stage_queries(const LatentArgs &a, const Segment &g, uint8_t *tile, uint32_t tmem) {
    using L = Layout<C>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5 & 3;
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
    const uint4 *q = query_row(a, g, warp * 16 + (lane & 15));
    constexpr int kParts = L::kInSmem * 8, kTurns = kParts / 2;  // 16-byte parts of a row, turns of a warp
    const unsigned long long at = reinterpret_cast<unsigned long long>(q);
    auto place = [&](int turn, int *row, int *part) {
        const int x = turn * 32 + lane;
        *row = x / kParts;
        *part = x - *row * kParts;
        return tile + *part / 8 * kBlock + swizzled<128>(warp * 16 + *row, *part % 8 * 16);
    };
    // In TMEM, lanes 0-15 hold a row's columns from 0 on (two elements a column), 16-31
    // from 64.
    uint4 head[L::kInTmem * 4 + 1];
#pragma unroll
    for (int i = 0; i < L::kInTmem * 4; ++i) head[i] = q ? __ldg(q + (lane >> 4) * 16 + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        int row, part;
        uint8_t *to = place(i, &row, &part);
        const uint4 *from = reinterpret_cast<const uint4 *>(__shfl_sync(0xffffffffu, at, row));
        copy16(smem_addr(to), from ? from + L::kInTmem * 8 + part : reinterpret_cast<const uint4 *>(a.q), from != nullptr);
    }
    if constexpr (L::kInTmem > 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 u = head[k * 8 + i];
                w[4 * i] = u.x ^ flip;
                w[4 * i + 1] = u.y ^ flip;
                w[4 * i + 2] = u.z ^ flip;
                w[4 * i + 3] = u.w ^ flip;
            }
            tmem_store_halves<64>(tmem + L::kQ + (static_cast<uint32_t>(warp) << 21) + k * 32, w);
        }
        tmem_store_wait();
    }
    copies_wait();
    if (flip) {  // of the lane's own copies
#pragma unroll 1
        for (int i = 0; i < kTurns; ++i) {
            int row, part;
            uint4 *u = reinterpret_cast<uint4 *>(place(i, &row, &part));
            *u = make_uint4(u->x ^ flip, u->y ^ flip, u->z ^ flip, u->w ^ flip);
        }
    }
    fence_async_proxy();
    fence_before_sync();
}

// The columns of 32 from position j on that token n of sequence b sees.
__device__ __forceinline__ uint32_t seen_columns(const LatentArgs &a, const Segment &g, int n, bool has, int j) {
    const int first = g.len - a.N;
    uint32_t s = first_bits(g.len - j);
    if (!has) return 0;
    if (!a.mask) return s & first_bits(first + n + 1 - j);
    const uint8_t *at = a.mask + (static_cast<long long>(g.b) * a.N + n) * a.N + (j - first);
    uint32_t m[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        m[i] = 1;
        if (j + i >= first && j + i < g.len) m[i] = at[i];
    }
#pragma unroll
    for (int i = 0; i < 32; ++i)
        if (m[i] == 0) s &= ~(1u << i);
    return s;
}

// A row's 32 weights 2^(v mul - ref), two bf16 a word; their sum.
__device__ __forceinline__ float weights(const float (&v)[32], float mul, float ref, uint32_t (&w)[16]) {
    F2 sum[2] = {pair_of(0.0f, 0.0f), pair_of(0.0f, 0.0f)};
    const F2 mul2 = pair_of(mul, mul), ref2 = pair_of(-ref, -ref);
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        const float2 y = parts_of(fma2(pair_of(v[c], v[c + 1]), mul2, ref2));
        const float2 e = make_float2(ex2(y.x), ex2(y.y));
        sum[c / 2 & 1] = add2(sum[c / 2 & 1], pair_of(e.x, e.y));
        w[c / 2] = bf16_pair(e.x, e.y);
    }
    const float2 s = parts_of(add2(sum[0], sum[1]));
    return s.x + s.y;
}

// The same, 0 where it does not see the position.
__device__ __forceinline__ float weights(const float (&v)[32], float mul, float ref, uint32_t (&w)[16], uint32_t seen) {
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        const float2 e = make_float2(seen >> c & 1u ? ex2(fmaf(v[c], mul, -ref)) : 0.0f,
                                     seen >> (c + 1) & 1u ? ex2(fmaf(v[c + 1], mul, -ref)) : 0.0f);
        sum += e.x + e.y;
        w[c / 2] = bf16_pair(e.x, e.y);
    }
    return sum;
}

// Clears, in a tile that some rows do not see whole, the positions past the end
// and the elements that are not finite, so that neither reaches a row through
// 0 * inf; whether an element of a held position was not finite.
template <int C>
__device__ __forceinline__ bool clean_tile(uint8_t *slots, uint32_t slot0, int held) {
    using L = Layout<C>;
    bool odd = false;
    for (int i = threadIdx.x % kGroup; i < kTile * (C / 8); i += kGroup) {
        const int row = i / (C / 8), part = i - row * (C / 8);
        const uint32_t slot = (slot0 + part / 16) % L::kSlots;
        uint4 *at = reinterpret_cast<uint4 *>(slots + slot * 2 * kBlock + part / 8 % 2 * kBlock + swizzled<128>(row, part % 8 * 16));
        if (row >= held) {
            *at = make_uint4(0, 0, 0, 0);
            continue;
        }
        const uint4 u = *at;
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

// Is element d of some position that row `row` sees in the segment's cleaned tiles
// not finite?
__device__ __forceinline__ bool odd_seen(const LatentArgs &a, const Segment &g, int row, int d) {
    const int n = (g.row0 + row) / a.H, first = g.len - a.N;
    for (int t = g.t0; t < g.t1; ++t) {
        if (sees_whole(a, g, t * kTile)) continue;
        for (int j = t * kTile; j < min(g.len, (t + 1) * kTile); ++j) {
            const int c = j - first;
            if (c >= 0 && (a.mask ? a.mask[(static_cast<long long>(g.b) * a.N + n) * a.N + c] == 0 : c > n)) continue;
            const int page = a.table[static_cast<long long>(g.b) * a.width + (j >> a.c.page_shift)];
            if (page < 0 || page >= a.c.num_pages) continue;
            const long long at = (static_cast<long long>(page) << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1));
            const float x = __bfloat162float(a.c.data[at * (a.c.C + a.c.R) + d]);
            if (!isfinite(x)) return true;
        }
    }
    return false;
}

__device__ __forceinline__ void scale_rows(float (&o)[32], const float *factor) {
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(factor + k);
        o[k] *= f.x;
        o[k + 1] *= f.y;
        o[k + 2] *= f.z;
        o[k + 3] *= f.w;
    }
}

__device__ __forceinline__ void put(__nv_bfloat16 *out, float y) { *out = __float2bfloat16_rn(y); }
__device__ __forceinline__ void put(float *out, float y) { *out = y; }

// Writes this lane's element of up to 32 rows; `left` are there.
template <int C, typename T>
__device__ __forceinline__ void write_rows(T *out, const float (&o)[32], int left) {
#pragma unroll
    for (int k = 0; k < 32; ++k)
        if (k < left) put(out + k * C, o[k]);
}

// What clean_tile took from the rows' results, row 0 at `out`: a latent element that
// is not finite is part of the position's key too, so that the score is NaN or +inf,
// and the row NaN anyway, or -inf, and 0 times the element is NaN.  A thread marks the
// elements that it wrote: of groups in turn half the rows, of every fourth 32 elements.
template <int C, typename T>
__device__ __forceinline__ void mark_odd(const LatentArgs &a, const Segment g, T *out) {
    const int tid = threadIdx.x;
    for (int c = tid / kGroup; c < C / 64; c += Layout<C>::kGroups) {
        const int d = c / 2 * 128 + tid % kGroup;
        for (int row = c % 2 * 32; row < min(g.rows, c % 2 * 32 + 32); ++row)
            if (odd_seen(a, g, row, d)) put(out + row * C + d, NAN);
    }
}

template <int C>
__global__ void __launch_bounds__(Layout<C>::kThreads, 1)
    latent_kernel(const __grid_constant__ LatentKernelArgs ka, const __grid_constant__ CUtensorMap map) {
    using L = Layout<C>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const LatentArgs &a = ka.a;
    const LatentPlan &p = ka.p;
    uint8_t *qt = smem, *pt = qt + L::kInSmem * kBlock, *ropes = pt + 2 * kBlock, *slots = ropes + L::kRopes * kBlock;
    Shared &sh = *reinterpret_cast<Shared *>(slots + L::kSlots * 2 * kBlock);
    Barriers &bar = sh.bar;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < L::kSlots; ++i) {
            bar_init(smem_addr(&bar.full[i]), 1);
            bar_init(smem_addr(&bar.empty[i]), 1);
        }
        for (int i = 0; i < L::kRopes; ++i) {
            bar_init(smem_addr(&bar.r_full[i]), 1);
            bar_init(smem_addr(&bar.r_empty[i]), 1);
        }
        bar_init(smem_addr(&bar.q_full), 4);
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_addr(&bar.s_full[i]), 1);
            bar_init(smem_addr(&bar.s_empty[i]), 4);
            bar_init(smem_addr(&bar.p_full[i]), 4);
            bar_init(smem_addr(&bar.pv_done[i]), 1);
            bar_init(smem_addr(&bar.drained[i]), 1);
        }
        sh.dead = sh.odd[0] = sh.odd[1] = 0;
        for (int i = 0; i < kAhead; ++i) sh.fail[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_proxy();
    }
    if (warp == L::kScores) tmem_alloc(smem_addr(&sh.tmem), 512);
    // Up to here this may run beside the kernel before it.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    long long from, to;
    find_begin<L::kThreads>(p, sh.begin, &from, &to);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = sh.tmem;
    volatile int *dead = &sh.dead;
    Walk walk(p, from, to, sh.begin);
    Segment g;

    if (warp >= L::kLoaders) {
        // ---- loads: of each tile the rotary part and the latent, by slots in turn
        if (elect_one()) {
            const uint32_t mine = warp - L::kLoaders;
            const int box = min(kTile, 1 << a.c.page_shift), boxes = kTile / box;  // positions of a copy, copies of a tile
            uint32_t seg = 0, n = 0, uses = 0, r_uses = 0;  // segments and tiles so far; uses of the rings
            bool live = true;
            for (; live && walk.next(&g); ++seg) {
                const int32_t *table = a.table + static_cast<long long>(g.b) * a.width;
                // The queries, where they lie side by side, are asked for a tile or two
                // before the softmax warps come to them.
                const long long token = static_cast<long long>(a.H) * (C + kRotary);
                if (mine == L::kSlotLoaders && a.q_stride == token)
                    prefetch_l2(a.q + g.b * (a.N * token) + static_cast<long long>(g.row0) * (C + kRotary),
                                static_cast<uint32_t>(g.rows) * (C + kRotary) * 2);
                int next[kBoxes];
                auto fetch = [&](int t) {  // the pages of tile t; -2: none
#pragma unroll
                    for (int k = 0; k < kBoxes; ++k) {
                        const int j = t * kTile + k * box;
                        next[k] = k < boxes && t < g.t1 && j < g.len ? table[j >> a.c.page_shift] : -2;
                    }
                };
                fetch(g.t0);
                for (int t = g.t0; live && t < g.t1; ++t, ++n) {
                    int id[kBoxes];
                    uint32_t bytes = 0;
                    bool bad = false;
#pragma unroll
                    for (int k = 0; k < kBoxes; ++k) {
                        const bool in = next[k] >= 0 && next[k] < a.c.num_pages;
                        id[k] = in ? next[k] : -1;
                        bad |= !in && next[k] != -2;
                        if (in) bytes += box * 128u;
                    }
                    fetch(t + 1);
                    const int y = (t * kTile) & ((1 << a.c.page_shift) - 1);  // 0 where a tile has several pages
                    for (uint32_t i = 0; i <= L::kPairs; ++i) {  // the rotary part, then its slots
                        const bool rotary = i == 0;
                        const uint32_t use = rotary ? n : n * L::kPairs + i - 1, ring = rotary ? L::kRopes : L::kSlots;
                        if (mine != (rotary ? L::kSlotLoaders : use % L::kSlotLoaders)) continue;
                        const uint32_t slot = use % ring, full = smem_addr(rotary ? &bar.r_full[slot] : &bar.full[slot]);
                        live = bar_wait(smem_addr(rotary ? &bar.r_empty[slot] : &bar.empty[slot]), (use / ring & 1) ^ 1, dead);
                        if (!live) break;
                        (rotary ? r_uses : uses) = use + 1;
                        if (bad) {  // by one whose part of the tile is waited for
                            *reinterpret_cast<volatile int *>(&sh.fail[seg % kAhead]) = 1;
                            atomicOr(a.err, static_cast<uint32_t>(SPEC_DATA_PAGE_RANGE));
                        }
                        bar_arrive_tx(full, rotary ? bytes : 2 * bytes);
                        const uint32_t dst = smem_addr(rotary ? ropes + slot * kBlock : slots + slot * 2 * kBlock);
                        const int x = rotary ? C : static_cast<int>(i - 1) * 128;
#pragma unroll
                        for (int k = 0; k < kBoxes; ++k) {
                            if (id[k] < 0) continue;
                            tma_load(dst + k * box * 128, &map, full, x, y, id[k]);
                            if (!rotary) tma_load(dst + kBlock + k * box * 128, &map, full, x + 64, y, id[k]);
                        }
                    }
                }
            }
            if (!live) {  // the copies in flight land before the CTA's memory goes
                for (uint32_t i = uses > L::kSlots ? uses - L::kSlots : 0; i < uses; ++i)
                    if (i % L::kSlotLoaders == mine) bar_drain(smem_addr(&bar.full[i % L::kSlots]), (i / L::kSlots) & 1);
                for (uint32_t i = r_uses > L::kRopes ? r_uses - L::kRopes : 0; i < r_uses; ++i)
                    bar_drain(smem_addr(&bar.r_full[i % L::kRopes]), (i / L::kRopes) & 1);
            }
        }
        __syncwarp();
    } else if (warp == L::kScores) {
        // ---- S, rotary part first
        if (elect_one()) {
            constexpr uint32_t kQk = mma_desc64(kTile), kHi = kMatrixHi<128>;
            const uint32_t q0 = matrix_lo(smem_addr(qt), 0), r0 = matrix_lo(smem_addr(ropes), 0);
            const uint32_t k0 = matrix_lo(smem_addr(slots), 0);
            uint32_t slot = 0, phase = 0, rope = 0, r_phase = 0, segs = 0, n = 0;
            bool live = true;
            while (live && walk.next(&g)) {
                live = bar_wait(smem_addr(&bar.q_full), segs++ & 1, dead);
                for (int t = g.t0; live && t < g.t1; ++t, ++n) {
                    if (!(live = bar_wait(smem_addr(&bar.s_empty[n & 1]), (n >> 1 & 1) ^ 1, dead))) break;
                    const uint32_t d = tmem + L::kS + (n & 1) * kTile;
                    if (!(live = bar_wait(smem_addr(&bar.r_full[rope]), r_phase, dead))) break;
                    fence_after_sync();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ss<false>(d, q0 + (((L::kInSmem - 1) * kBlock + k * 32) >> 4), kHi, r0 + ((rope * kBlock + k * 32) >> 4), kHi, kQk,
                                      k > 0);
                    mma_commit(smem_addr(&bar.r_empty[rope]));
                    if (++rope == L::kRopes) rope = 0, r_phase ^= 1;
#pragma unroll
                    for (int i = 0; i < L::kPairs; ++i) {
                        if (!(live = bar_wait(smem_addr(&bar.full[slot]), phase, dead))) break;
                        fence_after_sync();
                        const uint32_t b = k0 + (slot * 2 * kBlock >> 4);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int block = 2 * i + k / 4;
                            const uint32_t bk = b + ((k / 4 * kBlock + k % 4 * 32) >> 4);
                            if (block < L::kInTmem)
                                mma_ts(d, tmem + L::kQ + block * 32 + k % 4 * 8, bk, kHi, kQk, true);
                            else
                                mma_ss<false>(d, q0 + (((block - L::kInTmem) * kBlock + k % 4 * 32) >> 4), kHi, bk, kHi, kQk, true);
                        }
                        if (++slot == L::kSlots) slot = 0, phase ^= 1;
                    }
                    if (!live) break;
                    mma_commit(smem_addr(&bar.s_full[n & 1]));
                }
            }
            if (!live) {  // products in flight end before TMEM is freed
                mma_commit(smem_addr(&bar.drained[0]));
                bar_drain(smem_addr(&bar.drained[0]), 0);
            }
        }
        __syncwarp();
    } else if (warp == L::kValues) {
        // ---- O^T
        if (elect_one()) {
            constexpr uint32_t kPv = mma_desc(false, kRows, true, false), kHi = kMatrixHi<128>;
            const uint32_t v0 = matrix_lo(smem_addr(slots), kBlock), p0 = matrix_lo(smem_addr(pt), 0);
            uint32_t slot = 0, n = 0;
            bool live = true;
            while (live && walk.next(&g)) {
                for (int t = g.t0; t < g.t1; ++t, ++n) {
                    if (!(live = bar_wait(smem_addr(&bar.p_full[n & 1]), n >> 1 & 1, dead))) break;
                    fence_after_sync();
                    const uint32_t pn = p0 + ((n & 1) * kBlock >> 4), d = tmem + n % L::kGroups * (L::kPairs * kRows);
                    const bool more = t - L::kGroups >= g.t0;  // the accumulator holds some of the segment
#pragma unroll
                    for (int i = 0; i < L::kPairs; ++i) {
                        const uint32_t v = v0 + (slot * 2 * kBlock >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_ss<false>(d + i * kRows, v + (k * 16 * 128 >> 4), kHi, pn + (k * 32 >> 4), kHi, kPv, more || k > 0);
                        mma_commit(smem_addr(&bar.empty[slot]));
                        if (++slot == L::kSlots) slot = 0;
                    }
                    mma_commit(smem_addr(&bar.pv_done[n & 1]));
                }
            }
            if (!live) {
                mma_commit(smem_addr(&bar.drained[1]));
                bar_drain(smem_addr(&bar.drained[1]), 0);
            }
        }
        __syncwarp();
    } else {
        // ---- softmax
        const uint32_t group = warp >> 2;
        const int quarter = warp & 3;
        const uint32_t lanes = static_cast<uint32_t>(quarter) << 21, acc = tmem + lanes + group * (L::kPairs * kRows);
        const int row = quarter * 16 + (lane & 15), half = lane >> 4;
        const float mul = fabsf(a.scale) * kLog2e;
        uint32_t n0 = 0, seg = 0;  // tiles before the segment, segments so far
        bool ok = true;
        if (tid == 0) p.head[blockIdx.x].parts = 0;
        // Once a wait ran out nobody waits, and all go through the rest as it is: the
        // hardware barriers have no bound, so that all must come to each.
        auto waited = [&](uint32_t b, uint32_t parity) {
            if (ok) ok = bar_try(b, parity) || (*dead == 0 && bar_wait_on(b, parity, dead));
            ok = __all_sync(0xffffffffu, ok);
        };
        // The next segment's queries are laid down once the last scores are made, by the
        // group that saw them, so that its first ones are made while this one's results
        // are written.
        Segment ahead;
        auto more = [&](bool stage) {
            if (!walk.next(&ahead)) return false;
            if (stage) {
                stage_queries<C>(a, ahead, qt, tmem);
                __syncwarp();
                if (lane == 0) bar_arrive(smem_addr(&bar.q_full));
            }
            return true;
        };
        for (bool some = more(group == 0); some; ++seg) {
            g = ahead;
            const bool has = row < g.rows;
            const int token = has ? (g.row0 + row) / a.H : 0;
            float m = kNegInf, l = 0.0f;
            const uint32_t end = n0 + (g.t1 - g.t0), skip = (group - n0) % L::kGroups;  // this group's first tile
            int t = g.t0 + skip;
            for (uint32_t n = n0 + skip; n < end; n += L::kGroups, t += L::kGroups) {
                const bool later = t - L::kGroups >= g.t0;  // not this group's first of the segment
                const int j0 = t * kTile + half * 32;
                const bool whole = sees_whole(a, g, t * kTile);
                uint32_t seen = ~0u;
                if (!whole) seen = seen_columns(a, g, token, has, j0);
                waited(smem_addr(&bar.s_full[n & 1]), (n >> 1) & 1);
                fence_after_sync();
                float v[32];
                tmem_load_halves<32>(tmem + lanes + L::kS + (n & 1) * kTile, v);
                tmem_load_wait();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) bar_arrive(smem_addr(&bar.s_empty[n & 1]));
                // A row that sees any position has a maximum above -inf, so that one whose
                // scores are all -inf is told from one that sees nothing: its sum is 0, its
                // accumulators 0, or NaN, and 0 / 0 its result.
                float top[2] = {kNegInf, kNegInf};
                if (whole) {
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        top[0] = max3(top[0], v[c], v[c + 1]);
                        top[1] = max3(top[1], v[c + 2], v[c + 3]);
                    }
                    top[0] = fmaxf(fmaxf(top[0], top[1]) * mul, kLowest);
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float y = v[c] * mul;
                        if (seen >> c & 1u) top[c & 1] = fmaxf(top[c & 1], y);
                    }
                    top[0] = fmaxf(fmaxf(top[0], top[1]), seen ? kLowest : kNegInf);
                }
                const float most = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], 16));
                const bool up = most > m + kSlack;
                if (any_of(kVoteBarrier + group, kGroup, up)) {
                    // Some row's reference moves up: its sum and its column of O^T are rescaled.
                    const float keep = up ? ex2(m - most) : 1.0f;
                    if (up) m = most;
                    l *= keep;
                    if (later) {
                        const uint32_t before = n - L::kGroups;
                        waited(smem_addr(&bar.pv_done[before & 1]), before >> 1 & 1);
                        fence_after_sync();
                        if (half == 0) sh.row[group][row] = keep;
                        meet<kGroup>(kRowBarrier + group);
#pragma unroll 1
                        for (int c = 0; c < L::kPairs * kRows; c += 32) {
                            float o[32];
                            tmem_load32(acc + c, o);
                            tmem_load_wait();
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] *= sh.row[group][c % kRows + k];
                            tmem_store32(acc + c, reinterpret_cast<const uint32_t *>(o));
                        }
                        tmem_store_wait();
                        meet<kGroup>(kRowBarrier + group);
                    }
                }
                const float ref = m == kNegInf ? 0.0f : m;
                uint32_t w[16];
                if (whole)
                    l += weights(v, mul, ref, w);
                else
                    l += weights(v, mul, ref, w, seen);
                waited(smem_addr(&bar.pv_done[n & 1]), (n >> 1 & 1) ^ 1);  // of two tiles before
                if (!whole && ok) {  // the products of S are done with the tile
                    const uint32_t fill = n * L::kPairs;
                    for (uint32_t i = fill; i < fill + L::kPairs; ++i)
                        waited(smem_addr(&bar.full[i % L::kSlots]), (i / L::kSlots) & 1);
                    if (clean_tile<C>(slots, fill % L::kSlots, g.len - t * kTile)) sh.odd[group] = 1;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4 *>(pt + (n & 1) * kBlock + swizzled<128>(row, half * 64 + i * 16)) =
                        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                fence_async_proxy();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) bar_arrive(smem_addr(&bar.p_full[n & 1]));
            }
            some = more((end - 1) % L::kGroups == group);
            // This group's last tile; none where the segment's one tile was the other's.
            const uint32_t last = (end - 1) % L::kGroups == group ? end - 1 : end - 2;
            const bool any = static_cast<int>(last - n0) >= 0;
            if (any) waited(smem_addr(&bar.pv_done[last & 1]), last >> 1 & 1);
            fence_after_sync();
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            if (half == 0) sh.ml[group][row] = make_float2(m, l);
            fence_before_sync();
            meet<L::kSoftmax>(kAllBarrier);
            fence_after_sync();
            // All are past the segment's tiles: what they and the loads noted is there.
            const bool failed = *reinterpret_cast<volatile int *>(&sh.fail[seg % kAhead]) != 0;
            bool odd = false;
            float most = kNegInf, sum = 0.0f;
#pragma unroll
            for (int i = 0; i < L::kGroups; ++i) {
                odd |= *reinterpret_cast<volatile int *>(&sh.odd[i]) != 0;
                most = fmaxf(most, sh.ml[i][row].x);
            }
            const float ref = most == kNegInf ? 0.0f : most;
#pragma unroll
            for (int i = 0; i < L::kGroups; ++i) sum += sh.ml[i][row].y * ex2(sh.ml[i][row].x - ref);
            if (failed) sum = NAN;
            const bool alone = g.t0 == 0 && g.t1 == g.tiles;
            const int part = 2 * static_cast<int>(blockIdx.x) + (g.t0 == 0 ? 1 : 0);
            if (half == 0) {
                const float whole = !alone ? 1.0f : most == kNegInf && !failed ? 0.0f : 1.0f / sum;
                sh.row[group][row] = whole * ex2(m - ref);
                const long long at = static_cast<long long>(g.b) * a.N * a.H + g.row0 + row;
                if (group == 0 && alone && a.lse && has) a.lse[at] = sum == 0.0f ? kNegInf : (most + log2f(sum)) / kLog2e;
                if (group == 0 && !alone && has) p.ml[part * p.rc + row] = make_float2(most, sum);
            }
            if (tid == 0 && !alone && g.t0 == 0) p.head[blockIdx.x] = {g.b, g.row0, g.rows, g.parts};
            meet<L::kSoftmax>(kAllBarrier);
            // ---- the rows' results: a lane holds an element, of each row in turn
            const long long first = alone ? static_cast<long long>(g.b) * a.N * a.H + g.row0 : static_cast<long long>(part) * p.rc;
            const bool both = L::kGroups == 2 && g.t1 - g.t0 > 1;
            const int of = L::kGroups == 2 ? static_cast<int>(n0 & 1) : 0;  // the group of the first tile
#pragma unroll 1
            for (int c = group; c < L::kPairs * 2; c += L::kGroups) {
                const int r0 = c % 2 * 32, d = c / 2 * 128 + quarter * 32 + lane;
                if (r0 >= g.rows) continue;
                float o[32];
                tmem_load32(tmem + lanes + of * (L::kPairs * kRows) + c * 32, o);
                tmem_load_wait();
                scale_rows(o, sh.row[of] + r0);
                if (both) {
                    float x[32];
                    tmem_load32(tmem + lanes + (of ^ 1) * (L::kPairs * kRows) + c * 32, x);
                    tmem_load_wait();
                    scale_rows(x, sh.row[of ^ 1] + r0);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] += x[k];
                }
                if (alone)
                    write_rows<C>(a.out + (first + r0) * C + d, o, g.rows - r0);
                else
                    write_rows<C>(p.o + (first + r0) * C + d, o, g.rows - r0);
            }
            if (odd) {
                if (alone)
                    mark_odd<C>(a, g, a.out + first * C);
                else
                    mark_odd<C>(a, g, p.o + first * C);
            }
            fence_before_sync();
            meet<L::kSoftmax>(kAllBarrier);
            // Before this thread's next vote, after which its group may set it again.
            if (tid % kGroup == 0) sh.odd[group] = 0;
            if (tid == 0) sh.fail[seg % kAhead] = 0;
            n0 = end;
        }
        if (!ok && lane == 0) atomicOr(a.err, static_cast<uint32_t>(SPEC_DATA_STALL));
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == L::kScores) tmem_free(tmem, 512);
}

constexpr int kJoinThreads = 256;
static_assert(kMaxGrid <= kJoinThreads, "a thread per head");
constexpr int kJoinWarps = kJoinThreads / 32;

// A row's running result: a lane holds C / 32 elements, four at a time.
template <int C>
struct Running {
    float m = kNegInf, l = 0.0f;
    float4 o[C / 128] = {};

    __device__ void add(float2 ml, const float4 (&y)[C / 128]) {
        if (isnan(ml.y)) l = NAN;
        const float top = fmaxf(m, ml.x);
        if (top == kNegInf) return;  // nothing seen: the part's accumulators are 0
        const float keep = ex2(m - top), f = ml.x == kNegInf ? 0.0f : ex2(ml.x - top);
        m = top;
        l = fmaf(f, ml.y, l * keep);
#pragma unroll
        for (int i = 0; i < C / 128; ++i) {
            o[i].x = fmaf(f, y[i].x, o[i].x * keep);
            o[i].y = fmaf(f, y[i].y, o[i].y * keep);
            o[i].z = fmaf(f, y[i].z, o[i].z * keep);
            o[i].w = fmaf(f, y[i].w, o[i].w * keep);
        }
    }
};

// Blocks [0, joins): the rows of units cut between CTAs, a warp a row, or (SPLIT) a
// block 128 elements of a row, its warps the parts in turn, for units cut into many
// (a token over 2049 positions, 33 parts: 8 us in blocks of a row for every CTA).
// The other blocks: sequences without positions, and those whose length is out of range.
template <int C, bool SPLIT>
__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(const __grid_constant__ LatentKernelArgs ka, int joins) {
    constexpr int kWidth = SPLIT ? 128 : C, kV = kWidth / 128;
    const LatentArgs &a = ka.a;
    const LatentPlan &p = ka.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (static_cast<int>(blockIdx.x) >= joins) {
        for (int b = blockIdx.x - joins; b < p.B; b += gridDim.x - joins) {
            const int len = a.lens[b];
            if (len > 0 && len <= p.most) continue;
            const uint32_t fill = len == 0 ? 0u : 0x7fff7fffu;  // NaN
            uint32_t *out = reinterpret_cast<uint32_t *>(a.out + static_cast<long long>(b) * p.rows * C);
            for (int i = threadIdx.x; i < p.rows * (C / 2); i += kJoinThreads) out[i] = fill;
            if (a.lse)
                for (int i = threadIdx.x; i < p.rows; i += kJoinThreads)
                    a.lse[static_cast<long long>(b) * p.rows + i] = len == 0 ? kNegInf : NAN;
            if (len != 0 && threadIdx.x == 0) atomicOr(a.err, static_cast<uint32_t>(SPEC_DATA_PAGE_RANGE));
        }
        return;
    }
    constexpr int kBlockRows = SPLIT ? 1 : kJoinWarps;
    const int chunks = p.rc / kBlockRows, chunk = blockIdx.x / (C / kWidth);
    const int first = (blockIdx.x - chunk * (C / kWidth)) * kWidth + lane * 4;  // this lane's first element
    const int row = chunk % chunks * kBlockRows + (SPLIT ? 0 : warp);
    int cta = chunk / chunks;
    if constexpr (SPLIT) {  // a unit's number so far: its head is looked up (a block for every CTA's would be thousands)
        __shared__ int found;
        const int unit = cta, b = unit / p.units, row0 = (unit - b * p.units) * kRows;
        if (threadIdx.x == 0) found = -1;
        __syncthreads();
        if (threadIdx.x < static_cast<unsigned>(p.groups * p.width)) {
            const Head h = p.head[threadIdx.x];
            if (h.parts > 0 && h.b == b && h.row0 == row0) found = threadIdx.x;
        }
        __syncthreads();
        if ((cta = found) < 0) return;
    }
    const Head h = p.head[cta];
    if (h.parts == 0 || row >= h.rows) return;
    Running<kWidth> x;
#pragma unroll 4
    for (int i = SPLIT ? warp : 0; i < h.parts; i += SPLIT ? kJoinWarps : 1) {
        const long long at = (2ll * (cta + i * p.width) + (i == 0 ? 1 : 0)) * p.rc + row;
        const float2 ml = p.ml[at];
        float4 y[kV];
#pragma unroll
        for (int k = 0; k < kV; ++k) y[k] = *reinterpret_cast<const float4 *>(p.o + at * C + k * 128 + first);
        x.add(ml, y);
    }
    if constexpr (SPLIT) {
        __shared__ float2 ml[kJoinWarps];
        __shared__ float4 part[kJoinWarps][32][kV];
        if (lane == 0) ml[warp] = make_float2(x.m, x.l);
#pragma unroll
        for (int k = 0; k < kV; ++k) part[warp][lane][k] = x.o[k];
        __syncthreads();
        if (warp > 0) return;
        for (int w = 1; w < kJoinWarps; ++w) x.add(ml[w], part[w][lane]);
    }
    const long long at = static_cast<long long>(h.b) * p.rows + h.row0 + row;
    const float inv = x.m == kNegInf && !isnan(x.l) ? 0.0f : 1.0f / x.l;  // nothing seen: 0
#pragma unroll
    for (int k = 0; k < kV; ++k)
        *reinterpret_cast<uint2 *>(a.out + at * C + k * 128 + first) =
            make_uint2(bf16_pair(x.o[k].x * inv, x.o[k].y * inv), bf16_pair(x.o[k].z * inv, x.o[k].w * inv));
    if (a.lse && first == 0) a.lse[at] = x.l == 0.0f ? kNegInf : (x.m + log2f(x.l)) / kLog2e;
}

// ------------------------------------------------------------------ host

// What beginning a band costs, in tiles: its first queries, scores and products one
// after the other, and its results (of 4, 8, 12 and 18 the best).
constexpr int start_of(int C) { return C == 512 ? 8 : 12; }

// Fills the plan's sizes and carves its arrays; returns the bytes needed.
size_t carve_plan(LatentPlan *p, int N, int H, int C, char *work) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) / 256 * 256;
        return work + at;
    };
    p->N = N;
    p->rows = N * H;
    p->units = (p->rows + kRows - 1) / kRows;
    p->start = start_of(C);
    p->rc = p->rows < kRows ? (p->rows + 7) / 8 * 8 : kRows;
    const size_t parts = 2 * kMaxGrid * static_cast<size_t>(p->rc);
    p->head = reinterpret_cast<Head *>(take(kMaxGrid * sizeof(Head)));
    p->ml = reinterpret_cast<float2 *>(take(parts * sizeof(float2)));
    p->o = reinterpret_cast<float *>(take(parts * C * sizeof(float)));
    return off;
}

// How many units go through a sequence's tiles together.  Taken one by one, each
// reads the tiles for itself (1.03 times as long for 22 units, 1.2 for three); taken
// together, a last band of fewer units and CTAs left over idle (three units by twos
// leave a quarter idle: 257 us of 184).
void choose_width(LatentPlan *p, int grid) {
    double best = 0.0;
    for (int w = 1; w <= 8 && w <= p->units && w <= grid; ++w) {
        const int bands = (p->units + w - 1) / w, groups = grid / w;
        const double busy = static_cast<double>(p->units) / (bands * w) * (groups * w) / grid;
        const double score = w == 1 ? busy / 1.2 : busy;
        if (score < best) continue;
        best = score;
        p->width = w;
        p->bands = bands;
        p->groups = groups;
    }
}

// The cache as [num_pages][page][C + R]; a box is up to 64 positions of 64 columns.
bool make_map(CUtensorMap *map, const LatentView &c) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t page = 1ull << c.page_shift, W = c.C + c.R;
    const cuuint64_t dims[3] = {W, page, static_cast<cuuint64_t>(c.num_pages)};
    const cuuint64_t strides[2] = {W * 2, W * 2 * page};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(page < kTile ? page : kTile), 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, c.data, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int C>
int launch_shape(const LatentKernelArgs &ka, const CUtensorMap &map, cudaStream_t st) {
    static int done[64];
    const LatentPlan &p = ka.p;
    const int grid = p.groups * p.width;
    if (!allow_smem(latent_kernel<C>, Layout<C>::kBytes, done)) return SPEC_ERR_CUDA;
    if (!launch_early(latent_kernel<C>, dim3(grid), dim3(Layout<C>::kThreads), Layout<C>::kBytes, st, ka, map)) return SPEC_ERR_CUDA;
    // Bands over four groups and more each: few rows, many parts.
    const bool split = 4ll * p.B * p.bands <= p.groups;
    const int joins = split ? p.B * p.units * p.rc * (C / 128) : grid * (p.rc / kJoinWarps), fills = p.B < 152 ? p.B : 152;
    return launch_early(split ? latent_join_kernel<C, true> : latent_join_kernel<C, false>, dim3(joins + fills), dim3(kJoinThreads), 0,
                        st, ka, joins)
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}

}  // namespace

size_t latent_work_bytes(int, int N, int H, int C) {
    LatentPlan p = {};
    return carve_plan(&p, N, H, C, nullptr);
}

int launch_latent(const LatentArgs &a, cudaStream_t st) {
    LatentKernelArgs ka = {};
    ka.a = a;
    ka.p.B = a.B;
    ka.p.lens = a.lens;
    ka.p.most = a.width << a.c.page_shift;
    carve_plan(&ka.p, a.N, a.H, a.c.C, a.work);
    const int sms = multiprocessors();
    CUtensorMap map;
    if (sms <= 0 || !make_map(&map, a.c)) return SPEC_ERR_CUDA;
    choose_width(&ka.p, sms < kMaxGrid ? sms : kMaxGrid);
    return a.c.C == 512 ? launch_shape<512>(ka, map, st) : a.c.C == 256 ? launch_shape<256>(ka, map, st) : launch_shape<128>(ka, map, st);
}

}  // namespace specv
