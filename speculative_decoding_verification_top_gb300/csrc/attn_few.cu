// attn_few.cu -- attention of units with few query rows: a chain of drafts, a
// single token, and whatever else has at most 64 rows (new tokens x query
// heads of a group) per key/value head.
//
// attn_few_kernel   persistent, one CTA per SM; its share of the tiles (see
//                   attn.cu) segment by segment.  Memory-bound: a tile's keys
//                   and values are read once and used for few rows.
// The products are taken transposed, so that the 128 positions of a tile fill
// the tensor core's 128 rows and the query rows are its columns (NR = 32 or
// 64): S^T = K Q^T, O^T += V^T P^T.  That makes a product cost a quarter of
// what 128 padded query rows would, gives a softmax thread a position and NR
// scores, and leaves room in TMEM for two S ahead per group.
//   warps 0-3, 4-7   two softmax groups, a thread per position, on alternate
//                    tiles, each with its own (m, l, O); over an e4m3 cache they
//                    widen the tile's values to bf16 first, while its scores are
//                    on their way
//   warps 8, 10      load key and value tiles page by page (TMA) into a ring each,
//                    warp 10 an e4m3 tile's exponents too
//   warp 9           issues the products (tcgen05); scores run up to two tiles
//                    ahead of the values.  (Scores and values issued by two warps
//                    took 70 us where this takes 62, one sequence of 131077 e4m3
//                    positions.)
//   warp 11          the query tile, and what belongs to its rows, of the next
//                    segment; tells the softmax groups which it is
// The reference maximum of a row is common to a group's 128 threads; a vote per
// tile (one hardware barrier) says whether any score outgrew it, which after
// the first tile of a segment is rare, so maxima are reduced only then.  l is
// kept per thread and summed once a segment.
// Measured: 64 chains of 6 over e4m3 caches of 4100 to 8200 positions, 8 heads
// of 128 (819 MB): 183 us, 4.5 TB/s (its loads alone 152): bound by what the groups
// issue (the call takes 202 us, without the widening 164).  128 chains of 4 over bf16 caches of 2500 to
// 5003, 4 heads of 64, capped (497 MB): 110 us (its loads alone 102).  Beside the
// loads a call costs about 20 us of launch, line and first tiles, which is what a
// single token over 2049 positions takes.
// Dropped: four warps more that widen (the groups' registers made room for by
// setmaxnreg), all of it or a part: 234 to 271 us a call, where this takes 201; half
// a tile at a time by them: 457.

#include "attn_plan.cuh"

namespace specv {
namespace {

// Key slots: at most as many as there are score buffers, so that a slot is free
// when the buffer of the tile kMaxKeys before is full.
constexpr int kMaxKeys = 4;
constexpr int kGroupBarrier = 1;  // hardware barrier of softmax group 0; + 1 for group 1
constexpr int kFirstBarrier = 3;  // of both
constexpr float kNone = -FLT_MAX; // reference of a row that has seen nothing: below any score

struct Barriers {
    unsigned long long k_full[kMaxKeys], v_full[kMaxSlots], v_empty[kMaxSlots];
    unsigned long long q_full[2], q_empty[2];
    unsigned long long s_full[4], p_full[4];
    unsigned long long done[2];  // a group's last product of a segment; over e4m3 every one
    unsigned long long drained;
};

template <int NR>
struct alignas(16) Rows {  // what belongs to the query rows of a segment
    float rs[NR];       // score factor (the log2 e and the query's own in it)
    float slope[NR];    // slope * log2 e
    float at[NR];       // position index less the segment's origin
    int pos[NR];        // position index
};

template <int NR>
struct Shared {
    Barriers bar;
    Start start;
    Rows<NR> rows[2];
    Segment seg[2];        // the segment of each query tile; rows = 0: no more
    alignas(16) float ref[2][NR];  // per group: reference maximum; +inf for no row
    alignas(16) float keep[2][NR]; // per group: factor of the last growth
    float red[2][4][NR];   // per group and warp
    float factor[2][NR];   // e4m3: the query rows' own factors
    uint32_t tmem;
    int dead;              // a wait ran out: everyone leaves
    int fail[16];          // per segment (mod 16): a page id out of range
    int odd[2][2];         // per group and segment (mod 2): a tile it cleaned held values that are not finite
};

template <int D, bool E4M3, int NR>
struct Layout : Shape<D, E4M3> {
    using S = Shape<D, E4M3>;
    static constexpr int kQBlock = NR * S::kRow;                     // a block of the query tile
    static constexpr int kQ = kQBlock * (E4M3 ? 2 : S::kHalves);
    static constexpr int kPRow = 2 * NR;                             // bytes of a row of weights
    static constexpr int kP = kTile * kPRow;                         // one buffer of weights
    static constexpr int kPBufs = E4M3 ? 2 : 4;
    static constexpr int kExps = E4M3 ? 2 * kTile : 0;               // a tile's exponents
    static constexpr int kWide = E4M3 ? Shape<D, false>::kSlot : 0;  // a value tile widened to bf16
    static constexpr int kFixed = static_cast<int>((sizeof(Shared<NR>) + 127) / 128 * 128);
    static constexpr int kMost = 2 * kMaxKeys + 4;
    static constexpr int kRoom = (kSmemMax - kFixed - 2 * kQ - kPBufs * kP - 2 * kWide - kMost * kExps) / S::kSlot;
    static constexpr int kSlots = kRoom < kMost ? kRoom : kMost;
    static constexpr int kHalf = kSlots / 2 < kMaxKeys ? kSlots / 2 : kMaxKeys;
    // Of values; over e4m3 an even number, so that a group's tiles have slots of their own.
    static constexpr int kV = E4M3 ? (kSlots - kHalf) / 2 * 2 : kSlots - kHalf;
    static constexpr int kK = kSlots - kV < kMaxKeys ? kSlots - kV : kMaxKeys;  // of keys
    static constexpr int kBytes = kFixed + 2 * kQ + kPBufs * kP + 2 * kWide + (kK + kV) * S::kSlot + kV * kExps;
    static_assert(kK >= 1 && kV >= 2, "two groups' value tiles");
    static constexpr uint32_t kColumns = NR == 32 ? 256 : 512;       // TMEM: 4 S and 2 O of NR columns
};

// Folds v[0..NR) over a warp's lanes with f: lane i ends up with column(s) i
// (NR = 32), or 2 i and 2 i + 1 (NR = 64).
template <int NR, typename F>
__device__ __forceinline__ void fold_columns(const float (&v)[NR], float (&out)[NR / 32], F f) {
    const int lane = threadIdx.x & 31;
    float x[NR / 2];
    const bool up = lane & 16;
#pragma unroll
    for (int k = 0; k < NR / 2; ++k) {
        const float mine = up ? v[k + NR / 2] : v[k], other = up ? v[k] : v[k + NR / 2];
        x[k] = f(mine, __shfl_xor_sync(0xffffffffu, other, 16));
    }
#pragma unroll
    for (int o = 8; o > 0; o /= 2) {
        const int n = NR / 2 * o / 16;  // columns after this step
        const bool hi = lane & o;
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const float mine = hi ? x[k + n] : x[k], other = hi ? x[k] : x[k + n];
            x[k] = f(mine, __shfl_xor_sync(0xffffffffu, other, o));
        }
    }
#pragma unroll
    for (int k = 0; k < NR / 32; ++k) out[k] = x[k];
}

// The rows (bits) that see this thread's position, in a tile that some rows do
// not see whole.  Rows of a token see alike: four tokens at a time, their mask
// bytes in flight together.
template <int NR>
__device__ __forceinline__ unsigned long long seen_rows(const AttnArgs &a, const Segment &g, const Rows<NR> &rows, int j,
                                                        int pos_j) {
    constexpr int kAtOnce = 4;
    const int c = j - (g.len - a.N), tokens = g.rows / a.G;
    const bool held = j < g.len, node = !g.shared && held && c >= 0;
    const unsigned long long per = a.G >= 64 ? ~0ull : (1ull << a.G) - 1;
    unsigned long long seen = 0;
    for (int n0 = 0; n0 < tokens; n0 += kAtOnce) {
        uint8_t m[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int n = min(n0 + k, tokens - 1);
            m[k] = !node ? 1 : a.mask ? a.mask[(static_cast<long long>(g.b) * a.N + n) * a.N + c] : c <= n;
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int n = min(n0 + k, tokens - 1);
            const bool y = held && m[k] != 0 &&
                           (a.window == 0 || static_cast<long long>(rows.pos[n * a.G]) - pos_j < a.window);
            if (y && n0 + k < tokens) seen |= per << (n * a.G);
        }
    }
    return seen;
}

// Adds to the unit's rows of output column d what the products left out:
// values that are not finite, of the positions each row sees in the segment's
// tiles.  (In a tile that was not cleaned they are in the sum already, and
// adding them again changes nothing.)
template <int D, bool E4M3, int NR>
__device__ __noinline__ void add_odd_values(const AttnArgs &a, const Segment g, const Rows<NR> &rows, int d, float *o) {
    for (int j = g.t0 * kTile; j < min(g.len, g.t1 * kTile); ++j) {
        int slot;
        const int page = page_of(a.c, pages_of(a, g), INT_MAX, j, &slot);
        if (page < 0) continue;
        const float y = odd_value<E4M3>(a.c, cache_row(a.c, page, g.h, slot) * D + d);
        if (isfinite(y)) continue;
        const int c = j - (g.len - a.N);
        const int pos_j = !g.shared && c >= 0 && a.pos ? a.pos[static_cast<long long>(g.b) * a.N + c]
                                                       : (g.shared ? 0 : a.shared_len) + j;
        const unsigned long long seen = seen_rows<NR>(a, g, rows, j, pos_j);
        for (int i = 0; i < g.rows; ++i)
            if (seen >> i & 1) o[static_cast<long long>(i) * D] += y;
    }
}

template <int D, bool E4M3, bool EXTRA, int NR>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_few_kernel(const __grid_constant__ KernelArgs ka, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap) {
    using S = Layout<D, E4M3, NR>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const AttnArgs &a = ka.a;
    const Plan &p = ka.p;
    uint8_t *k_ring = smem, *v_ring = k_ring + S::kK * S::kSlot, *wide = v_ring + S::kV * S::kSlot;
    uint8_t *pt = wide + 2 * S::kWide, *qt = pt + S::kPBufs * S::kP;
    int8_t *exps = reinterpret_cast<int8_t *>(qt + 2 * S::kQ);  // [kV][2][kTile]
    Shared<NR> &sh = *reinterpret_cast<Shared<NR> *>(exps + S::kV * S::kExps);
    Barriers &bar = sh.bar;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < S::kK; ++i) bar_init(smem_addr(&bar.k_full[i]), 1);
        for (int i = 0; i < S::kV; ++i) {
            bar_init(smem_addr(&bar.v_full[i]), E4M3 ? 33 : 1);  // the tile, and its exponents by 32 lanes
            bar_init(smem_addr(&bar.v_empty[i]), E4M3 ? 4 : 1);  // the group's warps, or the product
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_addr(&bar.q_full[i]), 1);
            bar_init(smem_addr(&bar.q_empty[i]), 9);  // the products, and eight softmax warps
            bar_init(smem_addr(&bar.done[i]), 1);
        }
        for (int i = 0; i < 4; ++i) {
            bar_init(smem_addr(&bar.s_full[i]), 1);
            bar_init(smem_addr(&bar.p_full[i]), 4);
        }
        bar_init(smem_addr(&bar.drained), 1);
        sh.dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_proxy();
    }
    if (warp == 9) tmem_alloc(smem_addr(&sh.tmem), S::kColumns);
    // Up to here this may run beside the kernel before it.  (Beside the prefix's
    // kernel all of it may: that one has waited for what came before the call.)
    if (!ka.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    long long from, to;
    const int prefix_first = find_share(p, sh.start, &from, &to);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = sh.tmem;
    volatile int *dead = &sh.dead;
    Walk walk(p, from, to, sh.start.b0, sh.start.base0, prefix_first);
    Segment g;
    const float mul = a.cap > 0.0f ? fabsf(a.scale) / a.cap : fabsf(a.scale) * kLog2e;

    // A segment's query tile and rows into half i of the ring of two.
    auto stage = [&](int i, int me, int threads) {
        stage_queries<D, E4M3>(a, g, 0, g.rows, NR, qt + i * S::kQ, sh.factor[i], me, threads);
    };
    auto stage_rows = [&](int i, int me, int threads) {
        const int origin = (g.shared ? 0 : a.shared_len) + g.len;
        for (int r = me; r < NR; r += threads) {
            const bool has = r < g.rows;
            const int tok = (g.shared ? 0 : g.b * a.N) + (has ? r / a.G : 0), b = tok / a.N;
            const int pos = !has ? 0 : a.pos ? a.pos[tok] : a.shared_len + (g.shared ? a.lens[b] : g.len) - a.N + tok % a.N;
            sh.rows[i].rs[r] = mul * (E4M3 ? sh.factor[i][r] : 1.0f);
            sh.rows[i].slope[r] = EXTRA && a.slopes && has ? a.slopes[g.h * a.G + r % a.G] * kLog2e : 0.0f;
            sh.rows[i].at[r] = static_cast<float>(pos - origin);
            sh.rows[i].pos[r] = pos;
        }
    };
    if (warp == 8) {
        // ---- key loads
        Loader<D, E4M3, S::kK> load;
        PageIds ids;
        bool live = true;
        for (uint32_t seg = 0; live && walk.next(&g); ++seg) {
            if (lane == 0) sh.fail[seg & 15] = 0;
            __syncwarp();
            ids.begin(a, g);
            for (int t = g.t0; live && t < g.t1; ++t) {
                // The slot's last tile n: its scores are in buffer n % 4.
                const int n = static_cast<int>(load.n) - S::kK;
                if (n >= 0) live = bar_wait(smem_addr(&bar.s_full[n & 3]), (n >> 2) & 1, dead);
                live = __all_sync(0xffffffffu, live) &&
                       load.tile(a, g, ids, t, &kmap, smem_addr(k_ring), bar.k_full, 0, dead, &sh.fail[seg & 15]);
            }
        }
        if (!live) load.drain(bar.k_full);
    } else if (warp == 10) {
        // ---- value loads
        Loader<D, E4M3, S::kV> load;
        PageIds ids;
        bool live = true;
        while (live && walk.next(&g)) {
            ids.begin(a, g);
            for (int t = g.t0; live && t < g.t1; ++t)
                live = load.tile(a, g, ids, t, &vmap, smem_addr(v_ring), bar.v_full, smem_addr(&bar.v_empty[load.slot]), dead,
                                 nullptr, E4M3 ? smem_addr(exps) : 0);
        }
        if (!live) load.drain(bar.v_full);
    } else if (warp == 9) {
        // ---- products
        if (elect_one()) {
            using T = Shape<D, false>;  // the values as the product takes them
            constexpr uint32_t kQk = mma_desc(E4M3, NR, false, false), kPv = mma_desc(false, NR, true, true);
            constexpr uint32_t kHi = kMatrixHi<S::kRow>, kPHi = kMatrixHi<S::kPRow>, kVHi = kMatrixHi<T::kRow>;
            // Values narrower than 128 columns: the second block is the first again,
            // and its rows of O are not read.
            constexpr uint32_t kLead = D == 128 ? T::kMat : 0;
            const uint32_t q0 = matrix_lo(smem_addr(qt), 0), k0 = matrix_lo(smem_addr(k_ring), 0);
            const uint32_t v0 = matrix_lo(smem_addr(E4M3 ? wide : v_ring), kLead), p0 = matrix_lo(smem_addr(pt), 0);
            const uint32_t k_full = smem_addr(&bar.k_full[0]), v_full = smem_addr(&bar.v_full[0]);
            const uint32_t v_empty = smem_addr(&bar.v_empty[0]), q_full = smem_addr(&bar.q_full[0]);
            const uint32_t s_full = smem_addr(&bar.s_full[0]), p_full = smem_addr(&bar.p_full[0]);
            // Two walks over the same tiles: the scores', and the values' behind it.
            Walk ahead = walk;
            Segment s;
            uint32_t is = 0, iv = 0, seg_s = 0, seg_v = 0, ks = 0, kp = 0, vs = 0, vp = 0, q = q0;
            bool more_s = ahead.next(&s), live = true, begin = true;
            int left_s = s.t1 - s.t0;
            while (live && walk.next(&g)) {
                int left_v = g.t1 - g.t0;
                uint32_t first = 2;  // tiles to come that are their group's first of the segment
                while (live && left_v > 0) {
                    // At most two tiles ahead, and one segment: the query ring holds two.  A
                    // score buffer is free then: its last tile's weights have been waited for.
                    if (more_s && is <= iv + 2 && seg_s <= seg_v + 1) {
                        if (begin) {
                            live = bar_wait(q_full + 8 * (seg_s & 1), (seg_s >> 1) & 1, dead);
                            q = q0 + (seg_s & 1) * (S::kQ >> 4);
                            begin = false;
                        }
                        live = live && bar_wait(k_full + 8 * ks, kp, dead);
                        fence_after_sync();
                        const uint32_t k = k0 + ks * (S::kSlot >> 4), d = tmem + (is & 3) * NR;
                        if (E4M3) {
#pragma unroll
                            for (int i = 0; i < 2 * (D / 32); ++i) {
                                const uint32_t term = i / (D / 32), j = i % (D / 32);
                                mma_ss<true>(d, k + (j * 32 >> 4), kHi, q + ((term * S::kQBlock + j * 32) >> 4), kHi, kQk,
                                             i > 0);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < D / 16; ++i)
                                mma_ss<false>(d, k + (((i / 4) * S::kMat + (i % 4) * 32) >> 4), kHi,
                                              q + (((i / 4) * S::kQBlock + (i % 4) * 32) >> 4), kHi, kQk, i > 0);
                        }
                        mma_commit(s_full + 8 * (is & 3));
                        if (++ks == S::kK) {
                            ks = 0;
                            kp ^= 1;
                        }
                        ++is;
                        if (--left_s == 0) {
                            mma_commit(smem_addr(&bar.q_empty[seg_s & 1]));
                            more_s = ahead.next(&s);
                            left_s = s.t1 - s.t0;
                            ++seg_s;
                            begin = true;
                        }
                        continue;
                    }
                    live = (E4M3 || bar_wait(v_full + 8 * vs, vp, dead)) && bar_wait(p_full + 8 * (iv & 3), (iv >> 2) & 1, dead);
                    fence_after_sync();
                    const uint32_t v = v0 + (E4M3 ? (iv & 1) * (S::kWide >> 4) : vs * (S::kSlot >> 4));
                    const uint32_t pb = p0 + (iv & (S::kPBufs - 1)) * (S::kP >> 4), d = tmem + (4 + (iv & 1)) * NR;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mma_ss<false>(d, v + (i * 16 * T::kRow >> 4), kVHi, pb + (i * 16 * S::kPRow >> 4), kPHi, kPv,
                                      i > 0 || first == 0);
                    if (!E4M3) mma_commit(v_empty + 8 * vs);
                    if (E4M3 || left_v <= 2) mma_commit(smem_addr(&bar.done[iv & 1]));
                    if (++vs == S::kV) {
                        vs = 0;
                        vp ^= 1;
                    }
                    ++iv;
                    first -= first > 0;
                    --left_v;
                }
                ++seg_v;
            }
            if (!live) {  // products in flight end before TMEM is freed
                mma_commit(smem_addr(&bar.drained));
                bar_drain(smem_addr(&bar.drained), 0);
            }
        }
        __syncwarp();
    } else if (warp == 11) {
        // ---- query tiles, a segment ahead (the softmax groups stage the first)
        bool live = true, more = walk.next(&g);
        for (uint32_t seg = 1; live && more; ++seg) {
            more = walk.next(&g);
            live = bar_wait(smem_addr(&bar.q_empty[seg & 1]), ((seg >> 1) & 1) ^ 1, dead);
            live = __all_sync(0xffffffffu, live);
            if (!live) break;
            if (more) {
                stage(seg & 1, lane, 32);
                __syncwarp();
                stage_rows(seg & 1, lane, 32);
            } else {
                g.rows = 0;
            }
            if (lane == 0) sh.seg[seg & 1] = g;
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) bar_arrive(smem_addr(&bar.q_full[seg & 1]));
        }
    } else {
        // ---- softmax groups
        const int w = warp >> 2, quad = warp & 3, row = tid & 127;  // row: the thread's position in a tile
        const uint32_t lanes = static_cast<uint32_t>(quad) << 21;   // this warp's TMEM lanes
        const uint32_t ot = tmem + lanes + (4 + w) * NR;
        float *ref = sh.ref[w], *keep = sh.keep[w];
        auto vote = [&](bool x) {
            __syncwarp();
            return any_of(kGroupBarrier + w, 128, x);
        };
        uint32_t seg = 0, tile = 0, cnt = 0;  // segments, tiles of the CTA, tiles of this group
        uint32_t ended = 0;                   // segments this group had a tile of
        bool live = true;
        // The first segment's query tile: all eight warps, while the loads start.
        if (!walk.next(&g)) g.rows = 0;
        if (g.rows) stage(0, tid, 256);
        __syncwarp();
        if (E4M3) any_of(kFirstBarrier, 256, false);  // the rows' factors
        if (g.rows) stage_rows(0, tid, 256);
        if (tid == 0) sh.seg[0] = g;
        fence_async_proxy();
        __syncwarp();
        any_of(kFirstBarrier, 256, false);
        if (tid == 0) bar_arrive(smem_addr(&bar.q_full[0]));
        bool ok = true;
        while (g.rows) {
            const uint32_t half = seg & 1;
            const Units &u = g.shared ? p.shared : p.own;
            const long long part = static_cast<long long>(g.slot) * 2 + w;
            float2 *ml = u.ml + part * u.rc;
            const Rows<NR> &rows = sh.rows[half];
            const int n_rows = g.rows, first_tile = g.t0 + ((tile ^ w) & 1);  // this group's first
            const int origin = (g.shared ? 0 : a.shared_len) + g.len;
            const int last_pos = a.window > 0 ? last_position(a, g) : 0;
            float l[NR];
#pragma unroll
            for (int i = 0; i < NR; ++i) l[i] = 0.0f;
            if (row < NR) ref[row] = row < n_rows ? kNone : INFINITY;
            if (row == 0) sh.odd[w][half] = 0;
            if (vote(!ok)) {  // the reference and the flag are set
                live = false;
                break;
            }
            for (int t = first_tile; t < g.t1; t += 2, ++cnt) {
                const int j0 = t * kTile, j = j0 + row;
                const uint32_t buf = w + 2 * (cnt & 1), phase = (cnt >> 1) & 1;
                float fk = 1.0f;  // e4m3: 2^(the key's exponent)
                const bool whole = sees_whole(a, g, j0, last_pos);
                // Position index of this thread's position, and the rows that see it.
                int pos_j = (g.shared ? 0 : a.shared_len) + j;
                unsigned long long seen = ~0ull;
                const uint32_t vi = tile + (t - g.t0);
                if (!whole) {
                    const int c = j - (g.len - a.N);
                    if (!g.shared && c >= 0 && j < g.len && a.pos) pos_j = a.pos[static_cast<long long>(g.b) * a.N + c];
                    seen = seen_rows<NR>(a, g, rows, j, pos_j);
                }
                if constexpr (E4M3) {
                    // The values widened, while the scores are on their way.  Their buffer, and the
                    // weights', is free after the group's last product; the slot's earlier fill was
                    // this group's.
                    if (cnt > 0) ok = ok && bar_wait(smem_addr(&bar.done[w]), (cnt - 1) & 1, dead);
                    ok = ok && bar_wait(smem_addr(&bar.v_full[vi % S::kV]), (vi / S::kV) & 1, dead);
                    const int8_t *e = exps + vi % S::kV * S::kExps + row;
                    fk = power_of(e[0]);
                    if (ok && widen_values<D, 4>(v_ring + vi % S::kV * S::kSlot, wide + w * S::kWide, row, power_of(e[kTile]),
                                                 j < g.len, !whole))
                        sh.odd[w][half] = 1;
                    __syncwarp();
                    if (lane == 0) bar_arrive(smem_addr(&bar.v_empty[vi % S::kV]));
                }
                ok = ok && bar_wait(smem_addr(&bar.s_full[buf]), phase, dead);
                fence_after_sync();
                __syncwarp();
                float s[NR];
#pragma unroll
                for (int c = 0; c < NR; c += 32) tmem_load32(tmem + lanes + buf * NR + c, s + c);
                tmem_load_wait();
                const float at = static_cast<float>(pos_j - origin);
                const bool cap = EXTRA && a.cap > 0.0f;
                const F2 fk2 = pair_of(fk, fk), rs2 = pair_of(mul, mul), at2 = pair_of(at, at);
                const F2 minus = pair_of(-1.0f, -1.0f);
                float over = kNegInf;
#pragma unroll
                for (int c0 = 0; c0 < NR; c0 += 16) {
                    if (c0 >= n_rows) break;
                    if (cap) {
#pragma unroll
                        for (int c = c0; c < c0 + 16; ++c) s[c] *= E4M3 ? fk * rows.rs[c] : mul;
                        cap_scores<16>(s + c0, a.cap);
                    }
                    float top[2] = {kNegInf, kNegInf};
#pragma unroll
                    for (int c = c0; c < c0 + 16; c += 4) {
                        F2 y[2] = {pair_of(s[c], s[c + 1]), pair_of(s[c + 2], s[c + 3])};
                        const ulonglong2 m4 = *reinterpret_cast<const ulonglong2 *>(&ref[c]);
                        const F2 m[2] = {{m4.x}, {m4.y}};
                        if (!cap) {
                            if (E4M3) {
                                const ulonglong2 r4 = *reinterpret_cast<const ulonglong2 *>(&rows.rs[c]);
                                y[0] = mul2(mul2(y[0], fk2), F2{r4.x});
                                y[1] = mul2(mul2(y[1], fk2), F2{r4.y});
                            } else {
                                y[0] = mul2(y[0], rs2);
                                y[1] = mul2(y[1], rs2);
                            }
                        }
                        if (EXTRA) {
                            const ulonglong2 s4 = *reinterpret_cast<const ulonglong2 *>(&rows.slope[c]);
                            const ulonglong2 a4 = *reinterpret_cast<const ulonglong2 *>(&rows.at[c]);
                            y[0] = fma2(F2{s4.x}, fma2(F2{a4.x}, minus, at2), y[0]);
                            y[1] = fma2(F2{s4.y}, fma2(F2{a4.y}, minus, at2), y[1]);
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float2 t2 = parts_of(y[k]);
                            if (!whole) {
                                if (!(seen >> (c + 2 * k) & 1)) t2.x = kNegInf;
                                if (!(seen >> (c + 2 * k + 1) & 1)) t2.y = kNegInf;
                            }
                            s[c + 2 * k] = t2.x;
                            s[c + 2 * k + 1] = t2.y;
                            const float2 d = parts_of(fma2(m[k], minus, pair_of(t2.x, t2.y)));
                            top[k] = max3(top[k], d.x, d.y);
                        }
                    }
                    over = max3(over, top[0], top[1]);
                }
                const bool grown = vote(!ok || over > kSlack);
                if (grown) {
                    if (vote(!ok)) {
                        live = false;
                        break;
                    }
                    // Some row outgrew its reference: reduce the maxima, rescale.
#pragma unroll
                    for (int c = 0; c < NR; c += 16)
                        if (c >= n_rows)
                            for (int k = 0; k < 16; ++k) s[c + k] = kNegInf;
                    float top[NR / 32];
                    fold_columns<NR>(s, top, [](float x, float y) { return fmaxf(x, y); });
#pragma unroll
                    for (int k = 0; k < NR / 32; ++k) sh.red[w][quad][lane * (NR / 32) + k] = top[k];
                    vote(false);
                    if (row < NR) {
                        const float m0 = ref[row];
                        const float m1 = fmaxf(fmaxf(sh.red[w][0][row], sh.red[w][1][row]),
                                               fmaxf(sh.red[w][2][row], sh.red[w][3][row]));
                        const bool up = m1 > m0 && (m0 == kNone || m1 - m0 > kSlack);
                        keep[row] = !up ? 1.0f : m0 == kNone ? 0.0f : ex2(m0 - m1);
                        if (up) ref[row] = m1;
                    }
                    vote(false);
                    const bool wrote = t >= g.t0 + 2;
                    if (wrote) {  // the products so far have to be in
                        if (!E4M3) ok = bar_wait(smem_addr(&bar.v_empty[(vi - 2) % S::kV]), ((vi - 2) / S::kV) & 1, dead);
                        ok = __all_sync(0xffffffffu, ok);
                        fence_after_sync();
                    }
#pragma unroll
                    for (int c = 0; c < NR; c += 32) {
                        if (wrote) {
                            float o[32];
                            tmem_load32(ot + c, o);
                            tmem_load_wait();
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] *= keep[c + k];
                            tmem_store32(ot + c, reinterpret_cast<const uint32_t *>(o));
                            tmem_store_wait();
                        }
#pragma unroll
                        for (int k = 0; k < 32; ++k) l[c + k] *= keep[c + k];
                    }
                }
                // Weights, and their place as the product's operand: a row per position.
                // (Over bf16 their buffer is free: these scores came after the product that read it.)
                uint8_t *pb = pt + (E4M3 ? w : buf) * S::kP;
#pragma unroll
                for (int c0 = 0; c0 < NR; c0 += 16) {
                    if (c0 >= n_rows) break;
                    uint32_t pk[8];  // bf16 pairs
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int c = c0 + 4 * k;
                        const ulonglong2 m4 = *reinterpret_cast<const ulonglong2 *>(&ref[c]);
                        const float2 u = parts_of(fma2(F2{m4.x}, minus, pair_of(s[c], s[c + 1])));
                        const float2 v = parts_of(fma2(F2{m4.y}, minus, pair_of(s[c + 2], s[c + 3])));
                        const float x0 = ex2(u.x), x1 = ex2(u.y), x2 = ex2(v.x), x3 = ex2(v.y);
                        l[c] += x0, l[c + 1] += x1, l[c + 2] += x2, l[c + 3] += x3;
                        pk[2 * k] = bf16_pair(x0, x1);
                        pk[2 * k + 1] = bf16_pair(x2, x3);
                    }
                    *reinterpret_cast<uint4 *>(pb + swizzled<S::kPRow>(row, 2 * c0)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    *reinterpret_cast<uint4 *>(pb + swizzled<S::kPRow>(row, 2 * c0 + 16)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
                }
                if constexpr (!E4M3) {
                    if (!whole) {
                        // A wait by parity tells its fill of the slot from the one before only once
                        // that one is known to be over.  These scores came after the product of tile
                        // vi - 3; with two slots the one before is tile vi - 2, whose product is waited for.
                        if (S::kV < 3 && vi >= S::kV)
                            ok = ok && bar_wait(smem_addr(&bar.v_empty[vi % S::kV]), ((vi - S::kV) / S::kV) & 1, dead);
                        ok = ok && bar_wait(smem_addr(&bar.v_full[vi % S::kV]), (vi / S::kV) & 1, dead);
                        if (ok && clean_values<D>(v_ring + vi % S::kV * S::kSlot, row, j < g.len)) sh.odd[w][half] = 1;
                    }
                }
                fence_async_proxy();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) bar_arrive(smem_addr(&bar.p_full[buf]));
            }
            if (!live) break;
            // ---- the group's partial result of the segment
            const bool wrote = first_tile < g.t1;
            // What comes next, while the last product runs.
            ok = ok && bar_wait(smem_addr(&bar.q_full[half ^ 1]), ((seg + 1) >> 1) & 1, dead);
            const Segment next = sh.seg[half ^ 1];
            if (wrote) {
                ok = ok && bar_wait(smem_addr(&bar.done[w]), (E4M3 ? cnt - 1 : ended++) & 1, dead);
                fence_after_sync();
                __syncwarp();
                float sum[NR / 32];
                fold_columns<NR>(l, sum, [](float x, float y) { return x + y; });
#pragma unroll
                for (int k = 0; k < NR / 32; ++k) sh.red[w][quad][lane * (NR / 32) + k] = sum[k];
            }
            if (vote(!ok)) {
                live = false;
                break;
            }
            // (A group without a tile of the segment has not waited for its loads: it
            // leaves the flags to the other.)
            const bool failed = wrote && reinterpret_cast<volatile int *>(sh.fail)[seg & 15] != 0;
            const bool odd = wrote && reinterpret_cast<volatile int *>(sh.odd[w])[half] != 0;
            if (row < n_rows) {
                const float m = ref[row];
                const float sum = !wrote ? 0.0f : (sh.red[w][0][row] + sh.red[w][1][row]) + (sh.red[w][2][row] + sh.red[w][3][row]);
                ml[row] = make_float2(m == kNone ? kNegInf : m, failed ? NAN : sum);
            }
            if (wrote && row < D) {
                float *o = u.o + part * u.rc * D + row;
#pragma unroll
                for (int c = 0; c < NR; c += 32) {
                    if (c >= n_rows) break;
                    float v[32];
                    tmem_load32(ot + c, v);
                    tmem_load_wait();
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (c + k < n_rows) o[static_cast<long long>(c + k) * D] = v[k];
                }
                if (odd) add_odd_values<D, E4M3, NR>(a, g, rows, row, o);
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) bar_arrive(smem_addr(&bar.q_empty[half]));
            ++seg;
            tile += g.t1 - g.t0;
            g = next;
        }
        if (!live && row == 0) atomicOr(a.err, static_cast<uint32_t>(SPEC_DATA_STALL));
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 9) tmem_free(tmem, S::kColumns);
    // Launched beside the prefix's kernel: this grid ends after that one.
    if (ka.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D, bool E4M3, bool EXTRA, int NR>
int launch_shape(KernelArgs &ka, int grid, const CUtensorMap &kmap, const CUtensorMap &vmap,
                 cudaStream_t st) {
    static int done[64];
    auto kernel = attn_few_kernel<D, E4M3, EXTRA, NR>;
    if (!allow_smem(kernel, Layout<D, E4M3, NR>::kBytes, done)) return SPEC_ERR_CUDA;
    return launch_early(kernel, dim3(grid), dim3(kAttnThreads), Layout<D, E4M3, NR>::kBytes, st, ka, kmap, vmap)
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}

template <int D, bool E4M3, bool EXTRA>
int launch_rows(KernelArgs &ka, int grid, const CUtensorMap &kmap, const CUtensorMap &vmap,
                cudaStream_t st) {
    const int rows = ka.p.do_shared ? ka.p.shared.rows : ka.p.own.rows;
    return rows <= 32 ? launch_shape<D, E4M3, EXTRA, 32>(ka, grid, kmap, vmap, st)
                      : launch_shape<D, E4M3, EXTRA, 64>(ka, grid, kmap, vmap, st);
}

}  // namespace

int launch_few(KernelArgs &ka, int grid, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
    const bool extra = ka.a.cap > 0.0f || ka.a.slopes, wide = ka.a.c.D == 128;
    if (ka.a.c.e4m3)
        return extra ? (wide ? launch_rows<128, true, true>(ka, grid, kmap, vmap, st)
                             : launch_rows<64, true, true>(ka, grid, kmap, vmap, st))
                     : (wide ? launch_rows<128, true, false>(ka, grid, kmap, vmap, st)
                             : launch_rows<64, true, false>(ka, grid, kmap, vmap, st));
    return extra ? (wide ? launch_rows<128, false, true>(ka, grid, kmap, vmap, st)
                         : launch_rows<64, false, true>(ka, grid, kmap, vmap, st))
                 : (wide ? launch_rows<128, false, false>(ka, grid, kmap, vmap, st)
                         : launch_rows<64, false, false>(ka, grid, kmap, vmap, st));
}

}  // namespace specv
