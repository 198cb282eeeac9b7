// attn_wide.cu -- attention of units with many query rows: a candidate tree's
// nodes, or a whole batch over its shared prefix.
//
// attn_wide_kernel   persistent, one CTA per SM; its share of the tiles (see
//                    attn.cu) segment by segment.
//   warps 0-3, 4-7   two softmax groups, a thread per query row: S from TMEM,
//                    2^(t - m), P back into TMEM over S
//   warp 8           loads key and value tiles page by page (TMA)
//   warp 9           issues the products (tcgen05, M = 128 rows): S = Q K^T,
//                    then O += P V with P in TMEM
//   warps 10, 11     over an e4m3 cache: the keys' exponents as factors, and the
//                    value tiles widened to bf16, half a tile's positions each
//   (the softmax groups stage the query tiles of their next segment)
// A unit of over 128 rows gives each group 128 rows of its own and both work
// on every tile; a smaller one alternates its tiles between the groups, so
// that one group's softmax runs under the other's products.  TMEM: two S of
// 128 columns and two O of D.
//
// e4m3 cache: S = Q1 K^T + Q2 K^T with the query's two e4m3 terms, at the
// e4m3 rate, costs what one bf16 product does.  A key's exponent multiplies its
// column of S.  Values are multiplied as bf16, their exponent in them, so that
// weights are what they are over a bf16 cache.
//
// Bound by the chain softmax -> O += P V -> next S of a group, of which two are
// in flight: a tile of 256 rows takes 3400 cycles in bf16, where its products are
// 2048 and a group's softmax 1400.  The first half of P goes to its product while
// the second is made (16 trees of 85 nodes: 206 us a call against 214).  Loads
// (64 KB a bf16 tile) hold it up for a sixth.  Measured: 16 trees of 85 nodes, 8
// heads of 128, 4 query heads each, over bf16 caches of 3500 to 7001 with a distance
// bias (0.12 PFLOP): 178 us; 64 chains of 6 over one e4m3 prefix of 16001 (0.10
// PFLOP): 122 us.
// Tried and dropped: tiles in halves of 64 columns, so that a half's scores are
// made under the other's softmax (273 us against 246 at the time); the product
// loops written out per mode (250); registers moved between warps (more spills).

#include "attn_plan.cuh"

namespace specv {
namespace {

constexpr int kScaleRing = 4;
constexpr int kHelperBarrier = 1;  // hardware barrier of the e4m3 cache's two warps

struct Barriers {
    unsigned long long full[kMaxSlots], empty[kMaxSlots];
    unsigned long long scale_full[kScaleRing], scale_empty[kScaleRing];
    unsigned long long wide_full[2], wide_empty[2];
    unsigned long long q_full, left, o_full[2], s_full[2], p_half[2], p_full[2], drained;
};

struct Shared {
    Barriers bar;
    Start start;
    uint32_t tmem;
    int dead;      // a wait ran out: everyone leaves
    int fail[16];  // per segment (mod 16): a page id out of range
    int odd[16];   // per segment (mod 16): a cleaned tile held values that are not finite
};

template <int D, bool E4M3>
struct Layout : Shape<D, E4M3> {
    using S = Shape<D, E4M3>;
    static constexpr int kQ = E4M3 ? 2 * S::kMat : S::kSlot;  // a group's query tile
    static constexpr int kWide = E4M3 ? Shape<D, false>::kSlot : 0;  // a value tile widened to bf16
    // factors of the positions, and of the query rows
    static constexpr int kScale = E4M3 ? (kScaleRing * kTile + 2 * kGroupRows) * 4 : 0;
    static constexpr int kFixed = kScale + static_cast<int>((sizeof(Shared) + 127) / 128 * 128);
    static constexpr int kRoom = (kSmemMax - kFixed - 2 * kQ - 2 * kWide) / S::kSlot;
    static constexpr int kSlots = kRoom < kMaxSlots ? kRoom : kMaxSlots;
    static constexpr int kBytes = kFixed + 2 * kQ + 2 * kWide + kSlots * S::kSlot;
    static_assert(kSlots >= 5, "a tile's fill of a slot is told from the one before by what was multiplied since");
};

// What a softmax thread holds of its row.
struct Row {
    int b, n, tok;           // sequence, new token, token of the batch
    int first, pos_i;        // own position of token 0, the token's position index
    bool has;
    float rs, slope;         // score factor (the log2 e and the query's own in it), slope * log2 e
    float m, l;              // reference maximum and sum
};

// In a tile of positions that some rows do not see: the columns of each 32
// that this row sees, and the position index of this lane's column in each.
struct Seen {
    uint32_t rows[4];
    int pos[4];
};

// The first n of 32 bits, n clamped to 0..32.
__device__ __forceinline__ uint32_t first_bits(int n) {
    return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
}

// Loads that are not taken leave `otherwise`; no branch, so that many are in
// flight together.
__device__ __forceinline__ uint32_t byte_if(bool on, const uint8_t *at, uint32_t otherwise) {
    uint32_t r;
    asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u32 %0, %3;\n\t@p ld.global.u8 %0, [%1];\n\t}"
        : "=&r"(r)
        : "l"(at), "r"(static_cast<uint32_t>(on)), "r"(otherwise));
    return r;
}

// A row's set depends on its token alone, so the warp, a lane a column, finds
// the sets of its tokens (consecutive ones, from lo) four at a time, all their
// mask bytes in flight together (3 thousand cycles for 8 tokens of 85 columns,
// where loads under branches took 13); without a mask it is arithmetic.  (Out of
// line, with its arguments by value: inlined it would cost the main loop
// registers.)
__device__ __noinline__ Seen seen_columns(const uint8_t *mask, const int32_t *pos, int N, int window, int pos0, bool shared,
                                          int len, int first, bool has, int tok, int b_tok, int pos_i, int j0) {
    constexpr int kAtOnce = 4;
    const int lane = threadIdx.x & 31;
    Seen s;
    bool node[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = j0 + i * 32 + lane;
        node[i] = !shared && j >= first && j < len;
        s.pos[i] = pos0 + j;
        if (node[i] && pos) s.pos[i] = pos[b_tok + j - first];
        s.rows[i] = first_bits(len - (j0 + i * 32));
    }
    if (!shared && mask) {
        const uint32_t rows = __ballot_sync(0xffffffffu, has);
        const int lo = __shfl_sync(0xffffffffu, tok, 0), hi = __shfl_sync(0xffffffffu, tok, 31 - __clz(rows));
        const uint8_t *at = mask + static_cast<long long>(lo) * N + (j0 + lane - first);
        for (int t = lo; t <= hi; t += kAtOnce) {
            uint32_t m[kAtOnce][4];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) m[k][i] = byte_if(node[i] && t + k <= hi, at + i * 32, 1u);
                at += N;
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t word = __ballot_sync(0xffffffffu, m[k][i] != 0);
                    if (tok == t + k) s.rows[i] &= word;
                }
            }
        }
    } else if (!shared) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s.rows[i] &= first_bits(first + tok - b_tok + 1 - (j0 + i * 32));
    }
    if (window > 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t near = 0;
#pragma unroll 8
            for (int c = 0; c < 32; ++c)
                if (static_cast<long long>(pos_i) - __shfl_sync(0xffffffffu, s.pos[i], c) < window) near |= 1u << c;
            s.rows[i] &= near;
        }
    }
    if (!has) s.rows[0] = s.rows[1] = s.rows[2] = s.rows[3] = 0;
    return s;
}

// t of 32 columns from column `col` of a tile, from the raw products v in
// place; returns their maximum.  WHOLE: the row sees them all, and without a cap
// t is linear in the product and the column.
template <bool E4M3, bool EXTRA, bool WHOLE>
__device__ __forceinline__ float scores32(const AttnArgs &a, const Row &x, float base, int col, uint32_t seen, int pos_col,
                                          const float *fa, float (&v)[32]) {
    float top[2] = {kNegInf, kNegInf};
    if constexpr (WHOLE) {
        const F2 rs = pair_of(x.rs, x.rs), slope = pair_of(x.slope, x.slope), base2 = pair_of(base, base);
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
            F2 y = pair_of(v[c], v[c + 1]);
            F2 b;
            if (E4M3) y = mul2(y, *reinterpret_cast<const F2 *>(fa + col + c));
            b = EXTRA ? fma2(slope, pair_of(col + c, col + c + 1), base2) : pair_of(0.0f, 0.0f);
            const float2 t = parts_of(fma2(y, rs, b));
            v[c] = t.x;
            v[c + 1] = t.y;
            top[c / 2 & 1] = max3(top[c / 2 & 1], t.x, t.y);
        }
        return fmaxf(top[0], top[1]);
    }
    const bool by_pos = EXTRA && a.pos != nullptr;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
        if (E4M3) v[c] *= fa[col + c];
        v[c] *= x.rs;
    }
    if (EXTRA && a.cap > 0.0f) cap_scores<32>(v, a.cap);
#pragma unroll
    for (int c = 0; c < 32; ++c) {
        float y = v[c];
        if (EXTRA) {
            if (by_pos)
                y = fmaf(x.slope, static_cast<float>(__shfl_sync(0xffffffffu, pos_col, c) - x.pos_i), y);
            else
                y += fmaf(x.slope, static_cast<float>(col + c), base);
        }
        if (!(seen >> c & 1u)) y = kNegInf;
        v[c] = y;
        top[c & 1] = fmaxf(top[c & 1], y);
    }
    return fmaxf(top[0], top[1]);
}

// Weights 2^t of 32 columns, t already less the reference, into TMEM as the
// product's operand, 16 columns of bf16 pairs.  Returns their sum.
__device__ __forceinline__ float weights32(uint32_t dst, const F2 (&t)[16]) {
    F2 sum[2] = {pair_of(0.0f, 0.0f), pair_of(0.0f, 0.0f)};
    uint32_t pk[16];
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
        const float2 u = parts_of(t[c]), v = parts_of(t[c + 1]);
        const float x0 = ex2(u.x), x1 = ex2(u.y), x2 = ex2(v.x), x3 = ex2(v.y);
        sum[0] = add2(sum[0], pair_of(x0, x1));
        sum[1] = add2(sum[1], pair_of(x2, x3));
        pk[c] = bf16_pair(x0, x1);
        pk[c + 1] = bf16_pair(x2, x3);
    }
    tmem_store16(dst, pk);
    const float2 s = parts_of(add2(sum[0], sum[1]));
    return s.x + s.y;
}

// Moves the row's reference maximum up to `top` where that is needed,
// rescaling the sum and, if there is one, the accumulator in TMEM.
template <int D>
__device__ __forceinline__ void grow(Row &x, float top, bool wrote, uint32_t ot) {
    const bool up = top > x.m + kSlack;
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

// One tile of one row, twice over it, so that 32 values are worked on (and 32
// on their way) at a time: the maximum, with t back into TMEM where it is not
// cheap to take again; then the weights.
template <int D, bool E4M3, bool EXTRA>
__device__ __forceinline__ void softmax_tile(const AttnArgs &a, const Segment &g, Row &x, int j0, bool whole, bool wrote,
                                             uint32_t st, uint32_t ot, const float *fa, const Seen &seen, uint32_t half_bar) {
    const bool linear = whole && (!EXTRA || a.cap == 0.0f);
    // The bias: slope * (position index - pos_i), in a whole tile linear in the column.
    const float base = EXTRA ? x.slope * static_cast<float>((g.shared ? 0 : a.shared_len) + j0 - x.pos_i) : 0.0f;
    float top = kNegInf, t[2][32];
    if (linear) {
        tmem_load32(st, t[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            tmem_load_wait();
            if (c < 3) tmem_load32(st + (c + 1) * 32, t[(c + 1) & 1]);
            float(&v)[32] = t[c & 1];
            if constexpr (!E4M3 && !EXTRA) {
                float u[2] = {kNegInf, kNegInf};
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    u[0] = max3(u[0], v[k], v[k + 1]);
                    u[1] = max3(u[1], v[k + 2], v[k + 3]);
                }
                top = max3(top, u[0], u[1]);
            } else {
                top = fmaxf(top, scores32<E4M3, EXTRA, true>(a, x, base, c * 32, 0, 0, fa, v));
                if (E4M3) tmem_store32(st + c * 32, reinterpret_cast<const uint32_t *>(v));
            }
        }
        if (!E4M3 && !EXTRA) top *= x.rs;  // rs >= 0
    } else {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            tmem_load32(st + c * 32, t[0]);
            tmem_load_wait();
            uint32_t s = ~0u;
            int p = (g.shared ? 0 : a.shared_len) + j0 + c * 32 + (threadIdx.x & 31);
            if (!whole) {
                s = c == 0 ? seen.rows[0] : c == 1 ? seen.rows[1] : c == 2 ? seen.rows[2] : seen.rows[3];
                p = c == 0 ? seen.pos[0] : c == 1 ? seen.pos[1] : c == 2 ? seen.pos[2] : seen.pos[3];
            }
            top = fmaxf(top, scores32<E4M3, EXTRA, false>(a, x, base, c * 32, s, p, fa, t[0]));
            tmem_store32(st + c * 32, reinterpret_cast<const uint32_t *>(t[0]));
        }
    }
    grow<D>(x, top, wrote, ot);
    const float ref = x.m == kNegInf ? 0.0f : x.m;
    const bool stored = E4M3 || !linear;
    const float mul = stored ? 1.0f : x.rs, slope = stored ? 0.0f : x.slope, add = (stored ? 0.0f : base) - ref;
    const F2 mul_2 = pair_of(mul, mul), slope_2 = pair_of(slope, slope), add_2 = pair_of(add, add);
    tmem_store_wait();
    tmem_load32(st, t[0]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        tmem_load_wait();
        if (c < 3) tmem_load32(st + (c + 1) * 32, t[(c + 1) & 1]);
        F2 y[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const F2 v = pair_of(t[c & 1][2 * k], t[c & 1][2 * k + 1]);
            if (E4M3)
                y[k] = add2(v, add_2);
            else if (EXTRA)
                y[k] = fma2(v, mul_2, fma2(slope_2, pair_of(c * 32 + 2 * k, c * 32 + 2 * k + 1), add_2));
            else
                y[k] = fma2(v, mul_2, add_2);
        }
        x.l += weights32(st + c * 16, y);
        if (c == 1) {  // the product may begin with these
            tmem_store_wait();
            fence_before_sync();
            __syncwarp();
            if ((threadIdx.x & 31) == 0) bar_arrive(half_bar);
        }
    }
    tmem_store_wait();
}

// Adds to the 32 output columns from `col` on what the products left out:
// values that are not finite, of the positions the row sees in the segment's
// cleaned tiles.  (In a tile that was not cleaned they are in the sum already,
// and adding them again changes nothing.)
template <int D, bool E4M3>
__device__ __noinline__ void add_odd_values(const AttnArgs &a, const Segment g, const Row x, int col, float *dst) {
    for (int t = g.t0; t < g.t1; ++t) {
        for (int j = t * kTile; j < min(g.len, (t + 1) * kTile); ++j) {
            int pj, slot;
            if (g.shared ? a.window > 0 && static_cast<long long>(x.pos_i) - j >= a.window
                         : !sees(a, x.b, x.n, x.pos_i, x.first, g.len, j, &pj))
                continue;
            const int page = page_of(a.c, pages_of(a, g), INT_MAX, j, &slot);
            if (page < 0) continue;
            const long long at = cache_row(a.c, page, g.h, slot) * D + col;
            for (int k = 0; k < 32; ++k) {
                const float y = odd_value<E4M3>(a.c, at + k);
                if (!isfinite(y)) dst[k] += y;
            }
        }
    }
}

template <int D, bool E4M3, bool EXTRA>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_wide_kernel(const __grid_constant__ KernelArgs ka, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
    using S = Layout<D, E4M3>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const AttnArgs &a = ka.a;
    const Plan &p = ka.p;
    uint8_t *qt = smem, *ring = qt + 2 * S::kQ, *wide = ring + S::kSlots * S::kSlot;
    float *scales = reinterpret_cast<float *>(wide + 2 * S::kWide);  // [kScaleRing][kTile], e4m3
    float *q_factor = scales + kScaleRing * kTile;                    // [2][kGroupRows], e4m3
    Shared &sh = *reinterpret_cast<Shared *>(reinterpret_cast<uint8_t *>(scales) + S::kScale);
    Barriers &bar = sh.bar;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < S::kSlots; ++i) {
            bar_init(smem_addr(&bar.full[i]), 1);
            bar_init(smem_addr(&bar.empty[i]), 1);
        }
        for (int i = 0; i < kScaleRing; ++i) {
            bar_init(smem_addr(&bar.scale_full[i]), 2);
            bar_init(smem_addr(&bar.scale_empty[i]), 8);
        }
        for (int w = 0; w < 2; ++w) {
            bar_init(smem_addr(&bar.wide_full[w]), 1);
            bar_init(smem_addr(&bar.wide_empty[w]), 1);
            bar_init(smem_addr(&bar.o_full[w]), 1);
            bar_init(smem_addr(&bar.s_full[w]), 1);
            bar_init(smem_addr(&bar.p_half[w]), 4);
            bar_init(smem_addr(&bar.p_full[w]), 4);
        }
        bar_init(smem_addr(&bar.q_full), 8);
        bar_init(smem_addr(&bar.left), 8);
        bar_init(smem_addr(&bar.drained), 1);
        sh.dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_proxy();
    }
    if (warp == 9) tmem_alloc(smem_addr(&sh.tmem), 512);
    // Up to here this may run beside the kernel before it.
    asm volatile("griddepcontrol.wait;" ::: "memory");
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
    {
        // The first segment's query tiles: everyone takes a share.
        Walk ahead = walk;
        if (ahead.next(&g))
            for (int w = 0; w < (g.dual ? 2 : 1); ++w)
                stage_queries<D, E4M3>(a, g, g.row0 + w * kGroupRows, min(kGroupRows, g.rows - w * kGroupRows), kGroupRows,
                                       qt + w * S::kQ, q_factor + w * kGroupRows, tid, kAttnThreads);
        fence_async_proxy();
        __syncthreads();
    }

    if (warp == 8) {
        // ---- loads.  Alternating tiles: K0 K1 V0 K2 V1 ...; both groups on each
        // tile: K0 V0 K1 V1 ...
        Loader<D, E4M3, S::kSlots> load;
        PageIds key_ids, value_ids;
        int seg = 0;
        bool live = true;
        while (live && walk.next(&g)) {
            if (lane == 0) sh.fail[seg & 15] = sh.odd[seg & 15] = 0;
            __syncwarp();
            key_ids.begin(a, g);
            value_ids = key_ids;
            const int n = g.t1 - g.t0;
            int kt = 0, vt = 0;
            for (int i = 0; live && i < 2 * n; ++i) {
                const bool key = kt < n && (kt == vt || (!g.dual && kt == vt + 1));
                live = load.tile(a, g, key ? key_ids : value_ids, g.t0 + (key ? kt++ : vt++), key ? &kmap : &vmap, smem_addr(ring),
                                 bar.full, smem_addr(&bar.empty[load.slot]), dead, &sh.fail[seg & 15]);
            }
            ++seg;
        }
        if (!live) load.drain(bar.full);
    } else if (warp == 9) {
        // ---- products
        if (elect_one()) {
            using T = Shape<D, false>;  // the values as the product takes them
            constexpr uint32_t kQk = mma_desc(E4M3, kTile, false, false), kPv = mma_desc(false, D, false, true);
            constexpr uint32_t kHi = kMatrixHi<S::kRow>, kVHi = kMatrixHi<T::kRow>;
            uint32_t segs = 0, pn[2] = {0, 0}, vn = 0;
            uint32_t slot = 0, phase = 0;  // the ring, in the order it is filled
            bool live = true;
            const uint32_t q0 = matrix_lo(smem_addr(qt), 0), k0 = matrix_lo(smem_addr(ring), 0);
            const uint32_t v0 = matrix_lo(smem_addr(E4M3 ? wide : ring), T::kMat);
            const uint32_t full0 = smem_addr(&bar.full[0]), empty0 = smem_addr(&bar.empty[0]);
            const uint32_t s_full = smem_addr(&bar.s_full[0]), p_full = smem_addr(&bar.p_full[0]);
            const uint32_t p_half = smem_addr(&bar.p_half[0]);
            auto advance = [&] {
                if (++slot == S::kSlots) {
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
            // O += P V of group w with the value tile in slot (or wide buffer) s, of the positions of half z
            auto values = [&](uint32_t w, uint32_t s, uint32_t z, bool first) {
                const uint32_t v = v0 + s * (T::kSlot >> 4), d = tmem + 2 * kTile + w * D, pt = tmem + w * kTile;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_ts(d, pt + (4 * z + i) * 8, v + ((4 * z + i) * 16 * T::kRow >> 4), kVHi, kPv, i > 0 || !first);
            };
            while (live && walk.next(&g)) {
                const int n = g.t1 - g.t0, lead = g.dual ? 1 : min(2, n);
                live = bar_wait(smem_addr(&bar.q_full), segs & 1, dead);
                for (int t = 0; live && t < lead; ++t) {  // scores of each group's first tile
                    if (!(live = bar_wait(full0 + 8 * slot, phase, dead))) break;
                    fence_after_sync();
                    if (g.dual) {
                        scores(0, 0, slot);
                        mma_commit(s_full);
                        scores(1, 1, slot);
                        mma_commit(s_full + 8);
                    } else {
                        scores(t, 0, slot);
                        mma_commit(s_full + 8 * t);
                    }
                    mma_commit(empty0 + 8 * slot);
                    advance();
                }
                for (int t = 0; live && t < n; ++t, ++vn) {
                    // Over e4m3 the two helper warps take the tile from the ring.
                    const uint32_t vs = E4M3 ? vn & 1 : slot, vp = E4M3 ? (vn >> 1) & 1 : phase;
                    const uint32_t v_full = E4M3 ? smem_addr(&bar.wide_full[vs]) : full0 + 8 * vs;
                    const uint32_t v_empty = E4M3 ? smem_addr(&bar.wide_empty[vs]) : empty0 + 8 * vs;
                    advance();
                    const bool more = t + lead < n;
                    const uint32_t ks = slot, kp = phase;
                    if (more) advance();
                    if (!(live = bar_wait(v_full, vp, dead))) break;
                    const uint32_t w0 = g.dual ? 0 : t & 1, w1 = g.dual ? 1 : t & 1;
                    for (uint32_t w = w0; w <= w1; ++w) {
                        const uint32_t pp = pn[w]++ & 1;
                        if (!(live = bar_wait(p_half + 8 * w, pp, dead))) break;
                        fence_after_sync();
                        values(w, vs, 0, g.dual ? t == 0 : t < 2);
                        if (!(live = bar_wait(p_full + 8 * w, pp, dead))) break;
                        fence_after_sync();
                        values(w, vs, 1, false);
                        if (w == w1) mma_commit(v_empty);
                        if (!more) continue;
                        if (!(live = bar_wait(full0 + 8 * ks, kp, dead))) break;
                        scores(w, g.dual ? w : 0, ks);
                        mma_commit(s_full + 8 * w);
                        if (w == w1) mma_commit(empty0 + 8 * ks);
                    }
                }
                if (live) {
                    mma_commit(smem_addr(&bar.o_full[segs++ & 1]));
                }
            }
            if (!live) {  // products in flight end before TMEM is freed
                mma_commit(smem_addr(&bar.drained));
                bar_drain(smem_addr(&bar.drained), 0);
            }
        }
        __syncwarp();
    } else if (warp >= 10) {
        // ---- the e4m3 cache, a warp for each half of a tile's positions, two rows a
        // thread: 2^ek of every position, a tile ahead, and the value tile widened.
        // A thread's page ids are read three tiles ahead, its exponents two.
        if constexpr (E4M3) {
            const int half = warp - 10, row = half * 64 + lane;
            uint32_t n = 0, n_ring = 0, seg = 0;
            bool live = true;
            auto page_ids = [&](int t, int (&id)[2]) {
                for (int i = 0; i < 2; ++i) {
                    const int j = t * kTile + row + 32 * i;
                    id[i] = t < g.t1 && j < g.len ? pages_of(a, g)[j >> a.c.page_shift] : -1;
                    if (id[i] >= a.c.num_pages) id[i] = -1;
                }
            };
            auto exponents = [&](int t, const int (&id)[2], int (&e)[2][2]) {
                for (int i = 0; i < 2; ++i) {
                    const long long at =
                        cache_row(a.c, max(id[i], 0), g.h, (t * kTile + row + 32 * i) & ((1 << a.c.page_shift) - 1));
                    e[i][0] = id[i] < 0 ? 0 : a.c.k_exp[at];
                    e[i][1] = id[i] < 0 ? 0 : a.c.v_exp[at];
                }
            };
            auto factors = [&](uint32_t m, const int (&e)[2][2]) {
                const uint32_t s = m % kScaleRing;
                live = live && bar_wait(smem_addr(&bar.scale_empty[s]), ((m / kScaleRing) & 1) ^ 1, dead);
                live = __all_sync(0xffffffffu, live);
                for (int i = 0; i < 2; ++i) scales[s * kTile + row + 32 * i] = power_of(e[i][0]);
                __syncwarp();
                if (lane == 0) bar_arrive(smem_addr(&bar.scale_full[s]));
            };
            while (live && walk.next(&g)) {
                const int T = g.t1 - g.t0, last_pos = a.window > 0 ? last_position(a, g) : 0;
                int id[2], now[2][2], next[2][2], after[2][2];
                page_ids(g.t0, id);
                exponents(g.t0, id, now);
                page_ids(g.t0 + 1, id);
                factors(n, now);
                exponents(g.t0 + 1, id, next);
                page_ids(g.t0 + 2, id);
                for (int t = g.t0; t < g.t1; ++t, ++n) {
                    if (t + 1 < g.t1) factors(n + 1, next);
                    exponents(t + 2, id, after);
                    page_ids(t + 3, id);
                    const int idx = t - g.t0;
                    // The tile's slot as the loads number them.  The buffer is free once the product of
                    // the tile two before is over: all fills before the slot's present one then are.
                    const uint32_t vi = n_ring + (g.dual || idx == T - 1 ? 2 * idx + 1 : 2 * idx + 2);
                    live = live && bar_wait(smem_addr(&bar.wide_empty[n & 1]), ((n >> 1) & 1) ^ 1, dead) &&
                           bar_wait(smem_addr(&bar.full[vi % S::kSlots]), (vi / S::kSlots) & 1, dead);
                    if (live) {
                        const bool clean = !sees_whole(a, g, t * kTile, last_pos);
                        bool odd = false;
                        for (int i = 0; i < 2; ++i)
                            odd |= widen_values<D, 2>(ring + vi % S::kSlots * S::kSlot, wide + (n & 1) * S::kWide, row + 32 * i,
                                                      power_of(now[i][1]), t * kTile + row + 32 * i < g.len, clean);
                        if (odd) sh.odd[seg & 15] = 1;
                        fence_async_proxy();
                    }
                    __syncwarp();
                    // The two warps leave together: this barrier's wait has no bound of its own.
                    live = !any_of(kHelperBarrier, 64, !live);
                    if (!live) break;
                    if (warp == 10 && lane == 0) {
                        bar_arrive(smem_addr(&bar.empty[vi % S::kSlots]));
                        bar_arrive(smem_addr(&bar.wide_full[n & 1]));
                    }
                    for (int i = 0; i < 2; ++i)
                        for (int k = 0; k < 2; ++k) now[i][k] = next[i][k], next[i][k] = after[i][k];
                }
                n_ring += 2 * T;
                ++seg;
            }
        }
    } else if (warp < 8) {
        // ---- softmax groups
        const int w = warp >> 2, row = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // this warp's TMEM lanes
        const uint32_t st = tmem + lanes + w * kTile, ot = tmem + lanes + 2 * kTile + w * D;
        const float mul = (a.cap > 0.0f ? fabsf(a.scale) / a.cap : fabsf(a.scale) * kLog2e);
        uint32_t segs = 0, sn = 0, n_ring = 0, n_scale = 0;
        bool live = true, more = walk.next(&g);
        if (more && lane == 0) bar_arrive(smem_addr(&bar.q_full));  // the first segment's queries are there
        while (live && more) {
            const int T = g.t1 - g.t0, row0 = g.row0 + (g.dual ? w * kGroupRows : 0);
            const int rows = min(kGroupRows, g.rows - (g.dual ? w * kGroupRows : 0));
            const bool has = row < rows, active = (row & ~31) < rows;
            const int r = row0 + row, tok_in = has ? r / a.G : 0, head = g.h * a.G + (has ? r % a.G : 0);
            Row x;
            x.tok = g.shared ? tok_in : g.b * a.N + tok_in;
            x.b = g.shared ? (has ? x.tok / a.N : 0) : g.b;
            x.n = has ? x.tok - x.b * a.N : 0;
            x.first = (g.shared ? (has ? a.lens[x.b] : 0) : g.len) - a.N;
            x.pos_i = !has ? 0 : a.pos ? a.pos[x.tok] : a.shared_len + x.first + x.n;
            x.has = has;
            x.rs = mul;
            if (E4M3) {
                live = bar_wait(smem_addr(&bar.q_full), segs & 1, dead);
                live = __all_sync(0xffffffffu, live);
                if (!live) break;
                x.rs *= q_factor[(g.dual ? w : 0) * kGroupRows + row];
            }
            x.slope = EXTRA && a.slopes && has ? a.slopes[head] * kLog2e : 0.0f;
            x.m = kNegInf;
            x.l = 0.0f;
            const int last_pos = a.window > 0 ? last_position(a, g) : 0;
            bool wrote = false;
            for (int t = g.t0; t < g.t1; ++t) {
                const int idx = t - g.t0;
                if (!g.dual && (idx & 1) != w) continue;
                const int j0 = t * kTile;
                const bool whole = sees_whole(a, g, j0, last_pos);
                const uint32_t s_bar = smem_addr(&bar.s_full[w]), s_phase = sn++ & 1;
                // What the masks leave of the tile is told while its scores are on their way,
                // and its values cleaned.  (Where the tiles alternate, after the scores: only they
                // tell that the slot's fill before this one is over.)
                Seen seen;
                if (!whole) {
                    if (active)
                        seen = seen_columns(a.mask, a.pos, a.N, a.window, g.shared ? 0 : a.shared_len, g.shared, g.len, x.first,
                                            x.has, x.tok, x.b * a.N, x.pos_i, j0);
                    if constexpr (!E4M3) {
                        // the tile's values: slot index as the loads number them
                        const uint32_t vi = n_ring + (g.dual ? 2 * idx + 1 : idx == T - 1 ? 2 * idx + 1 : 2 * idx + 2);
                        if (!g.dual) live = bar_wait(s_bar, s_phase, dead);
                        live = live && bar_wait(smem_addr(&bar.full[vi % S::kSlots]), (vi / S::kSlots) & 1, dead);
                        live = __all_sync(0xffffffffu, live);
                        if (!live) break;
                        if (clean_values<D>(ring + vi % S::kSlots * S::kSlot, row, j0 + row < g.len)) sh.odd[segs & 15] = 1;
                        fence_async_proxy();
                    }
                }
                live = bar_wait(s_bar, s_phase, dead);
                const float *fa = nullptr;
                if (E4M3) {
                    const uint32_t s = (n_scale + idx) % kScaleRing;
                    live = live && bar_wait(smem_addr(&bar.scale_full[s]), ((n_scale + idx) / kScaleRing) & 1, dead);
                    fa = scales + s * kTile;
                }
                live = __all_sync(0xffffffffu, live);
                if (!live) break;
                fence_after_sync();
                if (active)
                    softmax_tile<D, E4M3, EXTRA>(a, g, x, j0, whole, wrote, st, ot, fa, seen, smem_addr(&bar.p_half[w]));
                else if (lane == 0)
                    bar_arrive(smem_addr(&bar.p_half[w]));
                wrote = true;
                fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(smem_addr(&bar.p_full[w]));
                    if (E4M3) bar_arrive(smem_addr(&bar.scale_empty[(n_scale + idx) % kScaleRing]), g.dual ? 1 : 2);
                }
            }
            if (!live) break;
            Segment next;  // found while the last products run
            more = walk.next(&next);
            live = bar_wait(smem_addr(&bar.o_full[segs & 1]), (segs >> 1) & 1, dead);
            live = __all_sync(0xffffffffu, live);
            if (!live) break;
            fence_after_sync();
            // ---- the group's partial result of the segment
            const Units &k = g.shared ? p.shared : p.own;
            const long long at = (static_cast<long long>(g.slot) * 2 + w) * k.rc + row;
            const bool failed = reinterpret_cast<volatile int *>(sh.fail)[segs & 15] != 0;
            const bool odd = reinterpret_cast<volatile int *>(sh.odd)[segs & 15] != 0;
            if (has)
                k.ml[at] = make_float2(x.m, failed ? NAN : x.l);
            if (active && wrote) {
                // Rows go out through this warp's part of the query tile's memory (its
                // products are done), so that a store instruction covers whole lines.
                constexpr int kCols = S::kQ >= 32768 ? 32 : 16, kQuads = kCols / 4;
                float4 *buf = reinterpret_cast<float4 *>(qt + (g.dual ? w : 0) * S::kQ) +
                              (g.dual ? warp & 3 : warp) * 32 * kQuads;
                float *o = k.o + (at - lane) * D;  // the warp's first row
                const int n = min(32, rows - (row & ~31));
#pragma unroll 1
                for (int c = 0; c < D; c += kCols) {
                    float v[kCols];
                    if constexpr (kCols == 32)
                        tmem_load32(ot + c, v);
                    else
                        tmem_load16(ot + c, v);
                    tmem_load_wait();
#pragma unroll
                    for (int i = 0; i < kQuads; ++i)
                        buf[lane * kQuads + (i ^ (lane & (kQuads - 1)))] =
                            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    __syncwarp();
#pragma unroll
                    for (int i = lane; i < 32 * kQuads; i += 32) {
                        const int r = i / kQuads, q = i % kQuads;
                        if (r < n)
                            *reinterpret_cast<float4 *>(o + static_cast<long long>(r) * D + c + 4 * q) =
                                buf[r * kQuads + (q ^ (r & (kQuads - 1)))];
                    }
                    __syncwarp();
                }
                if (odd && has)
                    for (int c = 0; c < D; c += 32) add_odd_values<D, E4M3>(a, g, x, c, k.o + at * D + c);
                __syncwarp();
            }
            fence_before_sync();
            // ---- the next segment's query tiles, once all have left this one's
            __syncwarp();
            if (lane == 0) bar_arrive(smem_addr(&bar.left));
            if (more) {
                live = bar_wait(smem_addr(&bar.left), segs & 1, dead);
                live = __all_sync(0xffffffffu, live);
                if (!live) break;
                if (next.dual) {
                    stage_queries<D, E4M3>(a, next, next.row0 + w * kGroupRows,
                                           min(kGroupRows, next.rows - w * kGroupRows), kGroupRows, qt + w * S::kQ,
                                           q_factor + w * kGroupRows, row, 128);
                } else {
                    stage_queries<D, E4M3>(a, next, next.row0, next.rows, kGroupRows, qt, q_factor, tid, 256);
                }
                fence_async_proxy();
                __syncwarp();
                if (lane == 0) bar_arrive(smem_addr(&bar.q_full));
            }
            ++segs;
            n_ring += 2 * T;
            n_scale += T;
            g = next;
        }
        if (!live && tid == 0) atomicOr(a.err, static_cast<uint32_t>(SPEC_DATA_STALL));
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 9) tmem_free(tmem, 512);
}

template <int D, bool E4M3, bool EXTRA>
int launch_shape(KernelArgs &ka, int grid, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
    static int done[64];
    auto kernel = attn_wide_kernel<D, E4M3, EXTRA>;
    if (!allow_smem(kernel, Layout<D, E4M3>::kBytes, done)) return SPEC_ERR_CUDA;
    return launch_early(kernel, dim3(grid), dim3(kAttnThreads), Layout<D, E4M3>::kBytes, st, ka, kmap, vmap)
               ? SPEC_OK
               : SPEC_ERR_CUDA;
}

}  // namespace

int launch_wide(KernelArgs &ka, int grid, const CUtensorMap &kmap, const CUtensorMap &vmap, cudaStream_t st) {
    const bool extra = ka.a.cap > 0.0f || ka.a.slopes, wide = ka.a.c.D == 128;
    if (ka.a.c.e4m3)
        return extra ? (wide ? launch_shape<128, true, true>(ka, grid, kmap, vmap, st)
                             : launch_shape<64, true, true>(ka, grid, kmap, vmap, st))
                     : (wide ? launch_shape<128, true, false>(ka, grid, kmap, vmap, st)
                             : launch_shape<64, true, false>(ka, grid, kmap, vmap, st));
    return extra ? (wide ? launch_shape<128, false, true>(ka, grid, kmap, vmap, st)
                         : launch_shape<64, false, true>(ka, grid, kmap, vmap, st))
                 : (wide ? launch_shape<128, false, false>(ka, grid, kmap, vmap, st)
                         : launch_shape<64, false, false>(ka, grid, kmap, vmap, st));
}

}  // namespace specv
