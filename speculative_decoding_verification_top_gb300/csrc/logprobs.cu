// logprobs.cu -- log probabilities of emitted tokens, the rows' entropies and
// their most likely tokens, in one pass over each row.
//
// With c = log2(e) / T and m near the row's largest logit, y_v = (l_v - m) c:
//   Z = sum 2^y,  A = sum 2^y y;
//   ln p(x) = (l_x - m) / T - ln Z,  entropy = ln 2 (log2 Z - A / Z).
// The order of tokens is by key: the logit's ordered bits above the index's
// complement, so that keys differ and equal logits go by index.
//
// A row is cut into slices, one per CTA of a cluster; a CTA goes through its slice
// in chunks of 10240 vectors of 16 bytes: the sums, the count of tokens before the
// emitted one, and each vector's maximum.  The chunk's candidates for the slice's
// `top` first come from the vectors (read once more, from L2) whose maximum is from
// a bar on: the top-th of what was seen before or, in the first chunk, the top-th
// largest of 64 groups' maxima (at least `top` elements reach it, and few more do).
// The slices' sums and lists meet in the first CTA's shared memory.
// Bound by what is issued for the sums (21 of 25 to 28 us; some 10 instructions an
// element) and by the chain bar, candidates, order, cluster after them.
// Measured: 64 x 6 entries (228 emitted) of 151936 bf16 logits, 20 alternatives, 25 to
// 28 us (69 MB, 2.5 to 2.8 TB/s), fp32 39 to 45 us (3.1 to 3.6); without alternatives
// 21.  Held in registers
// instead, a slice cut into chunks of 2048 vectors took 120 us, and of 2560 in three
// CTAs a multiprocessor 70: each chunk's selection is a chain of barriers.  A thread's
// maxima looked through one by one cost 9000 of 45000 cycles.

#include "logprobs.cuh"
#include "util.cuh"

namespace specv {
namespace {

using Key = unsigned long long;

constexpr int kVecs = 40;              // vectors a thread takes of a chunk
constexpr int kBatch = 4;              // of them at a time, the next ones in flight
constexpr int kChunk = kThreads * kVecs;
constexpr int kGroups = kThreads / 4;  // groups of threads whose maxima bound the first chunk
constexpr int kQueue = 512;            // vectors of a chunk that may hold candidates
constexpr int kCap = 1024;             // candidates kept of a chunk
constexpr int kTies = SPEC_MAX_TOP * 8;  // equal ones among them that are taken at a time, at most
constexpr int kMaxCluster = 8;
constexpr int kResident = 3;           // CTAs a multiprocessor has room for
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFar = -200.0f;        // 2^y is 0 from here down

struct Part {        // one slice's sums
    float m, z, a;   // reference, sum 2^y, sum 2^y y
    uint32_t before; // tokens before the emitted one
    uint32_t bad;    // kFlagNonFinite, or 0
};

struct Shared {
    Part part[kMaxCluster];              // in the first CTA: all slices'
    Key list[kMaxCluster][SPEC_MAX_TOP]; // in the first CTA: their `top` first keys, sorted, then 0
    Key mine[SPEC_MAX_TOP];              // this slice's so far, sorted
    Key cand[kCap];
    Key best[kWarps];
    alignas(16) uint16_t top[kThreads][kVecs];  // the chunk's vectors' maxima (up_bits), a thread's side by side
    uint16_t queue[kQueue];
    float group[kGroups];
    Part warp[kWarps];
    uint32_t ties[kWarps];
    uint32_t n, n_mine, n_queue;
    float bound;
};

__device__ __forceinline__ Key key_of(float v, int index) {
    return static_cast<Key>(okey<float>(v)) << 32 | static_cast<uint32_t>(~index);
}

__device__ __forceinline__ Key max_key(Key a, Key b) { return a > b ? a : b; }

// A vector of which elements [at, at + E) some lie outside the row: those are not
// read, and -inf.
template <typename T>
__device__ __noinline__ uint4 edge_vec(const T *row, int at, int V) {
    constexpr int E = Elem<T>::kPerVec;
    uint32_t w[4] = {Elem<T>::kNegInfWord, Elem<T>::kNegInfWord, Elem<T>::kNegInfWord, Elem<T>::kNegInfWord};
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if (at + i < 0 || at + i >= V) continue;
        if constexpr (sizeof(T) == 4)
            w[i] = __float_as_uint(row[at + i]);
        else
            w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | static_cast<uint32_t>(row[at + i]) << 16
                             : (w[i / 2] & 0xffff0000u) | row[at + i];
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A row's vectors lie on 16-byte boundaries: the first starts up to `head`
// elements before the row.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T *row, int at, int V) {
    if (at >= 0 && at + Elem<T>::kPerVec <= V) return ld_stream(row + at);
    return edge_vec(row, at, V);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// A shared-memory address of this CTA, in the cluster's first CTA.
template <typename X>
__device__ __forceinline__ X *remote(X *p) {
    X *r;
    asm("mapa.u64 %0, %1, 0;" : "=l"(r) : "l"(p));
    return r;
}

// The largest float below a finite x.
__device__ __forceinline__ float below(float x) {
    const int u = __float_as_int(x);
    return x == 0.0f ? __int_as_float(static_cast<int>(0x80000001u)) : __int_as_float(u + (u < 0 ? 1 : -1));
}

// The smallest float above x; +inf above the largest finite one.
__device__ __forceinline__ float above(float x) { return -below(-x); }

// x in 16 bits, rounded up (a bf16 as it is), and back.
__device__ __forceinline__ uint16_t up_bits(float x) {
    const uint32_t u = __float_as_uint(x);
    return static_cast<uint16_t>((u + (u >> 31 ? 0u : 0xffffu)) >> 16);
}

__device__ __forceinline__ float of_bits(uint16_t u) { return __uint_as_float(static_cast<uint32_t>(u) << 16); }

// The token whose rank is counted.
struct Emitted {
    int id;
    float logit, under;  // under: the largest float below the logit

    // How many of a vector's elements, from index `at` on, come before it: those
    // above its logit, and equal ones ahead of it.
    template <typename T>
    __device__ __forceinline__ uint32_t before(const uint4 &q, int at, int end) const {
        constexpr int E = Elem<T>::kPerVec;
        float f[E];
        unpack<T>(q, f);
        uint32_t n = 0;
        if (logit == kNegInf || (at <= id && id < at + E)) {
#pragma unroll
            for (int k = 0; k < E; ++k) n += f[k] > logit || (f[k] == logit && at + k >= 0 && at + k < min(id, end));
        } else {
            const float bar = at < id ? under : logit;
#pragma unroll
            for (int k = 0; k < E; ++k) n += f[k] > bar;
        }
        return n;
    }
};

// The row as vectors, and the slice's end.
template <typename T>
struct Slice {
    const T *row;
    int head, V, end;  // end: first element past the slice (and the row)

    __device__ __forceinline__ int at(int vec) const { return vec * Elem<T>::kPerVec - head; }

    // fn(element, key) of a vector's elements from `bar` on whose keys are above `least`.
    template <typename Fn>
    __device__ __forceinline__ void from(int vec, float bar, Key least, Fn fn) const {
        constexpr int E = Elem<T>::kPerVec;
        float f[E];
        unpack<T>(load_vec(row, at(vec), V), f);
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const int x = at(vec) + k;
            if (!(f[k] >= bar) || x < 0 || x >= end) continue;
            const Key y = key_of(f[k], x);
            if (y > least) fn(y);
        }
    }
};

// Brings the slice's list sh.mine up to date with the chunk from vector v on, of
// which a thread took `count`, with maximum `most`.  All threads call it; contains
// block barriers, the last thing it does is one.
template <typename T>
__device__ __forceinline__ void take_first(Shared &sh, const Slice<T> &slice, int v, int count, float most, int top) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int held = static_cast<int>(sh.n_mine);  // the last barrier was after its write
    float bar;
    Key least = 0;  // keys above it are candidates
    if (tid < held) sh.cand[tid] = sh.mine[tid];
    if (tid == 0) {
        sh.n = held;
        sh.n_queue = 0;
    }
    if (held < top) {
        float g = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
        if (lane % 4 == 0) sh.group[tid / 4] = g;
        if (tid == 0) sh.bound = kNegInf;
        __syncthreads();
        // Four threads count for a group: those above it, and equal ones ahead of it.
        const float x = sh.group[tid / 4];
        int n = 0;
#pragma unroll 4
        for (int i = 0; i < kGroups / 4; ++i) {
            const int j = i * 4 + tid % 4;
            const float y = sh.group[j];
            n += y > x || (y == x && j < tid / 4);
        }
        n += __shfl_xor_sync(0xffffffffu, n, 1);
        n += __shfl_xor_sync(0xffffffffu, n, 2);
        if (n == top - 1) sh.bound = x;
        __syncthreads();
        bar = sh.bound;
    } else {
        least = sh.mine[top - 1];
        bar = key_float(static_cast<uint32_t>(least >> 32));
        __syncthreads();
    }
    // Candidates: the elements from the bar on, or (where equal logits make those too
    // many, as in a masked row) above it, then equal ones by index until there are
    // `top`.
    bool fits = false, ties = false;
#pragma unroll 1
    for (int pass = 0; pass < 2 && !fits; ++pass) {
        ties = pass == 1;
        if (ties) {
            __syncthreads();
            if (tid == 0) {
                sh.n = held;
                sh.n_queue = 0;
            }
            __syncthreads();
        }
        const float from = ties ? above(bar) : bar;
        if (most >= from) {
#pragma unroll 1
            for (int i = 0; i < count; i += 8) {
                const uint4 u = *reinterpret_cast<const uint4 *>(&sh.top[tid][i]);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                uint32_t hits = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    hits |= (__uint_as_float(w[k] << 16) >= from ? 1u : 0u) << 2 * k |
                            (__uint_as_float(w[k] & 0xffff0000u) >= from ? 2u : 0u) << 2 * k;
                for (hits &= first_bits(count - i); hits; hits &= hits - 1) {
                    const uint32_t n = atomicAdd(&sh.n_queue, 1);
                    if (n < kQueue) sh.queue[n] = static_cast<uint16_t>((i + __ffs(hits) - 1) * kThreads + tid);
                }
            }
        }
        __syncthreads();
        const int vecs = static_cast<int>(sh.n_queue);
        if (vecs <= kQueue) {
            constexpr int E = Elem<T>::kPerVec;  // a thread an element
#pragma unroll 1
            for (int i = tid; i < vecs * E; i += kThreads) {
                const int x = slice.at(v + sh.queue[i / E]) + i % E;
                if (x < 0 || x >= slice.end) continue;
                const float f = to_f32(slice.row[x]);
                const Key k = key_of(f, x);
                if (!(f >= from) || k <= least) continue;
                const uint32_t n = atomicAdd(&sh.n, 1);
                if (n < kCap) sh.cand[n] = k;
            }
        }
        __syncthreads();
        fits = vecs <= kQueue && static_cast<int>(sh.n) <= (ties ? kCap - kTies : kCap);
    }
    if (fits && ties) {
        const uint32_t equal = okey<float>(bar);
#pragma unroll 1
        for (int i = 0; i < count && static_cast<int>(sh.n) < top; ++i) {  // sh.n as the last barrier left it
            const bool near = of_bits(sh.top[tid][i]) >= bar;
            bool some = false;
            if (near)
                slice.from(v + i * kThreads + tid, bar, least, [&](Key k) { some |= static_cast<uint32_t>(k >> 32) == equal; });
            const uint32_t mask = __ballot_sync(0xffffffffu, some);
            if (lane == 0) sh.ties[warp] = static_cast<uint32_t>(__popc(mask));
            __syncthreads();
            int place = __popc(mask & ((1u << lane) - 1u));
            for (int w = 0; w < warp; ++w) place += static_cast<int>(sh.ties[w]);
            if (some && place < top)  // the first `top` threads with any: by index
                slice.from(v + i * kThreads + tid, bar, least, [&](Key k) {
                    if (static_cast<uint32_t>(k >> 32) == equal) sh.cand[atomicAdd(&sh.n, 1)] = k;
                });
            __syncthreads();
        }
    }
    if (fits) {
        const int n = static_cast<int>(sh.n);
        for (int i = tid; i < n; i += kThreads) {
            const Key x = sh.cand[i];
            int place = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) place += sh.cand[j] > x;
            if (place < top) sh.mine[place] = x;
        }
        if (tid == 0) sh.n_mine = min(n, top);
        __syncthreads();
        return;
    }
    // Too many above the bar: the first `top` of list and chunk one by one.
    const Key old = tid < held ? sh.mine[tid] : 0;
    Key last = ~0ull;
    int k = 0;
#pragma unroll 1
    for (; k < top; ++k) {
        Key best = old < last ? old : 0;
#pragma unroll 1
        for (int i = 0; i < count; ++i) {
            if (!(of_bits(sh.top[tid][i]) >= bar)) continue;
            slice.from(v + i * kThreads + tid, bar, 0, [&](Key y) {
                if (y < last) best = max_key(best, y);
            });
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2) best = max_key(best, __shfl_xor_sync(0xffffffffu, best, o));
        __syncthreads();
        if (lane == 0) sh.best[warp] = best;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) best = max_key(best, sh.best[w]);
        if (best == 0) break;
        last = best;
        if (tid == 0) sh.mine[k] = best;
    }
    if (tid == 0) sh.n_mine = k;
    __syncthreads();
}

// Adds one part's sums to another's.
__device__ __forceinline__ void join_part(Part &p, const Part &x, float c) {
    const float top = fmaxf(p.m, x.m);
    const float y0 = p.m == kNegInf ? kFar : fmaxf((p.m - top) * c, kFar), k0 = ex2(y0);
    const float y1 = x.m == kNegInf ? kFar : fmaxf((x.m - top) * c, kFar), k1 = ex2(y1);
    p.a = k0 * fmaf(p.z, y0, p.a) + k1 * fmaf(x.z, y1, x.a);
    p.z = k0 * p.z + k1 * x.z;
    p.m = top;
    p.before += x.before;
    p.bad |= x.bad;
}

// SOME: top > 0.
template <typename T, bool SOME>
__global__ void __launch_bounds__(kThreads, kResident) logprobs_kernel(const LogprobArgs a) {
    started_early();
    constexpr int E = Elem<T>::kPerVec;
    __shared__ Shared sh;
    const int size = a.cluster, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t entry = blockIdx.x / static_cast<uint32_t>(size);
    const int rank = static_cast<int>(blockIdx.x - entry * size);
    const int b = static_cast<int>(entry / a.M), t = static_cast<int>(entry - static_cast<uint32_t>(b) * a.M);
    const int token = a.tokens[entry];
    const int r = a.rows && token != -1 ? a.rows[entry] : t;
    if (token < 0 || token >= a.V || r < 0 || r >= a.N) {  // the whole cluster alike
        if (rank) return;
        const float x = token == -1 ? 0.0f : NAN;
        if (tid == 0) {
            a.logprob[entry] = x;
            if (a.entropy) a.entropy[entry] = x;
            if (a.rank) a.rank[entry] = -1;
            if (token != -1) atomicOr(a.err, static_cast<uint32_t>(SPEC_DATA_TOKEN_RANGE));
        }
        if (SOME && tid < a.top) {
            a.top_ids[static_cast<long long>(entry) * a.top + tid] = -1;
            a.top_logprobs[static_cast<long long>(entry) * a.top + tid] = x;
        }
        return;
    }
    cluster_arrive();  // the first CTA is there before its memory is written
    const T *row = static_cast<const T *>(a.logits) + (static_cast<long long>(b) * a.N + r) * a.V;
    const int head = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int vecs = (head + a.V + E - 1) / E, per = (vecs + size - 1) / size;
    const int v0 = min(vecs, rank * per), v1 = min(vecs, v0 + per);
    const float c = a.c;
    float m = kNegInf;
    F2 z = pair_of(0.0f, 0.0f), s = z;
    const F2 c2 = pair_of(c, c);
    // Vectors [inner0, inner1) of the slice lie in the row whole.
    const int inner0 = head > 0 && v0 == 0 ? 1 : v0, inner1 = min(v1, (head + a.V) / E);
    uint32_t before = 0;
    bool odd = false;
    const Slice<T> slice = {row, head, a.V, min(a.V, v1 * E - head)};
    uint4 next[kBatch];
    auto batch = [&](int from, uint4 (&q)[kBatch]) {  // vectors from + i kThreads + tid
        if (from >= inner0 && min(v1, from + kBatch * kThreads) <= inner1) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                q[i] = neg_inf_vec<T>();
                if (from + i * kThreads + tid < v1) q[i] = ld_stream(row + slice.at(from + i * kThreads + tid));
            }
        } else {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int x = from + i * kThreads + tid;
                q[i] = x < v1 ? load_vec(row, slice.at(x), a.V) : neg_inf_vec<T>();
            }
        }
    };
    batch(v0, next);  // on its way while the token's own logit is fetched
    const float lt = to_f32(row[token]);
    const Emitted emitted = {token, lt, lt == kNegInf ? kNegInf : below(lt)};
    if (SOME) {
        if (tid == 0) sh.n_mine = 0;
        __syncthreads();
    }
#pragma unroll 1
    for (int v = v0; v < v1; v += kChunk) {
        float most = kNegInf;  // of the chunk
        int count = 0;
        const int until = min(v1, v + kChunk);
        uint4 q[kBatch];
#pragma unroll 1
        for (; v + count * kThreads < until; count += kBatch) {
            const int first = v + count * kThreads + tid;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) q[i] = next[i];
            if (v + (count + kBatch) * kThreads < v1) batch(v + (count + kBatch) * kThreads, next);
            float tops[kBatch], top = kNegInf;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                tops[i] = batch_max1<T>(q[i]);
                top = max_nan(top, tops[i]);
            }
            if (SOME) {
                static_assert(kBatch == 4, "a batch's maxima are one store");
                *reinterpret_cast<uint2 *>(&sh.top[tid][count]) =
                    make_uint2(up_bits(tops[0]) | static_cast<uint32_t>(up_bits(tops[1])) << 16,
                               up_bits(tops[2]) | static_cast<uint32_t>(up_bits(tops[3])) << 16);
            }
            odd |= !(top < INFINITY);
            most = fmaxf(most, top);
            // ---- sums, against this thread's own reference
            if (top > m) {
                const float y = m == kNegInf ? kFar : fmaxf((m - top) * c, kFar), keep = ex2(y);
                s = mul2(pair_of(keep, keep), fma2(z, pair_of(y, y), s));
                z = mul2(pair_of(keep, keep), z);
                m = top;
            }
            const float ref = m == kNegInf ? 0.0f : m;
            const F2 ref2 = pair_of(-ref, -ref);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                float f[E];
                unpack<T>(q[i], f);
#pragma unroll
                for (int k = 0; k < E; k += 2) {
                    const float2 y = parts_of(mul2(add2(pair_of(f[k], f[k + 1]), ref2), c2));
                    const F2 y2 = pair_of(fmaxf(y.x, kFar), fmaxf(y.y, kFar));
                    const F2 e = pair_of(ex2(parts_of(y2).x), ex2(parts_of(y2).y));
                    z = add2(z, e);
                    s = fma2(e, y2, s);
                }
            }
            if (top >= lt) {
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (tops[i] >= lt) before += emitted.before<T>(q[i], slice.at(first + i * kThreads), slice.end);
            }
        }
        if (SOME) take_first<T>(sh, slice, v, count, most, a.top);
    }
    // ---- the slice's sums
    Part mine = {m, parts_of(z).x + parts_of(z).y, parts_of(s).x + parts_of(s).y, __reduce_add_sync(0xffffffffu, before),
                 __any_sync(0xffffffffu, odd) ? kFlagNonFinite : 0u};
#pragma unroll
    for (int o = 16; o > 0; o /= 2) mine.m = fmaxf(mine.m, __shfl_xor_sync(0xffffffffu, mine.m, o));
    {
        const float y = m == kNegInf ? kFar : fmaxf((m - mine.m) * c, kFar), keep = ex2(y);
        mine.a = keep * fmaf(mine.z, y, mine.a);
        mine.z *= keep;
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        mine.z += __shfl_xor_sync(0xffffffffu, mine.z, o);
        mine.a += __shfl_xor_sync(0xffffffffu, mine.a, o);
    }
    if (lane == 0) sh.warp[warp] = mine;
    __syncthreads();
    cluster_wait();
    if (tid == 0) {
        Part p = sh.warp[0];
        for (int w = 1; w < kWarps; ++w) join_part(p, sh.warp[w], c);
        *remote(&sh.part[rank]) = p;
    }
    if (SOME && tid < a.top) *remote(&sh.list[rank][tid]) = tid < static_cast<int>(sh.n_mine) ? sh.mine[tid] : 0;
    cluster_arrive();
    cluster_wait();
    if (rank) return;
    // ---- the row
    Part p = sh.part[0];
    for (int i = 1; i < size; ++i) join_part(p, sh.part[i], c);
    const float R = p.m, Z = p.z, A = p.a;
    const uint32_t bad = p.bad ? p.bad : R == kNegInf ? kFlagAllNegInf : 0u;
    const float lz = log2f(Z);
    if (tid == 0) {
        if (bad) atomicOr(a.err, bad);
        a.logprob[entry] = bad ? NAN : (lt - R) * a.inv_t - kLn2 * lz;
        if (a.entropy) a.entropy[entry] = bad ? NAN : kLn2 * (lz - A / Z);
        if (a.rank) a.rank[entry] = bad ? -1 : static_cast<int32_t>(p.before);
    }
    if (!SOME) return;
    if (bad) {
        if (tid < a.top) {
            a.top_ids[static_cast<long long>(entry) * a.top + tid] = -1;
            a.top_logprobs[static_cast<long long>(entry) * a.top + tid] = NAN;
        }
        return;
    }
    for (int i = tid; i < size * a.top; i += kThreads) {
        const int of = i / a.top;
        const Key x = sh.list[of][i - of * a.top];
        int k = i - of * a.top;  // its place: after the keys above it in its own list and in the others
        for (int j = 0; j < size && k < a.top; ++j) {
            if (j == of) continue;
            for (int e = 0; e < a.top && sh.list[j][e] > x; ++e) ++k;
        }
        if (k >= a.top || x == 0) continue;
        a.top_ids[static_cast<long long>(entry) * a.top + k] = static_cast<int32_t>(~static_cast<uint32_t>(x));
        a.top_logprobs[static_cast<long long>(entry) * a.top + k] = (key_float(static_cast<uint32_t>(x >> 32)) - R) * a.inv_t - kLn2 * lz;
    }
}

template <typename T, bool SOME>
int launch_size(const LogprobArgs &a, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(a.B) * a.M * a.cluster);
    return launch_early_clusters(logprobs_kernel<T, SOME>, a.cluster, grid, dim3(kThreads), 0, st, a) ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

int launch_logprobs(LogprobArgs &a, int dtype, cudaStream_t st) {
    // As many CTAs a row as are resident at once: fewer leave multiprocessors idle, more
    // go through the chain in turns (384 rows of 151936, 20 alternatives: 25 to 28 us
    // with 2, 37 with 1, 34 with 4, 53 with 8).
    const int E = dtype == SPEC_F32 ? 4 : 8;
    const long long entries = static_cast<long long>(a.B) * a.M;
    a.cluster = 1;
    while (a.cluster < kMaxCluster && a.V > a.cluster * kThreads * E && entries * a.cluster < 152 * kResident) a.cluster *= 2;
    if (dtype == SPEC_F32) return a.top ? launch_size<float, true>(a, st) : launch_size<float, false>(a, st);
    return a.top ? launch_size<uint16_t, true>(a, st) : launch_size<uint16_t, false>(a, st);
}

}  // namespace specv
