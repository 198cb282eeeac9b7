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
// in chunks of 2048 vectors of 16 bytes that it holds in registers: the sums, the
// count of tokens before the emitted one, and the chunk's candidates for the
// slice's `top` first: those above the top-th of what was seen before or, in the
// first chunk, from the top-th largest of 64 groups' maxima on (at least `top`
// elements reach it, and few more do).  The slices' sums and lists meet in the
// first CTA's shared memory.

#include "logprobs.cuh"

namespace specv {
namespace {

using Key = unsigned long long;

constexpr int kVecs = 10;              // vectors a thread holds of a chunk
constexpr int kChunk = kThreads * kVecs;
constexpr int kGroups = kThreads / 4;  // groups of threads whose maxima bound the first chunk
constexpr int kCap = 1024;             // candidates kept of a chunk
constexpr int kMaxCluster = 8;
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
    float group[kGroups];
    float warp[3][kWarps];
    uint32_t before[kWarps];
    uint32_t bad, n, n_mine;
    float bound;
};

__device__ __forceinline__ Key key_of(float v, int index) {
    return static_cast<Key>(okey<float>(v)) << 32 | static_cast<uint32_t>(~index);
}

__device__ __forceinline__ Key max_key(Key a, Key b) { return a > b ? a : b; }

// The largest float below a finite x.
__device__ __forceinline__ float below(float x) {
    const int u = __float_as_int(x);
    return x == 0.0f ? __int_as_float(static_cast<int>(0x80000001u)) : __int_as_float(u + (u < 0 ? 1 : -1));
}

// A row's vectors lie on 16-byte boundaries: the first starts up to `head`
// elements before the row.  What lies outside the row is not read, and -inf.
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T *row, int at, int V) {
    constexpr int E = Elem<T>::kPerVec;
    if (at >= 0 && at + E <= V) return ld_stream(row + at);
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

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// A shared-memory address of this CTA, in the cluster's first CTA.
template <typename X>
__device__ __forceinline__ X *remote(X *p) {
    X *r;
    asm("mapa.u64 %0, %1, 0;" : "=l"(r) : "l"(p));
    return r;
}

// What a thread holds of a chunk.
template <typename T>
struct Held {
    uint4 q[kVecs];
    float top[kVecs];  // the vectors' maxima
    int at;            // index of vector 0's first element; the others follow kThreads vectors apart
    int end;           // first index past the slice (and the row)

    // fn(element, index) of those from `bar` on.
    template <typename Fn>
    __device__ __forceinline__ void from(float bar, Fn fn) const {
        constexpr int E = Elem<T>::kPerVec;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            if (!(top[i] >= bar)) continue;
            uint4 u = q[i];
            // Unpacked anew: kept from the sums, the floats would take 100 registers more.
            asm volatile("" : "+r"(u.x), "+r"(u.y), "+r"(u.z), "+r"(u.w));
            float f[E];
            unpack<T>(u, f);
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const int x = at + i * kThreads * E + k;
                if (f[k] >= bar && x >= 0 && x < end) fn(f[k], x);
            }
        }
    }
};

// Brings the slice's list sh.mine up to date with a chunk.  All threads call it;
// contains block barriers, the last thing it does is one.
template <typename T>
__device__ __forceinline__ void take_first(Shared &sh, const Held<T> &h, float most, int top) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int held = static_cast<int>(sh.n_mine);  // the last barrier was after its write
    float bar;
    Key least = 0;  // keys above it are candidates
    if (held < top) {
        float g = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
        if (lane % 4 == 0) sh.group[tid / 4] = g;
        if (tid == 0) sh.bound = kNegInf;
        __syncthreads();
        if (tid < kGroups) {
            const float x = sh.group[tid];
            int n = 0;
#pragma unroll 8
            for (int j = 0; j < kGroups; ++j) {
                const float y = sh.group[j];
                n += y > x || (y == x && j < tid);
            }
            if (n == top - 1) sh.bound = x;
        }
        if (tid < held) sh.cand[tid] = sh.mine[tid];
        if (tid == 0) sh.n = held;
        __syncthreads();
        bar = sh.bound;
    } else {
        least = sh.mine[top - 1];
        bar = key_float(static_cast<uint32_t>(least >> 32));
        if (tid < held) sh.cand[tid] = sh.mine[tid];
        if (tid == 0) sh.n = held;
        __syncthreads();
    }
    if (most >= bar)
        h.from(bar, [&](float v, int x) {
            const Key k = key_of(v, x);
            if (k <= least) return;
            const uint32_t n = atomicAdd(&sh.n, 1);
            if (n < kCap) sh.cand[n] = k;
        });
    __syncthreads();
    const int n = static_cast<int>(sh.n);
    if (n <= kCap) {
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
    // Too many at once (equal logits): the first `top` of list and chunk one by one.
    const Key old = tid < held ? sh.mine[tid] : 0;
    Key last = ~0ull;
    int k = 0;
    for (; k < top; ++k) {
        Key best = old < last ? old : 0;
        if (most >= bar)
            h.from(bar, [&](float v, int x) {
                const Key y = key_of(v, x);
                if (y < last) best = max_key(best, y);
            });
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

// SOME: top > 0.
template <typename T, bool SOME>
__global__ void __launch_bounds__(kThreads, 3) logprobs_kernel(const LogprobArgs a) {
    constexpr int E = Elem<T>::kPerVec;
    __shared__ Shared sh;
    const int size = a.cluster, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long entry = blockIdx.x / static_cast<unsigned>(size);
    const int rank = static_cast<int>(blockIdx.x - entry * size);
    const int b = static_cast<int>(entry / a.M), t = static_cast<int>(entry - static_cast<long long>(b) * a.M);
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
            a.top_ids[entry * a.top + tid] = -1;
            a.top_logprobs[entry * a.top + tid] = x;
        }
        return;
    }
    cluster_arrive();  // the first CTA is there before its memory is written
    const T *row = static_cast<const T *>(a.logits) + (static_cast<long long>(b) * a.N + r) * a.V;
    const int head = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int vecs = (head + a.V + E - 1) / E, per = (vecs + size - 1) / size;
    const int v0 = min(vecs, rank * per), v1 = min(vecs, v0 + per);
    const float lt = to_f32(row[token]), c = a.c;
    // An element before the token comes before it from lt on, one after it above lt.
    const bool lowest = lt == kNegInf;
    const float under = lowest ? kNegInf : below(lt);
    float m = kNegInf;
    float2 z = make_float2(0.0f, 0.0f), s = z;
    uint32_t before = 0;
    bool odd = false;
    if (tid == 0) sh.n_mine = sh.bad = 0;
    __syncthreads();
    for (int v = v0; v < v1; v += kChunk) {
        Held<T> h;
        h.at = (v + tid) * E - head;
        h.end = min(a.V, v1 * E - head);
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            h.q[i] = v + i * kThreads + tid < v1 ? load_vec(row, h.at + i * kThreads * E, a.V) : neg_inf_vec<T>();
        float top = kNegInf;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            h.top[i] = batch_max1<T>(h.q[i]);
            top = max_nan(top, h.top[i]);
        }
        odd |= !(top < INFINITY);
        // ---- sums, against this thread's own reference
        if (top > m) {
            const float y = m == kNegInf ? kFar : fmaxf((m - top) * c, kFar), keep = ex2(y);
            s = make_float2(keep * fmaf(z.x, y, s.x), keep * fmaf(z.y, y, s.y));
            z = make_float2(keep * z.x, keep * z.y);
            m = top;
        }
        const float ref = m == kNegInf ? 0.0f : m;
        const float2 ref2 = make_float2(-ref, -ref), c2 = make_float2(c, c), none = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            float f[E];
            unpack<T>(h.q[i], f);
            const int at = h.at + i * kThreads * E;
            const float bar = at + E <= token ? under : lt;
#pragma unroll
            for (int k = 0; k < E; k += 2) {
                float2 y = fma2(add2(make_float2(f[k], f[k + 1]), ref2), c2, none);
                y = make_float2(fmaxf(y.x, kFar), fmaxf(y.y, kFar));
                const float2 e = make_float2(ex2(y.x), ex2(y.y));
                z = add2(z, e);
                s = fma2(e, y, s);
            }
            if (!(h.top[i] >= lt)) continue;  // nothing of the vector comes before the token
#pragma unroll
            for (int k = 0; k < E; ++k) before += f[k] > bar;
            if (lowest || (at <= token && token < at + E)) {  // equal ones before it
#pragma unroll
                for (int k = 0; k < E; ++k)
                    before += f[k] == lt && at + k >= 0 && at + k < min(token, h.end) && (lowest || at + E > token);
            }
        }
        if (SOME) take_first<T>(sh, h, top, a.top);
    }
    // ---- the slice's sums
    float most = m;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (__any_sync(0xffffffffu, odd) && lane == 0) sh.bad = kFlagNonFinite;
    if (lane == 0) sh.warp[0][warp] = most;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) most = fmaxf(most, sh.warp[0][w]);
    float zs = z.x + z.y, as = s.x + s.y;
    {
        const float y = m == kNegInf ? kFar : fmaxf((m - most) * c, kFar), keep = ex2(y);
        as = keep * fmaf(zs, y, as);
        zs *= keep;
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        zs += __shfl_xor_sync(0xffffffffu, zs, o);
        as += __shfl_xor_sync(0xffffffffu, as, o);
    }
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) {
        sh.warp[1][warp] = zs;
        sh.warp[2][warp] = as;
        sh.before[warp] = before;
    }
    __syncthreads();
    cluster_wait();
    if (tid == 0) {
        Part p = {most, 0.0f, 0.0f, 0, sh.bad};
        for (int w = 0; w < kWarps; ++w) {
            p.z += sh.warp[1][w];
            p.a += sh.warp[2][w];
            p.before += sh.before[w];
        }
        *remote(&sh.part[rank]) = p;
    }
    if (SOME && tid < a.top) *remote(&sh.list[rank][tid]) = tid < static_cast<int>(sh.n_mine) ? sh.mine[tid] : 0;
    cluster_arrive();
    cluster_wait();
    if (rank) return;
    // ---- the row
    float R = kNegInf, Z = 0.0f, A = 0.0f;
    uint32_t bad = 0, place = 0;
    for (int i = 0; i < size; ++i) {
        R = fmaxf(R, sh.part[i].m);
        bad |= sh.part[i].bad;
    }
    if (!bad && R == kNegInf) bad = kFlagAllNegInf;
    for (int i = 0; i < size; ++i) {
        const Part p = sh.part[i];
        place += p.before;
        const float y = p.m == kNegInf ? kFar : fmaxf((p.m - R) * c, kFar), keep = ex2(y);
        A = fmaf(keep, fmaf(p.z, y, p.a), A);
        Z = fmaf(keep, p.z, Z);
    }
    const float lz = log2f(Z);
    if (tid == 0) {
        if (bad) atomicOr(a.err, bad);
        a.logprob[entry] = bad ? NAN : (lt - R) * a.inv_t - kLn2 * lz;
        if (a.entropy) a.entropy[entry] = bad ? NAN : kLn2 * (lz - A / Z);
        if (a.rank) a.rank[entry] = bad ? -1 : static_cast<int32_t>(place);
    }
    if (!SOME) return;
    if (bad) {
        if (tid < a.top) {
            a.top_ids[entry * a.top + tid] = -1;
            a.top_logprobs[entry * a.top + tid] = NAN;
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
        a.top_ids[entry * a.top + k] = static_cast<int32_t>(~static_cast<uint32_t>(x));
        a.top_logprobs[entry * a.top + k] = (key_float(static_cast<uint32_t>(x >> 32)) - R) * a.inv_t - kLn2 * lz;
    }
}

template <typename T, bool SOME>
int launch_size(const LogprobArgs &a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * a.M * a.cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {static_cast<unsigned>(a.cluster), 1, 1};
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, SOME>, a) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

int launch_logprobs(LogprobArgs &a, int dtype, cudaStream_t st) {
    const int E = dtype == SPEC_F32 ? 4 : 8;
    const long long entries = static_cast<long long>(a.B) * a.M;
    a.cluster = 1;
    while (a.cluster < kMaxCluster && (a.V > a.cluster * kChunk * E || (a.V > a.cluster * kThreads * E && entries * a.cluster < 152 * 8)))
        a.cluster *= 2;
    if (dtype == SPEC_F32) return a.top ? launch_size<float, true>(a, st) : launch_size<float, false>(a, st);
    return a.top ? launch_size<uint16_t, true>(a, st) : launch_size<uint16_t, false>(a, st);
}

}  // namespace specv
