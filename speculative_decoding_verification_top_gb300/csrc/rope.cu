// rope.cu -- rotary positions: of queries, of keys on their way into the paged
// cache, and of the rotary part of a latent cache's rows.
//
//   pair (u, v) of a token at index p -> a (u cos - v sin, v cos + u sin), angle
//   p theta.  The frequency comes as f = 2^64 theta / (2 pi): the low 64 bits of
//   f p are the angle's fraction of a turn, exact for any p, and their 32 bits
//   below the quadrant are more than fp32 holds.  (An fp32 angle would lose, at
//   position 10^5, all but 2^-7 of a turn's last radian.)
//
// A unit is 16 elements of a head, two vectors of 8: eight pairs, or 16
// elements that stay.  A thread takes one unit of up to four heads of a token, so
// that eight sines and cosines (about 30 instructions each) serve 32 pairs.
// All kernels are bound by memory: each element read once and written once.

#include "kvrows.cuh"
#include "target.cuh"

namespace specv {
namespace {

// A unit's two vectors in its head, and its first pair (-1: not turned).
struct Unit {
    int at0, at1, pair;
};

__device__ __forceinline__ Unit unit_of(const Turn &t, int unit) {
    const int e = unit * kW, i = e - t.first;
    if (i < 0 || i >= t.rot) return {e, e + kE, -1};
    if (t.interleaved) return {e, e + kE, i / 2};
    return {t.first + i / 2, t.first + i / 2 + t.rot / 2, i / 2};
}

// a cos and a sin of pairs pair .. pair + 7 at index p.
struct Angles {
    float c[kE], s[kE];
};

__device__ __forceinline__ Angles angles_of(const Turn &t, int pair, long long p) {
    Angles a = {};
    if (pair < 0) return a;
    ulonglong2 f[kE / 2];
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) f[i] = __ldg(reinterpret_cast<const ulonglong2 *>(t.freqs + pair) + i);
    const long long index = t.inverse ? -p : p;
#pragma unroll
    for (int i = 0; i < kE; ++i) {
        const unsigned long long turns = (i & 1 ? f[i / 2].y : f[i / 2].x) * static_cast<unsigned long long>(index);
        const uint32_t quadrant = static_cast<uint32_t>((turns + (1ull << 61)) >> 62);
        // the rest, within an eighth of a turn to either side
        const float x = static_cast<float>(static_cast<int32_t>(static_cast<uint32_t>(turns >> 30))) * 0x1p-33f;
        float s, c;
        sincospif(x, &s, &c);
        const float u = quadrant & 1 ? s : c, v = quadrant & 1 ? c : s;
        a.c[i] = quadrant == 1 || quadrant == 2 ? -t.amplitude * u : t.amplitude * u;
        a.s[i] = quadrant >= 2 ? -t.amplitude * v : t.amplitude * v;
    }
    return a;
}

// A unit's elements turned.
__device__ __forceinline__ void turn(float (&x)[2][kE], const Angles &a, bool interleaved) {
#pragma unroll
    for (int i = 0; i < kE; ++i) {
        float &u = interleaved ? x[i / 4][i % 4 * 2] : x[0][i];
        float &v = interleaved ? x[i / 4][i % 4 * 2 + 1] : x[1][i];
        const float y = u * a.c[i] - v * a.s[i];
        v = v * a.c[i] + u * a.s[i];
        u = y;
    }
}

// Eight elements of a tensor that the same kernel may write: not by the
// read-only path.
__device__ __forceinline__ void fetch8(const float *p, float (&x)[kE]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

__device__ __forceinline__ void fetch8(const __nv_bfloat16 *p, float (&x)[kE]) {
    widen8(*reinterpret_cast<const uint4 *>(p), x);
}

// The heads h0 .. of one token, this thread's unit of each.
template <typename T, int HC>
__device__ __forceinline__ void turn_heads(const T *x, T *out, const Turn &t, int H, int D, int unit, int h0, long long p) {
    const Unit u = unit_of(t, unit);
    if (u.pair < 0 && x == out) return;
    float y[HC][2][kE];
#pragma unroll
    for (int i = 0; i < HC; ++i) {
        if (h0 + i >= H) break;
        fetch8(x + (h0 + i) * D + u.at0, y[i][0]);
        fetch8(x + (h0 + i) * D + u.at1, y[i][1]);
    }
    const Angles a = angles_of(t, u.pair, p);
#pragma unroll
    for (int i = 0; i < HC; ++i) {
        if (h0 + i >= H) break;
        if (u.pair >= 0) {
            if (t.interleaved)
                turn(y[i], a, true);
            else
                turn(y[i], a, false);
        }
        store8(out + (h0 + i) * D + u.at0, y[i][0]);
        store8(out + (h0 + i) * D + u.at1, y[i][1]);
    }
}

template <typename T, int HC>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
    const uint32_t units = a.D / kW, chunks = (a.H + HC - 1) / HC;
    const uint32_t item = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t token = item / (units * chunks), rest = item - token * units * chunks;
    if (token >= static_cast<uint32_t>(a.tokens)) return;
    const uint32_t chunk = rest / units;
    turn_heads<T, HC>(static_cast<const T *>(a.x) + token * a.x_stride, static_cast<T *>(a.out) + token * a.out_stride, a.t,
                      a.H, a.D, rest - chunk * units, chunk * HC, a.pos[token]);
}

// A unit of a cache row: rounded, or as bytes with the row's exponent.  Whole
// warps call it.
template <int D, bool E4M3>
__device__ __forceinline__ void write_unit(uint8_t *data, int8_t *exps, long long row, const Unit &u, int part, bool live,
                                           const float (&x)[2][kE]) {
    if (!E4M3) {
        if (live) {
            __nv_bfloat16 *p = reinterpret_cast<__nv_bfloat16 *>(data) + row * D;
            store8(p + u.at0, x[0]);
            store8(p + u.at1, x[1]);
        }
        return;
    }
    uint32_t w[4];
    const int e = quantise<D>(x, w);
    if (!live) return;
    *reinterpret_cast<uint2 *>(data + row * D + u.at0) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2 *>(data + row * D + u.at1) = make_uint2(w[2], w[3]);
    if (part == 0) exps[row] = static_cast<int8_t>(e);
}

// The first kv_blocks blocks write keys and values, the others turn queries.
template <typename T, int D, bool E4M3, int HC>
__global__ void __launch_bounds__(kThreads) kv_append_rope_kernel(const AppendRopeArgs ar) {
    constexpr int kUnits = D / kW;
    const AppendArgs &a = ar.a;
    const int unit = threadIdx.x % kUnits;
    if (blockIdx.x >= ar.kv_blocks) {
        const uint32_t chunks = (ar.Hq + HC - 1) / HC;
        const uint32_t item = (blockIdx.x - ar.kv_blocks) * (kThreads / kUnits) + threadIdx.x / kUnits;
        const uint32_t token = item / chunks;
        if (token >= static_cast<uint32_t>(a.B) * a.N) return;
        const uint32_t b = token / a.N;
        const long long p = ar.pos ? ar.pos[token] : static_cast<long long>(a.starts[b]) + static_cast<int>(token - b * a.N);
        turn_heads<T, HC>(static_cast<const T *>(ar.q) + token * ar.q_stride, static_cast<T *>(ar.out_q) + token * ar.out_q_stride,
                          ar.t, ar.Hq, D, unit, (item - token * chunks) * HC, p);
        return;
    }
    const uint32_t chunks = (a.c.Hkv + HC - 1) / HC;
    const uint32_t item = blockIdx.x * (kThreads / kUnits) + threadIdx.x / kUnits;
    const uint32_t bt = item / chunks;
    const Unit u = unit_of(ar.t, unit);
    int page = -1, slot = 0, h0 = 0, p = 0;
    float k[HC][2][kE] = {}, v[HC][2][kE] = {};
    if (bt < static_cast<uint32_t>(a.B) * a.M) {
        const uint32_t b = bt / a.M;
        const int t = static_cast<int>(bt - b * a.M), r = a.rows ? a.rows[bt] : t;
        h0 = static_cast<int>(item - bt * chunks) * HC;
        const long long at = static_cast<long long>(a.starts[b]) + t;
        if (r >= 0 && r < a.N && at <= INT_MAX) {
            const long long token = static_cast<long long>(b) * a.N + r;
            const T *pk = static_cast<const T *>(a.k) + token * a.stride, *pv = static_cast<const T *>(a.v) + token * a.stride;
            p = ar.pos ? ar.pos[token] : static_cast<int>(at);
            page = page_of(a.c, a.table + static_cast<long long>(b) * a.width, a.width, static_cast<int>(at), &slot);
            if (page >= 0) {
#pragma unroll
                for (int i = 0; i < HC; ++i) {
                    if (h0 + i >= a.c.Hkv) break;
                    load8(pk + (h0 + i) * D + u.at0, k[i][0]);
                    load8(pk + (h0 + i) * D + u.at1, k[i][1]);
                    load8(pv + (h0 + i) * D + u.at0, v[i][0]);
                    load8(pv + (h0 + i) * D + u.at1, v[i][1]);
                }
            }
        }
    }
    const Angles an = angles_of(ar.t, u.pair, p);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < HC; ++i) {
        const bool live = page >= 0 && h0 + i < a.c.Hkv;
        const long long row = live ? cache_row(a.c, page, h0 + i, slot) : 0;
        if (u.pair >= 0) {
            if (ar.t.interleaved)
                turn(k[i], an, true);
            else
                turn(k[i], an, false);
        }
        __syncwarp();
        write_unit<D, E4M3>(a.c.k, a.c.k_exp, row, u, unit, live, k[i]);
        write_unit<D, E4M3>(a.c.v, a.c.v_exp, row, u, unit, live, v[i]);
    }
}

// Rows of a latent cache, a unit a thread: C / 16 of the latent, then the rotary
// part's.
template <typename T>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(const LatentAppendArgs a) {
    const uint32_t units = (a.c.C + a.c.R) / kW;
    const uint32_t item = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t bt = item / units;
    if (bt >= static_cast<uint32_t>(a.B) * a.M) return;
    const int unit = static_cast<int>(item - bt * units);
    const uint32_t b = bt / a.M;
    const int t = static_cast<int>(bt - b * a.M), r = a.rows ? a.rows[bt] : t;
    const long long at = static_cast<long long>(a.starts[b]) + t;
    if (r < 0 || r >= a.N || at < 0 || at > INT_MAX) return;
    const int i = static_cast<int>(at) >> a.c.page_shift;
    if (i >= a.width) return;
    const int page = a.table[static_cast<long long>(b) * a.width + i];
    if (page < 0 || page >= a.c.num_pages) return;
    const long long token = static_cast<long long>(b) * a.N + r;
    const long long row = (static_cast<long long>(page) << a.c.page_shift) + (at & ((1 << a.c.page_shift) - 1));
    __nv_bfloat16 *to = a.c.data + row * (a.c.C + a.c.R);
    float x[2][kE];
    if (unit * kW < a.c.C) {
        const T *from = static_cast<const T *>(a.x) + token * a.x_stride + unit * kW;
        load8(from, x[0]);
        load8(from + kE, x[1]);
        store8(to + unit * kW, x[0]);
        store8(to + unit * kW + kE, x[1]);
        return;
    }
    const Unit u = unit_of(a.t, unit - a.c.C / kW);
    const T *from = static_cast<const T *>(a.r) + token * a.r_stride;
    load8(from + u.at0, x[0]);
    load8(from + u.at1, x[1]);
    if (u.pair >= 0) {
        const Angles an = angles_of(a.t, u.pair, a.pos ? a.pos[token] : static_cast<int>(at));
        if (a.t.interleaved)
            turn(x, an, true);
        else
            turn(x, an, false);
    }
    store8(to + a.c.C + u.at0, x[0]);
    store8(to + a.c.C + u.at1, x[1]);
}

// Heads a thread: four where that leaves every multiprocessor full, else one.
constexpr long long kFull = 152ll * 2048;

unsigned blocks_for(long long threads) { return static_cast<unsigned>((threads + kThreads - 1) / kThreads); }

int launched() { return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA; }

template <typename T>
int rope_heads(const RopeArgs &a, cudaStream_t st) {
    const long long each = static_cast<long long>(a.tokens) * (a.D / kW);
    if (each * a.H > 4 * kFull)
        rope_kernel<T, 4><<<blocks_for(each * ((a.H + 3) / 4)), kThreads, 0, st>>>(a);
    else
        rope_kernel<T, 1><<<blocks_for(each * a.H), kThreads, 0, st>>>(a);
    return launched();
}

template <typename T, int D, bool E4M3, int HC>
int append_heads(AppendRopeArgs &a, cudaStream_t st) {
    const long long entries = static_cast<long long>(a.a.B) * a.a.M, tokens = a.q ? static_cast<long long>(a.a.B) * a.a.N : 0;
    a.kv_blocks = blocks_for(entries * ((a.a.c.Hkv + HC - 1) / HC) * (D / kW));
    const unsigned q_blocks = blocks_for(tokens * ((a.Hq + HC - 1) / HC) * (D / kW));
    kv_append_rope_kernel<T, D, E4M3, HC><<<a.kv_blocks + q_blocks, kThreads, 0, st>>>(a);
    return launched();
}

template <typename T, int D, bool E4M3>
int append_rope(AppendRopeArgs &a, cudaStream_t st) {
    const long long rows = static_cast<long long>(a.a.B) * a.a.M * a.a.c.Hkv +
                           (a.q ? static_cast<long long>(a.a.B) * a.a.N * a.Hq : 0);
    return rows * (D / kW) > 4 * kFull ? append_heads<T, D, E4M3, 4>(a, st) : append_heads<T, D, E4M3, 1>(a, st);
}

template <typename T>
int append_rope_type(AppendRopeArgs &a, cudaStream_t st) {
    const bool e = a.a.c.e4m3 != 0, wide = a.a.c.D == 128;
    return e ? (wide ? append_rope<T, 128, true>(a, st) : append_rope<T, 64, true>(a, st))
             : (wide ? append_rope<T, 128, false>(a, st) : append_rope<T, 64, false>(a, st));
}

}  // namespace

int launch_rope(const RopeArgs &a, int dtype, cudaStream_t st) {
    return dtype == SPEC_F32 ? rope_heads<float>(a, st) : rope_heads<__nv_bfloat16>(a, st);
}

int launch_kv_append_rope(AppendRopeArgs &a, int dtype, cudaStream_t st) {
    return dtype == SPEC_F32 ? append_rope_type<float>(a, st) : append_rope_type<__nv_bfloat16>(a, st);
}

int launch_latent_append(const LatentAppendArgs &a, int dtype, cudaStream_t st) {
    const long long threads = static_cast<long long>(a.B) * a.M * ((a.c.C + a.c.R) / kW);
    if (dtype == SPEC_F32)
        latent_append_kernel<float><<<blocks_for(threads), kThreads, 0, st>>>(a);
    else
        latent_append_kernel<__nv_bfloat16><<<blocks_for(threads), kThreads, 0, st>>>(a);
    return launched();
}

}  // namespace specv
