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
// All kernels are bound by memory: each element read once and written once.  What
// a thread loads is held as it came until its turn, so that a multiprocessor has
// room for 16 and more warps with 128 bytes a thread on their way (widened at once,
// and keys with their values in one thread, 170 registers left room for 8: 284 us
// where 121 are needed).
// Measured: 8 x 4099 tokens of 16 fp32 heads of 128, 79 us (6.8 TB/s, the copy rate);
// their keys, values and queries, 32/8 bf16 heads, into a bf16 cache, 121 us (6.6);
// 16 x 6001 latent rows of 512 + 64, 39 us (5.6); the keys, values and queries into an
// e4m3 cache, 139 us (5.3).  Calls of a few hundred tokens take 4.4 to 6.1 us on the GPU
// (cold, timed alone) and are bound by the way there.

#include "kvrows.cuh"
#include "target.cuh"
#include "util.cuh"

namespace specv {
namespace {

// A unit's two vectors in its head, and whether they are turned; the vectors lie
// half a part (the turned one, or what stays before or after it) apart, so that
// neighbouring lanes' vectors lie side by side in either layout.
struct Unit {
    int at0, at1, turned;
};

__device__ __forceinline__ Unit unit_of(const Turn &t, int D, int unit) {
    const int e = unit * kW, end = t.first + t.rot;
    const int part = e < t.first ? 0 : e < end ? t.first : end;
    const int size = e < t.first ? t.first : e < end ? t.rot : D - end;
    const int at = part + (e - part) / 2;
    return {at, at + size / 2, e >= t.first && e < end};
}

// a cos and a sin of a unit's pairs at index p, in the order of its vectors.
struct Angles {
    float c[kE], s[kE];
};

__device__ __forceinline__ Angles angles_of(const Turn &t, const Unit &u, long long p) {
    Angles a = {};
    if (!u.turned) return a;
    // Half: the first vector's eight pairs.  Interleaved: each vector's four.
    const int i0 = u.at0 - t.first, p0 = t.interleaved ? i0 / 2 : i0, p1 = t.interleaved ? i0 / 2 + t.rot / 4 : i0 + kE / 2;
    ulonglong2 f[kE / 2];
#pragma unroll
    for (int i = 0; i < kE / 2; ++i)
        f[i] = __ldg(reinterpret_cast<const ulonglong2 *>(t.freqs + (i < kE / 4 ? p0 : p1)) + i % (kE / 4));
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

// Eight elements as they lie in memory.
template <typename T>
struct Raw;

template <>
struct Raw<float> {
    float4 a, b;
    __device__ __forceinline__ void widen(float (&x)[kE]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
};

template <>
struct Raw<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void widen(float (&x)[kE]) const { widen8(a, x); }
};

// Not by the read-only path: the same kernel may write the tensor.
__device__ __forceinline__ Raw<float> fetch(const float *p) {
    return {*reinterpret_cast<const float4 *>(p), *(reinterpret_cast<const float4 *>(p) + 1)};
}

__device__ __forceinline__ Raw<__nv_bfloat16> fetch(const __nv_bfloat16 *p) { return {*reinterpret_cast<const uint4 *>(p)}; }

// A unit of up to HC heads from head h0 on, of `n` heads, as it lies in memory.
template <typename T, int HC>
struct Heads {
    Raw<T> x[HC][2];

    __device__ __forceinline__ void load(const T *from, int D, const Unit &u, int h0, int n) {
#pragma unroll
        for (int i = 0; i < HC; ++i) {
            if (h0 + i >= n) break;
            x[i][0] = fetch(from + (h0 + i) * D + u.at0);
            x[i][1] = fetch(from + (h0 + i) * D + u.at1);
        }
    }

    // Head i's elements, turned if the unit is.
    __device__ __forceinline__ void get(int i, const Turn &t, const Unit &u, const Angles &a, float (&y)[2][kE]) const {
        x[i][0].widen(y[0]);
        x[i][1].widen(y[1]);
        if (!u.turned) return;
        if (t.interleaved)
            turn(y, a, true);
        else
            turn(y, a, false);
    }
};

// The heads h0 .. of one token, this thread's unit of each.
template <typename T, int HC>
__device__ __forceinline__ void turn_heads(const T *x, T *out, const Turn &t, int H, int D, int unit, int h0, long long p) {
    const Unit u = unit_of(t, D, unit);
    if (!u.turned && x == out) return;
    Heads<T, HC> heads;
    heads.load(x, D, u, h0, H);
    const Angles a = angles_of(t, u, p);
#pragma unroll
    for (int i = 0; i < HC; ++i) {
        if (h0 + i >= H) break;
        float y[2][kE];
        heads.get(i, t, u, a, y);
        store8(out + (h0 + i) * D + u.at0, y[0]);
        store8(out + (h0 + i) * D + u.at1, y[1]);
    }
}

template <typename T, int HC>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
    started_early();
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

// The first kv_blocks blocks write keys, the next as many values, the others turn
// queries.
template <typename T, int D, bool E4M3, int HC>
__global__ void __launch_bounds__(kThreads) kv_append_rope_kernel(const AppendRopeArgs ar) {
    started_early();
    constexpr int kUnits = D / kW;
    const AppendArgs &a = ar.a;
    const int unit = threadIdx.x % kUnits;
    if (blockIdx.x >= 2 * ar.kv_blocks) {
        const uint32_t chunks = (ar.Hq + HC - 1) / HC;
        const uint32_t item = (blockIdx.x - 2 * ar.kv_blocks) * (kThreads / kUnits) + threadIdx.x / kUnits;
        const uint32_t token = item / chunks;
        if (token >= static_cast<uint32_t>(a.B) * a.N) return;
        const uint32_t b = token / a.N;
        const long long p = ar.pos ? ar.pos[token] : static_cast<long long>(a.starts[b]) + static_cast<int>(token - b * a.N);
        turn_heads<T, HC>(static_cast<const T *>(ar.q) + token * ar.q_stride, static_cast<T *>(ar.out_q) + token * ar.out_q_stride,
                          ar.t, ar.Hq, D, unit, (item - token * chunks) * HC, p);
        return;
    }
    const bool values = blockIdx.x >= ar.kv_blocks;
    const uint32_t chunks = (a.c.Hkv + HC - 1) / HC;
    const uint32_t item = (values ? blockIdx.x - ar.kv_blocks : blockIdx.x) * (kThreads / kUnits) + threadIdx.x / kUnits;
    const uint32_t bt = item / chunks;
    Unit u = unit_of(ar.t, D, unit);
    if (values) u.turned = 0;
    int page = -1, slot = 0, h0 = 0, p = 0;
    Heads<T, HC> heads = {};
    if (bt < static_cast<uint32_t>(a.B) * a.M) {
        const uint32_t b = bt / a.M;
        const int t = static_cast<int>(bt - b * a.M), r = a.rows ? a.rows[bt] : t;
        h0 = static_cast<int>(item - bt * chunks) * HC;
        if (r >= 0 && r < a.N) {
            const long long token = static_cast<long long>(b) * a.N + r, at = static_cast<long long>(a.starts[b]) + t;
            heads.load(static_cast<const T *>(values ? a.v : a.k) + token * a.stride, D, u, h0, a.c.Hkv);
            p = ar.pos ? ar.pos[token] : static_cast<int>(at);
            if (at <= INT_MAX)
                page = page_of(a.c, a.table + static_cast<long long>(b) * a.width, a.width, static_cast<int>(at), &slot);
        }
    }
    const Angles an = angles_of(ar.t, u, p);
    uint8_t *data = values ? a.c.v : a.c.k;
    int8_t *exps = values ? a.c.v_exp : a.c.k_exp;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < HC; ++i) {
        const bool live = page >= 0 && h0 + i < a.c.Hkv;
        const long long row = live ? cache_row(a.c, page, h0 + i, slot) : 0;
        float y[2][kE];
        heads.get(i, ar.t, u, an, y);
        __syncwarp();
        write_unit<D, E4M3>(data, exps, row, u, unit, live, y);
    }
}

// Rows of a latent cache.  The first c_blocks blocks copy the latent, 32 elements a
// thread; the others turn the rotary part, a unit a thread (in warps of their own:
// beside the copies its sines and cosines would hold up every warp).
template <typename T>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(const LatentAppendArgs a, unsigned c_blocks) {
    started_early();
    const bool rotary = blockIdx.x >= c_blocks;
    const uint32_t units = rotary ? a.c.R / kW : a.c.C / (2 * kW);
    const uint32_t item = (rotary ? blockIdx.x - c_blocks : blockIdx.x) * kThreads + threadIdx.x;
    const uint32_t bt = item / units;
    if (bt >= static_cast<uint32_t>(a.B) * a.M) return;
    const int unit = static_cast<int>(item - bt * units);
    const uint32_t b = bt / a.M;
    const int t = static_cast<int>(bt - b * a.M), r = a.rows ? a.rows[bt] : t;
    if (r < 0 || r >= a.N) return;
    const long long at = static_cast<long long>(a.starts[b]) + t, token = static_cast<long long>(b) * a.N + r;
    // Where the token goes; null: nowhere.
    auto target = [&]() -> __nv_bfloat16 * {
        if (at < 0 || at > INT_MAX) return nullptr;
        const int i = static_cast<int>(at) >> a.c.page_shift;
        if (i >= a.width) return nullptr;
        const int page = a.table[static_cast<long long>(b) * a.width + i];
        if (page < 0 || page >= a.c.num_pages) return nullptr;
        const long long row = (static_cast<long long>(page) << a.c.page_shift) + (at & ((1 << a.c.page_shift) - 1));
        return a.c.data + row * (a.c.C + a.c.R);
    };
    if (!rotary) {
        constexpr int kV = 2 * kW / kE;  // vectors, a quarter of the row apart
        const int step = a.c.C / kV;
        const T *from = static_cast<const T *>(a.x) + token * a.x_stride + unit * kE;
        Raw<T> x[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) x[i] = fetch(from + i * step);
        __nv_bfloat16 *to = target();
        if (!to) return;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            float y[kE];
            x[i].widen(y);
            store8(to + unit * kE + i * step, y);
        }
        return;
    }
    const Unit u = unit_of(a.t, a.c.R, unit);
    Heads<T, 1> part;
    part.load(static_cast<const T *>(a.r) + token * a.r_stride, 0, u, 0, 1);
    __nv_bfloat16 *to = target();
    if (!to) return;
    const Angles an = angles_of(a.t, u, a.pos ? a.pos[token] : static_cast<int>(at));
    float y[2][kE];
    part.get(0, a.t, u, an, y);
    store8(to + a.c.C + u.at0, y[0]);
    store8(to + a.c.C + u.at1, y[1]);
}

// Heads a thread: four where that leaves every multiprocessor full, else one (64 x 6
// tokens of 32 heads: 5.5 us; with four, a fifth of the multiprocessors idle).
constexpr long long kFull = 152ll * 2048;

unsigned blocks_for(long long threads) { return static_cast<unsigned>((threads + kThreads - 1) / kThreads); }

template <typename... Params, typename... Args>
int launch(void (*kernel)(Params...), unsigned blocks, cudaStream_t st, const Args &...args) {
    return launch_early(kernel, dim3(blocks), dim3(kThreads), 0, st, args...) ? SPEC_OK : SPEC_ERR_CUDA;
}

template <typename T>
int rope_heads(const RopeArgs &a, cudaStream_t st) {
    const long long each = static_cast<long long>(a.tokens) * (a.D / kW);
    if (each * a.H > 4 * kFull)
        return launch(rope_kernel<T, 4>, blocks_for(each * ((a.H + 3) / 4)), st, a);
    return launch(rope_kernel<T, 1>, blocks_for(each * a.H), st, a);
}

template <typename T, int D, bool E4M3, int HC>
int append_heads(AppendRopeArgs &a, cudaStream_t st) {
    const long long entries = static_cast<long long>(a.a.B) * a.a.M, tokens = a.q ? static_cast<long long>(a.a.B) * a.a.N : 0;
    a.kv_blocks = blocks_for(entries * ((a.a.c.Hkv + HC - 1) / HC) * (D / kW));
    const unsigned q_blocks = blocks_for(tokens * ((a.Hq + HC - 1) / HC) * (D / kW));
    return launch(kv_append_rope_kernel<T, D, E4M3, HC>, 2 * a.kv_blocks + q_blocks, st, a);
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
    const long long entries = static_cast<long long>(a.B) * a.M;
    const unsigned c_blocks = blocks_for(entries * (a.c.C / (2 * kW))), blocks = c_blocks + blocks_for(entries * (a.c.R / kW));
    return dtype == SPEC_F32 ? launch(latent_append_kernel<float>, blocks, st, a, c_blocks)
                             : launch(latent_append_kernel<__nv_bfloat16>, blocks, st, a, c_blocks);
}

}  // namespace specv
