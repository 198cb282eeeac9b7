// kvcache.cu -- writing new tokens' keys and values into the paged cache, and
// reading positions back.
//
//   bf16   x as it is (fp32 inputs rounded to nearest).
//   e4m3   a = max |x_d| over the row, e = the smallest integer with
//          a <= 448 * 2^e, byte = e4m3(x * 2^-e).  With a = m * 2^(E),
//          m in [1, 2): 448 = 1.75 * 2^8, so e = E - 8 + (m > 1.75), read off
//          a's own bits.  The scaling is exact, the byte the only rounding.
//
// A row of D elements goes to D / 16 lanes when it is written (the row's
// maximum is then a shuffle reduction of two or three steps), to D / 8 when it
// is read.  Both are bound by memory: each new element read once, each cache
// byte written once, and the reverse.

#include "kvrows.cuh"

namespace specv {
namespace {

// One row's share: quantise (or round) x and write it to cache row `row` if
// the row is live.  Whole warps call it.
template <int D, bool E4M3>
__device__ __forceinline__ void write_row(uint8_t *data, int8_t *exps, long long row, int part,
                                          bool live, const float (&x)[2][kE]) {
    if (!E4M3) {
        if (live) {
            __nv_bfloat16 *p = reinterpret_cast<__nv_bfloat16 *>(data) + row * D + part * kW;
            store8(p, x[0]);
            store8(p + kE, x[1]);
        }
        return;
    }
    uint32_t w[4];
    const int e = quantise<D>(x, w);
    if (!live) return;
    *reinterpret_cast<uint4 *>(data + row * D + part * kW) = make_uint4(w[0], w[1], w[2], w[3]);
    if (part == 0) exps[row] = static_cast<int8_t>(e);
}

// A lane writes 16 elements of a row's keys and of its values.  Rows number
// (entry, head): below 2^31, so 32-bit arithmetic.  Eight sequences of 4099
// tokens, 8 heads of 128, e4m3 (202 MB): 41 us, 4.9 TB/s; 8 elements a lane
// took 47, with four rows a thread 85.
template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendArgs a) {
    constexpr int kLanes = D / kW;  // lanes a row
    const uint32_t items = static_cast<uint32_t>(a.B) * a.M * a.c.Hkv;
    const uint32_t item = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    const int part = threadIdx.x % kLanes;
    int page = -1, slot = 0, h = 0;
    float k[2][kE] = {}, v[2][kE] = {};
    if (item < items) {
        const uint32_t bt = item / a.c.Hkv, b = bt / a.M;
        const int t = static_cast<int>(bt - b * a.M), r = a.rows ? a.rows[bt] : t;
        h = static_cast<int>(item - bt * a.c.Hkv);
        const long long p = static_cast<long long>(a.starts[b]) + t;
        if (r >= 0 && r < a.N && p <= INT_MAX) {
            const long long src = (static_cast<long long>(b) * a.N + r) * a.stride + h * D + part * kW;
            const T *pk = static_cast<const T *>(a.k) + src, *pv = static_cast<const T *>(a.v) + src;
            load8(pk, k[0]);
            load8(pk + kE, k[1]);
            load8(pv, v[0]);
            load8(pv + kE, v[1]);
            page = page_of(a.c, a.table + static_cast<long long>(b) * a.width, a.width, static_cast<int>(p), &slot);
        }
    }
    __syncwarp();
    const bool live = page >= 0;
    const long long row = live ? cache_row(a.c, page, h, slot) : 0;
    write_row<D, E4M3>(a.c.k, a.c.k_exp, row, part, live, k);
    write_row<D, E4M3>(a.c.v, a.c.v_exp, row, part, live, v);
}

// Eight elements of a cache row as they lie there.
struct Raw {
    uint4 u;  // bf16, or in x and y eight bytes
    int e;
};

template <int D, bool E4M3>
__device__ __forceinline__ Raw read_raw(const uint8_t *data, const int8_t *exps, long long row, int part) {
    Raw r = {};
    if (!E4M3) {
        r.u = __ldg(reinterpret_cast<const uint4 *>(data + (row * D + part * kE) * 2));
    } else {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(data + row * D + part * kE));
        r.u.x = w.x;
        r.u.y = w.y;
        r.e = exps[row];
    }
    return r;
}

template <bool E4M3>
__device__ __forceinline__ void unpack(const Raw &r, float (&x)[kE]) {
    if (!E4M3) {
        const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
        return;
    }
    const float f = exp2i(max(-120, min(120, r.e)));  // the range that is written
    const uint32_t w[2] = {r.u.x, r.u.y};
#pragma unroll
    for (int i = 0; i < kE; i += 2) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i / 4] >> (8 * (i % 4))), __NV_E4M3);
        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        x[i] = y.x * f;
        x[i + 1] = y.y * f;
    }
}

template <typename T, int D, bool E4M3, int PER>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadArgs a) {
    constexpr int kLanes = D / kE, kRows = kThreads / kLanes;
    const uint32_t items = static_cast<uint32_t>(a.B) * a.M * a.c.Hkv;
    const int part = threadIdx.x % kLanes;
    Raw k[PER] = {}, v[PER] = {};
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t item = (blockIdx.x * PER + i) * kRows + threadIdx.x / kLanes;
        if (item >= items) continue;
        const uint32_t bt = item / a.c.Hkv, b = bt / a.M;
        const int h = static_cast<int>(item - bt * a.c.Hkv);
        const long long p = static_cast<long long>(a.starts[b]) + static_cast<int>(bt - b * a.M);
        int slot = 0;
        const int page = p > INT_MAX ? -1
                                     : page_of(a.c, a.table + static_cast<long long>(b) * a.width, a.width,
                                               static_cast<int>(p), &slot);
        if (page < 0) continue;
        const long long row = cache_row(a.c, page, h, slot);
        if (a.out_k) k[i] = read_raw<D, E4M3>(a.c.k, a.c.k_exp, row, part);
        if (a.out_v) v[i] = read_raw<D, E4M3>(a.c.v, a.c.v_exp, row, part);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t item = (blockIdx.x * PER + i) * kRows + threadIdx.x / kLanes;
        if (item >= items) continue;
        const long long o = static_cast<long long>(item) * D + part * kE;
        float x[kE];
        if (a.out_k) {
            unpack<E4M3>(k[i], x);
            store8(static_cast<T *>(a.out_k) + o, x);
        }
        if (a.out_v) {
            unpack<E4M3>(v[i], x);
            store8(static_cast<T *>(a.out_v) + o, x);
        }
    }
}

// Rows a thread of a large call (over 152 full multiprocessors of threads): 591
// MB back from e4m3 to bf16 took 93 us with four, 104 with one, 107 with eight.
constexpr int kMany = 4;

template <typename T, int D, bool E4M3>
int append_rows(const AppendArgs &a, cudaStream_t st) {
    const long long threads = static_cast<long long>(a.B) * a.M * a.c.Hkv * (D / kW);
    kv_append_kernel<T, D, E4M3><<<static_cast<unsigned>((threads + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

template <typename T, int D, bool E4M3>
int read_rows(const ReadArgs &a, cudaStream_t st) {
    const long long threads = static_cast<long long>(a.B) * a.M * a.c.Hkv * (D / kE);
    const bool large = threads > 152ll * 2048;
    const int per = large ? kMany : 1;
    const unsigned grid = static_cast<unsigned>((threads + kThreads * per - 1) / (kThreads * per));
    if (large)
        kv_read_kernel<T, D, E4M3, kMany><<<grid, kThreads, 0, st>>>(a);
    else
        kv_read_kernel<T, D, E4M3, 1><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

int launch_kv_append(const AppendArgs &a, int dtype, cudaStream_t st) {
    const bool e = a.c.e4m3 != 0, wide = a.c.D == 128;
    if (dtype == SPEC_F32)
        return e ? (wide ? append_rows<float, 128, true>(a, st) : append_rows<float, 64, true>(a, st))
                 : (wide ? append_rows<float, 128, false>(a, st) : append_rows<float, 64, false>(a, st));
    using H = __nv_bfloat16;
    return e ? (wide ? append_rows<H, 128, true>(a, st) : append_rows<H, 64, true>(a, st))
             : (wide ? append_rows<H, 128, false>(a, st) : append_rows<H, 64, false>(a, st));
}

int launch_kv_read(const ReadArgs &a, int dtype, cudaStream_t st) {
    const bool e = a.c.e4m3 != 0, wide = a.c.D == 128;
    if (dtype == SPEC_F32)
        return e ? (wide ? read_rows<float, 128, true>(a, st) : read_rows<float, 64, true>(a, st))
                 : (wide ? read_rows<float, 128, false>(a, st) : read_rows<float, 64, false>(a, st));
    using H = __nv_bfloat16;
    return e ? (wide ? read_rows<H, 128, true>(a, st) : read_rows<H, 64, true>(a, st))
             : (wide ? read_rows<H, 128, false>(a, st) : read_rows<H, 64, false>(a, st));
}

}  // namespace specv
