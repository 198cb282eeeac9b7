// kvcache.cu -- writing new tokens' keys and values into the paged cache, and
// reading positions back.
//
//   bf16   x as it is (fp32 inputs rounded to nearest).
//   e4m3   a = max |x_d| over the row, e = the smallest integer with
//          a <= 448 * 2^e, byte = e4m3(x * 2^-e).  With a = m * 2^(E),
//          m in [1, 2): 448 = 1.75 * 2^8, so e = E - 8 + (m > 1.75), read off
//          a's own bits.  The scaling is exact, the byte the only rounding.
//
// Both kernels give a row of D elements to D / 8 lanes, 8 elements each (one
// 16-byte load of bf16), so that the row's maximum is a shuffle reduction of
// three or four steps.  They are bound by memory: each new element read once,
// each cache byte written once, and the reverse.

#include "attn.cuh"

namespace specv {
namespace {

constexpr int kE = 8;  // elements a lane handles

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&x)[kE]);

template <>
__device__ __forceinline__ void load8<float>(const float *p, float (&x)[kE]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float (&x)[kE]) {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&x)[kE]);

template <>
__device__ __forceinline__ void store8<float>(float *p, const float (&x)[kE]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16 *p, const float (&x)[kE]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                               pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// One row's share: quantise (or round) x and write it to cache row `row` if
// the row is live.  Whole warps call it: the maximum is a shuffle reduction
// over the row's D / 8 lanes.
template <int D, bool E4M3>
__device__ __forceinline__ void write_row(uint8_t *data, int8_t *exps, long long row, int part,
                                          bool live, const float (&x)[kE]) {
    if (!E4M3) {
        if (live) store8(reinterpret_cast<__nv_bfloat16 *>(data) + row * D + part * kE, x);
        return;
    }
    uint32_t a = 0;  // bits of the largest finite |x|: ordered as integers
#pragma unroll
    for (int i = 0; i < kE; ++i) {
        const uint32_t u = __float_as_uint(x[i]) & 0x7fffffffu;
        a = max(a, u < 0x7f800000u ? u : 0u);
    }
#pragma unroll
    for (int s = D / kE / 2; s > 0; s /= 2) a = max(a, __shfl_xor_sync(0xffffffffu, a, s));
    int e = static_cast<int>(a >> 23) - 127 - 8 + ((a & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = a == 0 ? 0 : max(-120, min(120, e));
    const float f = exp2i(-e);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kE; ++i) {
        const uint32_t u = __float_as_uint(x[i]) & 0x7fffffffu;
        const uint32_t b = u < 0x7f800000u
                               ? __nv_cvt_float_to_fp8(x[i] * f, __NV_SATFINITE, __NV_E4M3)
                               : 0x7fu;
        w[i / 4] |= b << (8 * (i % 4));
    }
    if (!live) return;
    *reinterpret_cast<uint2 *>(data + row * D + part * kE) = make_uint2(w[0], w[1]);
    if (part == 0) exps[row] = static_cast<int8_t>(e);
}

template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendArgs a) {
    constexpr int kLanes = D / kE;  // lanes a row
    const long long items = static_cast<long long>(a.B) * a.M * a.c.Hkv;
    const long long item = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
    const int part = threadIdx.x % kLanes;
    int page = -1, slot = 0, h = 0;
    long long src = 0;
    if (item < items) {
        h = static_cast<int>(item % a.c.Hkv);
        const long long bt = item / a.c.Hkv;
        const int b = static_cast<int>(bt / a.M), t = static_cast<int>(bt % a.M);
        const int r = a.rows ? a.rows[bt] : t;
        const long long p = static_cast<long long>(a.starts[b]) + t;
        if (r >= 0 && r < a.N && p <= INT_MAX)
            page = page_of(a.c, a.table + static_cast<long long>(b) * a.width, a.width,
                           static_cast<int>(p), &slot);
        src = (static_cast<long long>(b) * a.N + r) * a.stride + h * D + part * kE;
    }
    const bool live = page >= 0;
    float k[kE] = {}, v[kE] = {};
    if (live) {
        load8(static_cast<const T *>(a.k) + src, k);
        load8(static_cast<const T *>(a.v) + src, v);
    }
    const long long row = live ? cache_row(a.c, page, h, slot) : 0;
    write_row<D, E4M3>(a.c.k, a.c.k_exp, row, part, live, k);
    write_row<D, E4M3>(a.c.v, a.c.v_exp, row, part, live, v);
}

// Eight elements of cache row `row` as fp32.
template <int D, bool E4M3>
__device__ __forceinline__ void read_row(const uint8_t *data, const int8_t *exps, long long row,
                                         int part, float (&x)[kE]) {
    if (!E4M3) {
        load8(reinterpret_cast<const __nv_bfloat16 *>(data) + row * D + part * kE, x);
        return;
    }
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(data + row * D + part * kE));
    const float f = exp2i(exps[row]);
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int i = 0; i < kE; i += 2) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>(w[i / 4] >> (8 * (i % 4))), __NV_E4M3);
        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        x[i] = y.x * f;
        x[i + 1] = y.y * f;
    }
}

template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadArgs a) {
    constexpr int kLanes = D / kE;
    const long long items = static_cast<long long>(a.B) * a.M * a.c.Hkv;
    const long long item = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) / kLanes;
    if (item >= items) return;
    const int part = threadIdx.x % kLanes;
    const int h = static_cast<int>(item % a.c.Hkv);
    const long long bt = item / a.c.Hkv;
    const int b = static_cast<int>(bt / a.M), t = static_cast<int>(bt % a.M);
    const long long p = static_cast<long long>(a.starts[b]) + t;
    int slot = 0;
    const int page = p > INT_MAX ? -1
                                 : page_of(a.c, a.table + static_cast<long long>(b) * a.width,
                                           a.width, static_cast<int>(p), &slot);
    float k[kE] = {}, v[kE] = {};
    if (page >= 0) {
        const long long row = cache_row(a.c, page, h, slot);
        if (a.out_k) read_row<D, E4M3>(a.c.k, a.c.k_exp, row, part, k);
        if (a.out_v) read_row<D, E4M3>(a.c.v, a.c.v_exp, row, part, v);
    }
    const long long o = item * D + part * kE;
    if (a.out_k) store8(static_cast<T *>(a.out_k) + o, k);
    if (a.out_v) store8(static_cast<T *>(a.out_v) + o, v);
}

template <typename Kernel, typename Args>
int launch_rows(Kernel kernel, const Args &a, cudaStream_t st) {
    const long long threads = static_cast<long long>(a.B) * a.M * a.c.Hkv * (a.c.D / kE);
    kernel<<<static_cast<unsigned>((threads + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

int launch_kv_append(const AppendArgs &a, int dtype, cudaStream_t st) {
    const bool e = a.c.e4m3 != 0, wide = a.c.D == 128;
    if (dtype == SPEC_F32)
        return launch_rows(e ? (wide ? kv_append_kernel<float, 128, true> : kv_append_kernel<float, 64, true>)
                             : (wide ? kv_append_kernel<float, 128, false> : kv_append_kernel<float, 64, false>),
                           a, st);
    return launch_rows(e ? (wide ? kv_append_kernel<__nv_bfloat16, 128, true>
                                 : kv_append_kernel<__nv_bfloat16, 64, true>)
                         : (wide ? kv_append_kernel<__nv_bfloat16, 128, false>
                                 : kv_append_kernel<__nv_bfloat16, 64, false>),
                       a, st);
}

int launch_kv_read(const ReadArgs &a, int dtype, cudaStream_t st) {
    const bool e = a.c.e4m3 != 0, wide = a.c.D == 128;
    if (dtype == SPEC_F32)
        return launch_rows(e ? (wide ? kv_read_kernel<float, 128, true> : kv_read_kernel<float, 64, true>)
                             : (wide ? kv_read_kernel<float, 128, false> : kv_read_kernel<float, 64, false>),
                           a, st);
    return launch_rows(e ? (wide ? kv_read_kernel<__nv_bfloat16, 128, true>
                                 : kv_read_kernel<__nv_bfloat16, 64, true>)
                         : (wide ? kv_read_kernel<__nv_bfloat16, 128, false>
                                 : kv_read_kernel<__nv_bfloat16, 64, false>),
                       a, st);
}

}  // namespace specv
