// kvrows.cuh -- rows of the paged cache as they are loaded, rounded and stored:
// shared by the kernels that write them (kvcache.cu, rope.cu) and the one that
// reads them back.  Not a public header.
#pragma once

#include "attn.cuh"

namespace specv {

constexpr int kE = 8;  // elements of a vector: 16 bytes of bf16

__device__ __forceinline__ void widen8(uint4 u, float (&x)[kE]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

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
    widen8(__ldg(reinterpret_cast<const uint4 *>(p)), x);
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

// Two floats as e4m3 bytes (nearest, ties to even).
__device__ __forceinline__ uint32_t e4m3_bytes(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

constexpr int kW = 16;  // elements a lane writes, two vectors

// The e4m3 bytes w and the exponent of this lane's 16 elements of a row that
// D / 16 lanes hold.  Whole warps call it: the maximum is a shuffle reduction.
template <int D>
__device__ __forceinline__ int quantise(const float (&x)[2][kE], uint32_t (&w)[4]) {
    uint32_t a = 0;  // bits of the largest |x|: ordered as integers, NaN the largest
#pragma unroll
    for (int i = 0; i < kW; ++i) a = max(a, __float_as_uint(x[i / kE][i % kE]) & 0x7fffffffu);
#pragma unroll
    for (int s = D / kW / 2; s > 0; s /= 2) a = max(a, __shfl_xor_sync(0xffffffffu, a, s));
    const bool odd = __any_sync(0xffffffffu, a >= 0x7f800000u);
    if (odd) {  // once more over the finite ones
        a = 0;
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            const uint32_t u = __float_as_uint(x[i / kE][i % kE]) & 0x7fffffffu;
            a = max(a, u < 0x7f800000u ? u : 0u);
        }
#pragma unroll
        for (int s = D / kW / 2; s > 0; s /= 2) a = max(a, __shfl_xor_sync(0xffffffffu, a, s));
    }
    int e = static_cast<int>(a >> 23) - 127 - 8 + ((a & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = a == 0 ? 0 : max(-120, min(120, e));
    const float f = exp2i(-e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float *y = &x[i / 2][4 * (i % 2)];
        w[i] = e4m3_bytes(y[0] * f, y[1] * f) | e4m3_bytes(y[2] * f, y[3] * f) << 16;
    }
    if (odd) {
#pragma unroll
        for (int i = 0; i < kW; ++i)
            if ((__float_as_uint(x[i / kE][i % kE]) & 0x7fffffffu) >= 0x7f800000u)
                w[i / 4] = (w[i / 4] & ~(0xffu << 8 * (i % 4))) | 0x7fu << 8 * (i % 4);
    }
    return e;
}

}  // namespace specv
