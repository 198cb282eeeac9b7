// attn.cuh -- launch arguments and device helpers shared by the cache and
// attention kernels (kvcache.cu, attn.cu) and their C entries (attn_api.cu).
// Not a public header.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "spec_attn.h"

namespace specv {

struct CacheView {
    uint8_t *k, *v;          // [num_pages, Hkv, page, D] elements
    int8_t *k_exp, *v_exp;   // [num_pages, Hkv, page] (e4m3), else unused
    int num_pages, Hkv, page_shift, D;
    int e4m3;
};

struct AppendArgs {
    CacheView c;
    const int32_t *table;
    int width;
    const int32_t *starts;
    const void *k, *v;
    long long stride;        // elements between consecutive tokens
    const int32_t *rows;     // [B, M] or null
    int B, N, M;
};

struct ReadArgs {
    CacheView c;
    const int32_t *table;
    int width;
    const int32_t *starts;
    void *out_k, *out_v;
    int B, M;
};

struct AttnArgs {
    CacheView c;
    const int32_t *shared_table;  // null without a prefix
    int shared_len;
    const int32_t *table;
    int width;
    const int32_t *lens;
    const __nv_bfloat16 *q;
    long long q_stride;
    const uint8_t *mask;
    const int32_t *pos;
    const float *slopes;
    int B, N, Hq, G;              // G = Hq / Hkv query heads per key/value head
    float scale, cap;
    int window;
    __nv_bfloat16 *out;
    float *lse;
    uint32_t *err;                // the workspace's error word
    char *work;                   // the workspace after it
};

// The page that holds `position` of a sequence and the slot in it; -1 where
// the table does not reach it or names no page.
__device__ __forceinline__ int page_of(const CacheView &c, const int32_t *table, int width,
                                       int position, int *slot) {
    if (position < 0) return -1;
    const int i = position >> c.page_shift;
    if (i >= width) return -1;
    *slot = position & ((1 << c.page_shift) - 1);
    const int id = table[i];
    return id < 0 || id >= c.num_pages ? -1 : id;
}

// Row (position) index of (page, head, slot) in the cache arrays; the
// element offset is this times D.  64 bits: a cache may pass 2^31 elements.
__device__ __forceinline__ long long cache_row(const CacheView &c, int page, int head, int slot) {
    return ((static_cast<long long>(page) * c.Hkv + head) << c.page_shift) + slot;
}

// 2^e in fp32 for e in [-126, 127].
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

int launch_kv_append(const AppendArgs &a, int dtype, cudaStream_t st);
int launch_kv_read(const ReadArgs &a, int dtype, cudaStream_t st);
size_t attn_work_bytes(int B, int N, int Hq, int Hkv, int D);
int launch_attn(const AttnArgs &a, cudaStream_t st);

}  // namespace specv
