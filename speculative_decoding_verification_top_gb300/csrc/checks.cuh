// checks.cuh -- argument checks shared by the C entries of include/spec_attn.h
// (attn_api.cu, target_api.cu).  Not a public header.
#pragma once

#include "attn.cuh"

#define SPEC_EXPORT extern "C" __attribute__((visibility("default")))

namespace specv {

constexpr size_t kErrBytes = 256;  // the workspace's error word, padded

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The cache descriptor's own checks; fills the kernels' view of it.
inline int view_of(const spec_kv_cache *cache, CacheView *c) {
    if (!cache) return SPEC_ERR_NULL;
    if (cache->dtype != SPEC_BF16 && cache->dtype != SPEC_E4M3) return SPEC_ERR_DTYPE;
    if (cache->num_pages < 1 || cache->Hkv < 1 || cache->Hkv > 1024 ||
        (cache->D != 64 && cache->D != 128) ||
        (cache->page != 16 && cache->page != 32 && cache->page != 64 && cache->page != 128) ||
        static_cast<long long>(cache->num_pages) * cache->Hkv > INT_MAX)
        return SPEC_ERR_SHAPE;
    const bool e4m3 = cache->dtype == SPEC_E4M3;
    if (!cache->k || !cache->v || (e4m3 && (!cache->k_exp || !cache->v_exp))) return SPEC_ERR_NULL;
    if (!aligned(cache->k, 16) || !aligned(cache->v, 16) ||
        (e4m3 && (!aligned(cache->k_exp, 4) || !aligned(cache->v_exp, 4))))
        return SPEC_ERR_ALIGN;
    c->k = static_cast<uint8_t *>(cache->k);
    c->v = static_cast<uint8_t *>(cache->v);
    c->k_exp = cache->k_exp;
    c->v_exp = cache->v_exp;
    c->num_pages = cache->num_pages;
    c->Hkv = cache->Hkv;
    c->page_shift = 31 - __builtin_clz(static_cast<unsigned>(cache->page));
    c->D = cache->D;
    c->e4m3 = e4m3;
    return SPEC_OK;
}

// A token stride: 0 stands for `packed`, else at least that and whole
// 16-byte groups of bf16.
inline bool stride_ok(int64_t *stride, long long packed) {
    if (*stride == 0) *stride = packed;
    return *stride >= packed && *stride % 8 == 0 && *stride <= (1LL << 40);
}

}  // namespace specv
