// target.cuh -- launch arguments of the rotary positions (rope.cu) and of the
// latent cache (rope.cu, latent.cu), for their C entries (target_api.cu).  Not a
// public header.
#pragma once

#include "attn.cuh"

namespace specv {

struct Turn {
    const unsigned long long *freqs;  // [rot / 2] 2^64 theta / (2 pi); null where rot is 0
    int rot, first;                   // elements turned, from this one of a head on
    float amplitude;
    int interleaved, inverse;
};

struct RopeArgs {
    const void *x;
    void *out;
    long long x_stride, out_stride;   // elements between consecutive tokens
    const int32_t *pos;
    int tokens, H, D;
    Turn t;
};

struct AppendRopeArgs {
    AppendArgs a;
    const int32_t *pos;               // [B, N] or null
    Turn t;
    const void *q;                    // [B, N, Hq, D] or null
    void *out_q;
    long long q_stride, out_q_stride;
    int Hq;
    unsigned kv_blocks;
};

struct LatentView {
    __nv_bfloat16 *data;              // [num_pages, page, C + R]
    int num_pages, page_shift, C, R;
};

struct LatentAppendArgs {
    LatentView c;
    const int32_t *table;
    int width;
    const int32_t *starts;
    const void *x, *r;                // [B, N, C], [B, N, R]
    long long x_stride, r_stride;
    const int32_t *rows, *pos;
    Turn t;
    int B, N, M;
};

struct LatentArgs {
    LatentView c;
    const int32_t *table;
    int width;
    const int32_t *lens;
    const __nv_bfloat16 *q;
    long long q_stride;
    const uint8_t *mask;
    int B, N, H;
    float scale;
    __nv_bfloat16 *out;
    float *lse;
    uint32_t *err;                    // the workspace's error word
    char *work;                       // the workspace after it
};

int launch_rope(const RopeArgs &a, int dtype, cudaStream_t st);
int launch_kv_append_rope(AppendRopeArgs &a, int dtype, cudaStream_t st);
int launch_latent_append(const LatentAppendArgs &a, int dtype, cudaStream_t st);
size_t latent_work_bytes(int B, int N, int H, int C);
int launch_latent(const LatentArgs &a, cudaStream_t st);

}  // namespace specv
