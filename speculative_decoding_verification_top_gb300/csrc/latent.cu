// latent.cu -- attention of a target pass's new tokens to a latent cache.
//
// For one query row (token i, head h) over the positions j it sees:
//   t_j = log2(e) scale q . (c_j, r_j);  m = max t_j;  l = sum 2^(t_j - m);
//   out = sum 2^(t_j - m) c_j / l.
//
// A warp takes a row and goes through its positions one at a time.

#include "target.cuh"

namespace specv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <int C>
__global__ void __launch_bounds__(kThreads) latent_kernel(const LatentArgs a) {
    constexpr int kW = C + 64, kPairs = kW / 64, kOut = C / 64;  // element pairs a lane
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= a.B * a.N * a.H) return;
    const int token = row / a.H, b = token / a.N, n = token - b * a.N, len = a.lens[b];
    uint32_t *out = reinterpret_cast<uint32_t *>(a.out + static_cast<long long>(row) * C);
    bool bad = len < 0 || len > a.width << a.c.page_shift;
    float2 q[kPairs], o[kOut] = {};
    const __nv_bfloat162 *pq =
        reinterpret_cast<const __nv_bfloat162 *>(a.q + token * a.q_stride + static_cast<long long>(row - token * a.H) * kW);
    for (int i = 0; i < kPairs; ++i) q[i] = __bfloat1622float2(pq[i * 32 + lane]);
    const float mul = a.scale * kLog2e;
    float m = kNegInf, l = 0.0f;
    const int first = len - a.N;
    for (int j = 0; j < len && !bad; ++j) {
        const int page = a.table[static_cast<long long>(b) * a.width + (j >> a.c.page_shift)];
        if (page < 0 || page >= a.c.num_pages) {
            bad = true;
            break;
        }
        if (j >= first && (a.mask ? a.mask[static_cast<long long>(token) * a.N + j - first] == 0 : j - first > n)) continue;
        const long long at = (static_cast<long long>(page) << a.c.page_shift) + (j & ((1 << a.c.page_shift) - 1));
        const __nv_bfloat162 *pk = reinterpret_cast<const __nv_bfloat162 *>(a.c.data + at * kW);
        float2 k[kPairs];
        float s = 0.0f;
        for (int i = 0; i < kPairs; ++i) {
            k[i] = __bfloat1622float2(pk[i * 32 + lane]);
            s = fmaf(q[i].x, k[i].x, fmaf(q[i].y, k[i].y, s));
        }
        for (int x = 16; x > 0; x /= 2) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= mul;
        const float top = fmaxf(m, s), keep = m == kNegInf ? 0.0f : ex2(m - top), w = ex2(s - top);
        m = top;
        l = l * keep + w;
        for (int i = 0; i < kOut; ++i) o[i] = make_float2(fmaf(w, k[i].x, o[i].x * keep), fmaf(w, k[i].y, o[i].y * keep));
    }
    if (bad) {
        l = NAN;
        if (lane == 0) atomicOr(a.err, static_cast<uint32_t>(SPEC_DATA_PAGE_RANGE));
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    for (int i = 0; i < kOut; ++i) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(o[i].x * inv, o[i].y * inv);
        out[i * 32 + lane] = *reinterpret_cast<const uint32_t *>(&y);
    }
    if (a.lse && lane == 0) a.lse[row] = l == 0.0f ? kNegInf : (m + log2f(l)) / kLog2e;
}

}  // namespace

size_t latent_work_bytes(int, int, int, int) { return 0; }

int launch_latent(const LatentArgs &a, cudaStream_t st) {
    const unsigned grid = (static_cast<unsigned>(a.B) * a.N * a.H + kWarps - 1) / kWarps;
    if (a.c.C == 512)
        latent_kernel<512><<<grid, kThreads, 0, st>>>(a);
    else if (a.c.C == 256)
        latent_kernel<256><<<grid, kThreads, 0, st>>>(a);
    else
        latent_kernel<128><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace specv
