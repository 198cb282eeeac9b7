// attn.cu -- attention of a target pass's new tokens to the paged cache.
//
// For one query row (token i, query head h) over the positions j it sees:
//   s_j = scale q.k_j, capped and biased;  m = max s_j;
//   l = sum 2^((s_j - m) log2 e);  out = sum 2^((s_j - m) log2 e) v_j / l.
// One pass: m, l and the output's accumulator are kept as running values,
// rescaled by 2^((m_old - m_new) log2 e) when the maximum grows.
//
// attn_kernel   one warp per query row, 32 positions at a time: a lane takes
//               a position's score, then the lanes take D / 32 output
//               elements each.

#include "attn.cuh"

namespace specv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <int D, bool E4M3>
__device__ __forceinline__ float element(const uint8_t *data, long long row, int d) {
    if (E4M3) {
        __nv_fp8_e4m3 x;
        x.__x = data[row * D + d];
        return static_cast<float>(x);
    }
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(data)[row * D + d]);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads) attn_kernel(const AttnArgs a) {
    __shared__ float qs[kWarps][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = static_cast<long long>(blockIdx.x) * kWarps + warp;
    if (row >= static_cast<long long>(a.B) * a.N * a.Hq) return;
    const int hq = static_cast<int>(row % a.Hq);
    const long long bn = row / a.Hq;
    const int b = static_cast<int>(bn / a.N), n = static_cast<int>(bn % a.N), h = hq / a.G;
    const __nv_bfloat16 *q = a.q + bn * a.q_stride + static_cast<long long>(hq) * D;
    for (int d = lane; d < D; d += 32) qs[warp][d] = __bfloat162float(q[d]);
    __syncwarp();
    const int32_t *table = a.table + static_cast<long long>(b) * a.width;
    const int most = a.width << a.c.page_shift;
    const int len = a.lens[b];
    bool bad = len < 0 || len > most;
    const int own = bad ? 0 : len, Ls = a.shared_len, total = Ls + own;
    const int first = own - a.N;  // own position of new token 0 (may be negative: padding)
    const int pos_i = a.pos ? a.pos[bn] : Ls + first + n;
    const float slope = a.slopes ? a.slopes[hq] : 0.0f;
    float m = kNegInf, l = 0.0f, acc[D / 32] = {};
    for (int j0 = 0; j0 < total; j0 += 32) {
        const int j = j0 + lane;
        bool seen = j < total;
        long long at = -1;
        float s = kNegInf;
        if (seen) {
            int slot = 0, page, pos_j = j;
            if (j < Ls) {
                page = page_of(a.c, a.shared_table, INT_MAX, j, &slot);
            } else {
                const int o = j - Ls, c = o - first;
                page = page_of(a.c, table, a.width, o, &slot);
                if (c >= 0) {  // a new token
                    seen = a.mask ? a.mask[bn * a.N + c] != 0 : c <= n;
                    if (a.pos) pos_j = a.pos[static_cast<long long>(b) * a.N + c];
                }
            }
            if (page < 0) bad = true;
            seen = seen && page >= 0 &&
                   (a.window == 0 || static_cast<long long>(pos_i) - pos_j < a.window);
            if (seen) {
                at = cache_row(a.c, page, h, slot);
                float x = 0.0f;
                for (int d = 0; d < D; ++d) x += qs[warp][d] * element<D, E4M3>(a.c.k, at, d);
                if (E4M3) x *= exp2i(a.c.k_exp[at]);
                x *= a.scale;
                if (a.cap > 0.0f) x = a.cap * tanhf(x / a.cap);
                s = (x - slope * static_cast<float>(pos_i - pos_j)) * kLog2e;
            }
        }
        float top = s;
        for (int o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float mn = fmaxf(m, top);
        if (mn == kNegInf) continue;
        const float keep = ex2(m - mn), p = seen ? ex2(s - mn) : 0.0f;
        m = mn;
        l = l * keep + p;
        for (int i = 0; i < D / 32; ++i) acc[i] *= keep;
        for (int t = 0; t < 32; ++t) {
            const long long r = __shfl_sync(0xffffffffu, at, t);
            if (r < 0) continue;
            float w = __shfl_sync(0xffffffffu, p, t);
            if (E4M3) w *= exp2i(a.c.v_exp[r]);
            for (int i = 0; i < D / 32; ++i) acc[i] += w * element<D, E4M3>(a.c.v, r, lane + 32 * i);
        }
    }
    for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(0xffffffffu, l, o);
    bad = __any_sync(0xffffffffu, bad);
    if (bad && lane == 0) atomicOr(a.err, static_cast<uint32_t>(SPEC_DATA_PAGE_RANGE));
    for (int i = 0; i < D / 32; ++i) {
        const float o = bad ? NAN : l > 0.0f ? acc[i] / l : l == 0.0f ? 0.0f : NAN;
        a.out[row * D + lane + 32 * i] = __float2bfloat16(o);
    }
    if (a.lse && lane == 0)
        a.lse[row] = bad ? NAN : m == kNegInf && l == 0.0f ? kNegInf : (m + log2f(l)) / kLog2e;
}

}  // namespace

size_t attn_work_bytes(int, int, int, int, int) { return 0; }

int launch_attn(const AttnArgs &a, cudaStream_t st) {
    const long long rows = static_cast<long long>(a.B) * a.N * a.Hq;
    const unsigned grid = static_cast<unsigned>((rows + kWarps - 1) / kWarps);
    auto kernel = a.c.D == 128 ? (a.c.e4m3 ? attn_kernel<128, true> : attn_kernel<128, false>)
                               : (a.c.e4m3 ? attn_kernel<64, true> : attn_kernel<64, false>);
    kernel<<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace specv
