// Attention of one new token per sequence over a paged key-value cache.
//
//   s_t = scale * q . k_t,   o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),   m = max_t s_t
//
// in one pass: the running maximum and sum of the softmax, the sum over the values rescaled whenever the
// maximum grows.

#include <cmath>

#include "kda_serve.cuh"

namespace kda {
namespace {

constexpr int AT = 128;                       // threads: four warps, each on every fourth token

__device__ __forceinline__ bool visible(const AttnParams& p, int t, int len) {
    return t < len && (p.window == 0 || t >= len - p.window || t < p.sinks);
}

template <typename T, int D>
__global__ void __launch_bounds__(AT) kda_attn_simple_kernel(AttnParams p) {
    constexpr int W = AT / 32, E = (D + 31) / 32;
    const int b = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq, kvh = h / (p.Hq / p.Hkv);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ float sm_m[W], sm_l[W], sm_o[W][D];
    int len = p.lens[b];
    if (len < 0 || len > p.max_pages * p.page_size) {
        if (threadIdx.x == 0) atomicOr(p.err, KDA_DEVERR_PAGES);
        len = 0;
    }
    const T* q = static_cast<const T*>(p.q) + ((int64_t)b * p.Hq + h) * D;
    float qr[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qr[e] = lane + 32 * e < D ? to_float(q[lane + 32 * e]) * p.scale : 0.f;
        acc[e] = 0.f;
    }
    for (int t = warp; t < len; t += W) {
        if (!visible(p, t, len)) continue;
        int page = p.table[(int64_t)b * p.max_pages + t / p.page_size];
        if (page < 0 || page >= p.num_pages) {
            if (lane == 0) atomicOr(p.err, KDA_DEVERR_PAGES);
            page = 0;
        }
        const int64_t at = ((int64_t)kvh * p.page_size + t % p.page_size) * D;
        T* kc = static_cast<T*>(p.k_pages) + page * p.k_stride + at;
        T* vc = static_cast<T*>(p.v_pages) + page * p.v_stride + at;
        const bool is_new = p.k_new && t == len - 1;
        const int64_t nat = ((int64_t)b * p.Hkv + kvh) * D;
        const T* k = is_new ? static_cast<const T*>(p.k_new) + nat : kc;
        const T* v = is_new ? static_cast<const T*>(p.v_new) + nat : vc;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (lane + 32 * e < D) s += qr[e] * to_float(k[lane + 32 * e]);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
        const float c = expf(m - base), w = expf(s - base);
        l = l * c + w;
        m = mn;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (lane + 32 * e < D) {
                acc[e] = acc[e] * c + w * to_float(v[lane + 32 * e]);
                if (is_new && h % (p.Hq / p.Hkv) == 0) {
                    kc[lane + 32 * e] = k[lane + 32 * e];
                    vc[lane + 32 * e] = v[lane + 32 * e];
                }
            }
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (lane + 32 * e < D) sm_o[warp][lane + 32 * e] = acc[e];
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < W; ++w) top = fmaxf(top, sm_m[w]);
    const float base = top == -INFINITY ? 0.f : top;
    for (int w = 0; w < W; ++w) sum += sm_l[w] * expf(sm_m[w] - base);
    for (int i = threadIdx.x; i < D; i += AT) {
        float o = 0.f;
        for (int w = 0; w < W; ++w) o += sm_o[w][i] * expf(sm_m[w] - base);
        store_from_float(static_cast<T*>(p.o), ((int64_t)b * p.Hq + h) * D + i, sum > 0.f ? o / sum : 0.f);
    }
    if (p.lse && threadIdx.x == 0) p.lse[(int64_t)b * p.Hq + h] = sum > 0.f ? top + logf(sum) : -INFINITY;
}

template <typename T>
cudaError_t launch_simple(const AttnParams& p, cudaStream_t s) {
    const int grid = p.B * p.Hq;
    if (p.d == 16) kda_attn_simple_kernel<T, 16><<<grid, AT, 0, s>>>(p);
    else if (p.d == 64) kda_attn_simple_kernel<T, 64><<<grid, AT, 0, s>>>(p);
    else kda_attn_simple_kernel<T, 128><<<grid, AT, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t attn_workspace(int32_t, int32_t, int32_t, int32_t, kda_dtype) { return 0; }

cudaError_t launch_attention_decode(const AttnParams& p, kda_dtype dt, cudaStream_t s) {
    return dt == KDA_DTYPE_BF16 ? launch_simple<__nv_bfloat16>(p, s) : launch_simple<float>(p, s);
}

}  // namespace kda
