// A beam search's selection over beams and vocabulary.
//
//   s(b, v) = beam_scores[b] + (x_bv - lse_b),   lse_b = m_b + log sum_v exp(x_bv - m_b)
//
// and of the K * V continuations of a group the K best, the lowest b * V + v first among equal scores.

#include <cmath>

#include "kda_serve.cuh"

namespace kda {
namespace {

constexpr int BT = 256;

// Scores ordered as whole numbers, larger first, then the lowest place: no two candidates are equal.
__device__ __forceinline__ unsigned long long candidate(float s, unsigned place) {
    unsigned u = __float_as_uint(s + 0.f);                       // -0 and 0 are one score
    u = u & 0x80000000u ? ~u : u | 0x80000000u;
    return ((unsigned long long)u << 32) | (0xFFFFFFFFu - place);
}
__device__ __forceinline__ float candidate_score(unsigned long long c) {
    const unsigned u = (unsigned)(c >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ unsigned candidate_place(unsigned long long c) { return 0xFFFFFFFFu - (unsigned)c; }

__device__ __forceinline__ float beam_score(float bs, float x, float lse) {
    const float s = bs + (x - lse);
    return s != s ? -INFINITY : s;
}

template <typename T>
__global__ void __launch_bounds__(BT) kda_beam_simple_kernel(BeamParams p) {
    __shared__ float red[BT], lse[KDA_BEAM_MAX_K], bs[KDA_BEAM_MAX_K];
    __shared__ unsigned char fin[KDA_BEAM_MAX_K];
    __shared__ unsigned long long best[BT];
    const int n = blockIdx.x, tid = threadIdx.x;
    const T* x = static_cast<const T*>(p.logits) + (int64_t)n * p.K * p.row_stride;
    if (tid < p.K) {
        bs[tid] = p.beam_scores[n * p.K + tid];
        fin[tid] = p.finished && p.finished[n * p.K + tid];
    }
    for (int b = 0; b < p.K; ++b) {
        float m = -INFINITY;
        for (int v = tid; v < p.V; v += BT) {
            const float y = to_float(x[b * p.row_stride + v]);
            m = y != y || m != m ? NAN : fmaxf(m, y);
        }
        red[tid] = m;
        __syncthreads();
        for (int o = BT / 2; o; o /= 2) {
            if (tid < o) red[tid] = red[tid] != red[tid] || red[tid + o] != red[tid + o] ? NAN : fmaxf(red[tid], red[tid + o]);
            __syncthreads();
        }
        m = red[0];
        __syncthreads();
        float sum = 0.f;
        for (int v = tid; v < p.V; v += BT) sum += expf(to_float(x[b * p.row_stride + v]) - m);
        red[tid] = sum;
        __syncthreads();
        for (int o = BT / 2; o; o /= 2) {
            if (tid < o) red[tid] += red[tid + o];
            __syncthreads();
        }
        if (tid == 0) lse[b] = m + logf(red[0]);
        __syncthreads();
    }
    unsigned long long below = ~0ull;
    for (int k = 0; k < p.K; ++k) {
        unsigned long long mine = 0;
        for (int b = 0; b < p.K; ++b)
            for (int v = tid; v < p.V; v += BT) {
                const float s = fin[b] ? (v == p.eos && bs[b] == bs[b] ? bs[b] : -INFINITY)
                                       : beam_score(bs[b], to_float(x[b * p.row_stride + v]), lse[b]);
                const unsigned long long c = candidate(s, (unsigned)(b * p.V + v));
                if (c < below && c > mine) mine = c;
            }
        best[tid] = mine;
        __syncthreads();
        for (int o = BT / 2; o; o /= 2) {
            if (tid < o && best[tid + o] > best[tid]) best[tid] = best[tid + o];
            __syncthreads();
        }
        below = best[0];
        __syncthreads();
        if (tid == 0) {
            const unsigned place = candidate_place(below);
            const int b = place / p.V, v = place % p.V;
            p.scores[n * p.K + k] = candidate_score(below);
            p.parent[n * p.K + k] = n * p.K + b;
            p.token[n * p.K + k] = v;
            if (p.finished_out) p.finished_out[n * p.K + k] = fin[b] || v == p.eos;
        }
    }
}

}  // namespace

size_t beam_workspace(int32_t, int32_t, int32_t, kda_dtype) { return 0; }

cudaError_t launch_beam_select(const BeamParams& p, kda_dtype dt, cudaStream_t s) {
    if (dt == KDA_DTYPE_BF16) kda_beam_simple_kernel<__nv_bfloat16><<<p.N, BT, 0, s>>>(p);
    else kda_beam_simple_kernel<float><<<p.N, BT, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace kda
