// A beam search's selection over beams and vocabulary.
//
//   s(b, v) = beam_scores[b] + (x_bv - lse_b),   lse_b = m_b + log sum_v exp(x_bv - m_b)
//
// and of the K * V continuations of a group the K best, the lowest b * V + v first among equal scores.
//
// The logits are read once.  s is a monotone function of x within a row, so a chunk of a row contributes
// its K + 1 largest logits, its maximum and its sum of exponentials without knowing lse; a second kernel
// puts each row's lse together, scores what the chunks offer and takes the K best of the group.  Two logits
// that differ can round to one score, and then the lower place wins whatever its logit: the (K + 1)-th
// entry shows whether that can concern anything that a chunk left out, and then (rarely: beside scores so
// large that neighbouring logits fall together) the group's logits are searched for the places with
// exactly that score.  Rows that offer nothing (finished, no score) are not read.

#include <cmath>

#include "kda_serve.cuh"

namespace kda {
namespace {

constexpr int BT = 256;                       // threads
constexpr int BW = BT / 32;
constexpr int GROUPS = BT / 4;                // groups of four threads whose maxima bound the K-th logit
constexpr int CAP = 1024;                     // logits that a chunk compares with one another at the end
constexpr int THREAD_BYTES = 128;             // of logits in a thread's registers
static_assert(KDA_BEAM_MAX_K + 1 <= GROUPS, "the bound on the K-th logit");

// A value and its place as one whole number: larger values first, then lower places; no two are equal.
__device__ __forceinline__ unsigned order_bits(float x) {
    const unsigned u = __float_as_uint(x + 0.f);                 // -0 and 0 are one value
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ unsigned long long candidate(float x, unsigned place) {
    return ((unsigned long long)order_bits(x) << 32) | (0xFFFFFFFFu - place);
}
__device__ __forceinline__ float candidate_value(unsigned long long c) {
    const unsigned u = (unsigned)(c >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ unsigned candidate_place(unsigned long long c) { return 0xFFFFFFFFu - (unsigned)c; }

__device__ __forceinline__ float beam_score(float bs, float x, float lse) {
    const float s = bs + (x - lse);
    return s != s ? -INFINITY : s;
}

__device__ __forceinline__ float exp_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// The next value below a finite x in the logits' type.
__device__ __forceinline__ float below(float x, float) {
    const unsigned u = __float_as_uint(x + 0.f);
    return __uint_as_float(u == 0u ? 0x80000001u : u & 0x80000000u ? u + 1u : u - 1u);
}
__device__ __forceinline__ float below(float x, __nv_bfloat16) {
    const unsigned u = __float_as_uint(x + 0.f) >> 16;
    return __uint_as_float((u == 0u ? 0x8001u : u & 0x8000u ? u + 1u : u - 1u) << 16);
}

template <typename T>
constexpr int CHUNK = BT * THREAD_BYTES / (int)sizeof(T);        // logits of a CTA

template <typename T>
struct Workspace {
    float2* stats;               // [N * K][chunks] maximum, sum of exp(x - maximum)
    unsigned long long* list;    // [N * K][chunks][K + 1] largest logits, in order; 0: none
};
template <typename T>
__host__ __device__ inline Workspace<T> workspace(const BeamParams& p, int chunks) {
    Workspace<T> w;
    w.stats = reinterpret_cast<float2*>(p.workspace);
    w.list = reinterpret_cast<unsigned long long*>(w.stats + (size_t)p.N * p.K * chunks);
    return w;
}

// A row that is read: a beam that goes on and has a score.
__device__ __forceinline__ bool live(const BeamParams& p, int64_t row) {
    const float bs = p.beam_scores[row];
    return !(p.finished && p.finished[row]) && bs == bs && bs != -INFINITY;
}

// A thread's logits in registers: vector j of thread t holds the elements (j * BT + t) * PER .. + PER - 1 of
// the chunk, wherever the row starts, so that equal rows give equal sums.
template <typename T>
struct Logits {
    static constexpr int PER = 16 / (int)sizeof(T), NV = THREAD_BYTES / 16, COUNT = PER * NV;
    uint32_t w[THREAD_BYTES / 4];

    __device__ static int element(int i, int tid) { return (i / PER * BT + tid) * PER + i % PER; }
    __device__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
    __device__ void load(const T* x, int count, int tid) {
        if (reinterpret_cast<uintptr_t>(x) % 16 == 0) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int at = (j * BT + tid) * PER;
                if (at + PER <= count) {
                    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(x + at));
                    w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
                } else {
                    load_one_by_one(x, count, at, j);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) load_one_by_one(x, count, (j * BT + tid) * PER, j);
        }
    }

private:
    __device__ void load_one_by_one(const T* x, int count, int at, int j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (sizeof(T) == 4) {
                w[4 * j + e] = at + e < count ? __float_as_uint(x[at + e]) : 0xFF800000u;
            } else {
                const unsigned short* u = reinterpret_cast<const unsigned short*>(x);
                const int i = at + 2 * e;
                w[4 * j + e] = (i < count ? u[i] : 0xFF80u) | (i + 1 < count ? (uint32_t)u[i + 1] << 16 : 0xFF800000u);
            }
        }
    }
};

__device__ __forceinline__ unsigned long long warp_max(unsigned long long x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const unsigned long long y = __shfl_xor_sync(0xFFFFFFFFu, x, o);
        x = y > x ? y : x;
    }
    return x;
}

template <typename T>
__global__ void __launch_bounds__(BT) kda_beam_chunk_kernel(BeamParams p, int chunks) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ __align__(16) float group_max[GROUPS];
    __shared__ float warp_top[BW], warp_sum[BW], bound;
    __shared__ int found;
    __shared__ unsigned long long cand[CAP];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / chunks;
    const int chunk = blockIdx.x % chunks, L = p.K + 1;
    if (!live(p, row)) return;
    const int base = chunk * CHUNK<T>, count = min(p.V - base, CHUNK<T>);
    using X = Logits<T>;
    X x;
    x.load(static_cast<const T*>(p.logits) + row * p.row_stride + base, count, tid);

    float mine = -INFINITY;
#pragma unroll
    for (int i = 0; i < X::COUNT; ++i) mine = fmaxf(mine, x.get(i));
    float top = fmaxf(mine, __shfl_xor_sync(0xFFFFFFFFu, mine, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    if ((lane & 3) == 0) group_max[tid / 4] = top;
#pragma unroll
    for (int o = 4; o < 32; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (lane == 0) warp_top[warp] = top;
    if (tid == 0) found = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < BW; ++w) top = fmaxf(top, warp_top[w]);
    // the L-th largest of the groups' maxima: at least L logits are that large
    if (tid < GROUPS) {
        const float g = group_max[tid];
        int rank = 0;
#pragma unroll
        for (int j = 0; j < GROUPS / 4; ++j) {
            const float4 y = reinterpret_cast<const float4*>(group_max)[j];
            rank += (y.x > g || (y.x == g && 4 * j < tid)) + (y.y > g || (y.y == g && 4 * j + 1 < tid)) +
                    (y.z > g || (y.z == g && 4 * j + 2 < tid)) + (y.w > g || (y.w == g && 4 * j + 3 < tid));
        }
        if (rank == L - 1) bound = g;
    }
    // x - top first: the exponent of the largest logits, which make up the sum, is exact
    const float zero = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < X::COUNT; ++i) sum += exp_of(x.get(i) - zero);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) warp_sum[warp] = sum;
    __syncthreads();
    const float least = bound;
    if (mine >= least && mine > -INFINITY) {
#pragma unroll
        for (int i = 0; i < X::COUNT; ++i) {
            const float y = x.get(i);
            if (y >= least && y > -INFINITY) {
                const int at = atomicAdd(&found, 1);
                if (at < CAP) cand[at] = candidate(y, (unsigned)(base + X::element(i, tid)));
            }
        }
    }
    __syncthreads();
    const Workspace<T> w = workspace<T>(p, chunks);
    unsigned long long* list = w.list + (row * chunks + chunk) * L;
    if (tid == 0) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < BW; ++i) sum += warp_sum[i];
        w.stats[row * chunks + chunk] = make_float2(top, sum);
    }
    const int n = found;
    if (n <= CAP) {
        for (int i = tid; i < n; i += BT) {
            const unsigned long long c = cand[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += cand[j] > c;
            if (rank < L) list[rank] = c;
        }
        for (int i = n + tid; i < L; i += BT) list[i] = 0;
    } else {
        // many equal logits: the largest left, L times
        unsigned long long last = ~0ull;
        for (int k = 0; k < L; ++k) {
            unsigned long long best = 0;
#pragma unroll
            for (int i = 0; i < X::COUNT; ++i) {
                const float y = x.get(i);
                const unsigned long long c = candidate(y, (unsigned)(base + X::element(i, tid)));
                if (y > -INFINITY && c < last && c > best) best = c;
            }
            best = warp_max(best);
            if (lane == 0) cand[(k & 1) * BW + warp] = best;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < BW; ++i) best = cand[(k & 1) * BW + i] > best ? cand[(k & 1) * BW + i] : best;
            if (tid == 0) list[k] = best;
            last = best;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(BT) kda_beam_join_kernel(BeamParams p, int chunks) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float bs[KDA_BEAM_MAX_K], lse[KDA_BEAM_MAX_K];
    __shared__ unsigned char fin[KDA_BEAM_MAX_K], alive[KDA_BEAM_MAX_K];
    __shared__ unsigned long long best[KDA_BEAM_MAX_K], red[2][BW];
    __shared__ int doubt, counts[BW];
    const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = p.K, L = K + 1;
    const Workspace<T> w = workspace<T>(p, chunks);
    const float2* stats = w.stats + (int64_t)n * K * chunks;
    const unsigned long long* list = w.list + (int64_t)n * K * chunks * L;

    for (int b = warp; b < K; b += BW) {
        const int64_t row = (int64_t)n * K + b;
        const bool reads = live(p, row);
        float top = -INFINITY, sum = 0.f;
        if (reads) {
            for (int c = lane; c < chunks; c += 32) top = fmaxf(top, stats[b * chunks + c].x);
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            for (int c = lane; c < chunks; c += 32) {
                const float2 s = stats[b * chunks + c];
                sum += s.y * (s.x == -INFINITY ? 0.f : exp_of(s.x - top));
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        }
        if (lane == 0) {
            bs[b] = p.beam_scores[row];
            fin[b] = p.finished && p.finished[row];
            lse[b] = top + logf(sum);
            alive[b] = reads && top != -INFINITY && sum == sum;  // else every score of the row is -inf
        }
    }
    if (tid == 0) doubt = 0;
    __syncthreads();

    // the entries as scores with their places in the group; a finished beam offers its one word
    const int entries = K * chunks * L;
    auto entry = [&](int e) -> unsigned long long {
        const int b = e / (chunks * L);
        float s = -INFINITY;
        unsigned v = 0;
        if (alive[b]) {
            const unsigned long long c = list[e];
            if (c == 0) return 0;
            v = candidate_place(c);
            s = beam_score(bs[b], candidate_value(c), lse[b]);
        } else if (fin[b] && e == b * chunks * L) {
            v = (unsigned)p.eos;
            s = bs[b] != bs[b] ? -INFINITY : bs[b];
        }
        return s == -INFINITY ? 0 : candidate(s, (unsigned)b * p.V + v);
    };
    unsigned long long mine = 0;
    for (int e = tid; e < entries; e += BT) {
        const unsigned long long c = entry(e);
        mine = c > mine ? c : mine;
    }
    int chosen = 0;                                    // continuations with a score
    for (int k = 0; k < K; ++k) {
        unsigned long long c = warp_max(mine);
        if (lane == 0) red[k & 1][warp] = c;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < BW; ++i) c = red[k & 1][i] > c ? red[k & 1][i] : c;
        if (tid == 0) best[k] = c;
        if (c == 0) break;
        ++chosen;
        if (c == mine) {                               // this thread's next one
            mine = 0;
            for (int e = tid; e < entries; e += BT) {
                const unsigned long long d = entry(e);
                if (d < c && d > mine) mine = d;
            }
        }
    }
    __syncthreads();

    auto score_at = [&](int b, int v) -> float {
        if (fin[b]) return v == p.eos && bs[b] == bs[b] ? bs[b] : -INFINITY;
        if (!alive[b]) return -INFINITY;
        return beam_score(bs[b], to_float(static_cast<const T*>(p.logits)[((int64_t)n * K + b) * p.row_stride + v]), lse[b]);
    };
    if (chosen == K) {
        // Could a logit that a chunk left out share the last score?  It lies below the chunk's last entry.
        const float worst = candidate_value(best[K - 1]);
        for (int i = tid; i < K * chunks; i += BT) {
            const int b = i / chunks;
            const unsigned long long tail = alive[b] ? list[(int64_t)i * L + K] : 0;
            if (tail && beam_score(bs[b], below(candidate_value(tail), T()), lse[b]) >= worst) doubt = 1;
        }
        __syncthreads();
        if (doubt) {
            // everything above that score is chosen already; of those with exactly it, the lowest places
            int at = 0;
            while (at < K && candidate_value(best[at]) > worst) ++at;
            __syncthreads();
            constexpr int SPAN = 16;
            const int64_t places = (int64_t)K * p.V;
            for (int64_t t = 0; t < places && at < K; t += BT * SPAN) {
                int hits = 0;
                const int64_t from = t + (int64_t)tid * SPAN, to = min(from + SPAN, places);
                for (int64_t i = from; i < to; ++i) hits += score_at((int)(i / p.V), (int)(i % p.V)) == worst;
                int inc = hits;
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const int y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                    if (lane >= o) inc += y;
                }
                if (lane == 31) counts[warp] = inc;
                __syncthreads();
                int rank = at + inc - hits, all = 0;
                for (int i = 0; i < BW; ++i) {
                    if (i < warp) rank += counts[i];
                    all += counts[i];
                }
                if (hits && rank < K)
                    for (int64_t i = from; i < to && rank < K; ++i)
                        if (score_at((int)(i / p.V), (int)(i % p.V)) == worst) best[rank++] = candidate(worst, (unsigned)i);
                at += all;
                __syncthreads();
            }
        }
    } else if (tid == 0) {
        // too few: every score is listed, the lowest places without one follow
        unsigned place = 0;
        for (int k = chosen; k < K; ++k, ++place) {
            bool taken = true;
            while (taken) {
                taken = false;
                for (int i = 0; i < chosen; ++i) taken |= candidate_place(best[i]) == place;
                place += taken;
            }
            best[k] = candidate(-INFINITY, place);
        }
    }
    __syncthreads();
    if (tid < K) {
        const unsigned place = candidate_place(best[tid]);
        const int b = (int)(place / (unsigned)p.V), v = (int)(place % (unsigned)p.V);
        p.scores[n * K + tid] = candidate_value(best[tid]);
        p.parent[n * K + tid] = n * K + b;
        p.token[n * K + tid] = v;
        if (p.finished_out) p.finished_out[n * K + tid] = fin[b] || v == p.eos;
    }
}

template <typename T>
int chunk_count(int V) { return (V + CHUNK<T> - 1) / CHUNK<T>; }

template <typename T>
cudaError_t launch(const BeamParams& p, cudaStream_t s) {
    const int chunks = chunk_count<T>(p.V);
    kda_beam_chunk_kernel<T><<<(unsigned)p.N * p.K * chunks, BT, 0, s>>>(p, chunks);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(p.N);
    cfg.blockDim = dim3(BT);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kda_beam_join_kernel<T>, p, chunks);
}

}  // namespace

size_t beam_workspace(int32_t N, int32_t K, int32_t V, kda_dtype dt) {
    const size_t chunks = dt == KDA_DTYPE_BF16 ? chunk_count<__nv_bfloat16>(V) : chunk_count<float>(V);
    return (size_t)N * K * chunks * (sizeof(float2) + (K + 1) * sizeof(unsigned long long));
}

cudaError_t launch_beam_select(const BeamParams& p, kda_dtype dt, cudaStream_t s) {
    return dt == KDA_DTYPE_BF16 ? launch<__nv_bfloat16>(p, s) : launch<float>(p, s);
}

}  // namespace kda
