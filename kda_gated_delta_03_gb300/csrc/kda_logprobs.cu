// Log probabilities of given tokens, with entropy and top alternatives, and their gradient.
//
//   m = max x_j,  r = sum over the others of exp(x_j - m):   lse = m + log1p(r),  log p_y = (x_y - m) - log1p(r)
//   H = -sum p_j log p_j = log1p(r) - sum exp(x_j - m) (x_j - m) / (1 + r)
//   d / dx_j = g (1[j = y] - p_j) - h p_j (log p_j + H)      for g = d log p_y, h = dH
//
// The largest logit stays out of the sum r at every level (lane, warp, CTA, cluster), so that a word with nearly all
// the probability keeps its small -log p to fp32's relative precision: 1 + r would round it to 6e-8.
//
// One pass over the logits.  A row, or its parts on the CTAs of a cluster where there are few rows, streams through a ring
// of chunks in shared memory, the next ones under way while one is summed; a warp's lanes share their maximum, so that a rescale
// is a branch that all of them take or none.  The best words are gathered on the way: the top-th best of 64 maxima, taken after
// 1, 4, 16 .. chunks, bounds them from below, and vectors with a word above that, some hundreds a row, are written down and
// looked at again when the row is through.  Rows with too many (words in order, equal logits, fewer words above -inf than
// `top`) are gone through once more with the bound brought up to date after every chunk: 2,048 rows of 131,072 bf16 words with
// three allowed and top 5 take 450 us, ordinary ones 110.  Nothing depends on the order of the atomics: they place candidates
// in a list whose entries are then ranked.  Short rows are a chain of about ten barriers for a load or two: 20,000 rows of 500
// and of 2,000 bf16 words 90 and 104 us with top 5, 45 and 52 without.
//
// The gradient at the given word is g - g p, each in fp32: off by 6e-8 of g also where p is next to 1, unlike -log p.
#include <cooperative_groups.h>

#include "kda_prompt.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int NT = 128, NW = NT / 32;
constexpr int LOADS = 2;                      // 16-byte loads of a thread and chunk
constexpr int STAGES = 3;                     // chunks under way (2, 3, 4: 121.5, 119.4, 119.7 us)
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr int GROUPS = 64;                    // of threads, whose maxima give the bound: twice as many as a top may ask for
constexpr int MAX_TOP = KDA_LOGPROBS_MAX_TOP, MAX_CLUSTER = 8;

// Vectors of a row that are looked at again, for a list of that many words (1: no list).
constexpr int vectors_of(int list) { return list == 1 ? 1 : 2 * list > 1200 ? 2 * list : 1200; }

template <typename T>
struct Elems {
    static constexpr int W = 16 / sizeof(T), EPT = LOADS * W, CHUNK = NT * EPT;
    static constexpr int LIST = MAX_TOP + MAX_TOP * EPT;      // kept ones, and all words of `top` threads
    static constexpr int VECTORS = vectors_of(LIST);
};

__device__ __forceinline__ void unpack(const uint4& r, float* x, __nv_bfloat16) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& r, float* x, float) {
    x[0] = __uint_as_float(r.x), x[1] = __uint_as_float(r.y), x[2] = __uint_as_float(r.z), x[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ uint32_t bits16(__nv_bfloat16 x) { return __bfloat16_as_ushort(x); }

// The words from e0 on, as a vector of 16 bytes; what lies outside the row reads as -inf.
__device__ __forceinline__ uint4 load_vec(const __nv_bfloat16* row, int64_t e0, int V) {
    if (e0 >= 0 && e0 + 8 <= V) return __ldcs(reinterpret_cast<const uint4*>(row + e0));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t a = e0 + 2 * i, b = a + 1;
        const uint32_t lo = a >= 0 && a < V ? bits16(row[a]) : 0xFF80u, hi = b >= 0 && b < V ? bits16(row[b]) : 0xFF80u;
        w[i] = lo | hi << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 load_vec(const float* row, int64_t e0, int V) {
    if (e0 >= 0 && e0 + 4 <= V) return __ldcs(reinterpret_cast<const uint4*>(row + e0));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = e0 + i >= 0 && e0 + i < V ? __float_as_uint(row[e0 + i]) : 0xFF800000u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// A word's place in the order: larger values first, then lower words.  A value that is not a number counts as -inf.
__device__ __forceinline__ unsigned long long key_of(float x, int word) {
    x = x != x ? -INFINITY : x + 0.f;
    const uint32_t b = __float_as_uint(x), o = b & 0x80000000u ? ~b : b | 0x80000000u;
    return (unsigned long long)o << 32 | (0xFFFFFFFFu - (uint32_t)word);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ int key_word(unsigned long long k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }

// Sums of a set of words: reference m, r without one word that has it, and sum exp(x - m) (x - m) log2 e.
struct Sums {
    float m, r, t;
};
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
    const Sums &hi = a.m >= b.m ? a : b, &lo = a.m >= b.m ? b : a;
    if (lo.m == -INFINITY) return Sums{hi.m, hi.r + lo.r, hi.t};           // nothing there, or a NaN to hand on
    const float d = (lo.m - hi.m) * LOG2E, f = exp2_approx(d), all = 1.f + lo.r;
    return Sums{hi.m, hi.r + all * f, hi.t + (f > 0.f ? f * (lo.t + all * d) : 0.f)};
}

template <int LIST>
struct alignas(16) Shared {
    unsigned long long list[LIST + 2];        // (two more: it is ranked in pairs)
    int vectors[vectors_of(LIST)];
    unsigned long long best[MAX_CLUSTER * MAX_TOP > NT ? MAX_CLUSTER * MAX_TOP : NT];      // thread maxima; at the end the best of all CTAs
    float most[GROUPS];                       // group maxima
    float least;
    unsigned long long out[MAX_TOP];
    unsigned long long bound;                 // key of the k-th best so far, 0 with fewer
    Sums sums[NW];
    Sums cta;
    int count, found;
};

// How many of n keys, in pairs from a 16-byte place, are above k; keys[n] may be anything.
__device__ __forceinline__ int keys_above(const unsigned long long* keys, int n, unsigned long long k) {
    int rank = 0;
    const ulonglong2* pairs = reinterpret_cast<const ulonglong2*>(keys);
#pragma unroll 8
    for (int j = 0; j < n / 2; ++j) {
        const ulonglong2 x = pairs[j];
        rank += (x.x > k) + (x.y > k);
    }
    if (n & 1) rank += keys[n - 1] > k;
    return rank;
}

// Ranks the list and keeps its best `top` in out, in order; all threads.
template <int LIST>
__device__ __forceinline__ void rank_list(Shared<LIST>& sm, int top, int tid) {
    const int n = sm.count;
    for (int e = tid; e < n; e += NT) {
        const unsigned long long k = sm.list[e];
        const int rank = keys_above(sm.list, n, k);
        if (rank < top) sm.out[rank] = k;
    }
    __syncthreads();
    if (tid == 0) {
        sm.found = n < top ? n : top;
        sm.bound = n >= top ? sm.out[top - 1] : 0ull;
    }
    __syncthreads();
}

// Takes a chunk's words into the list, whatever they are, and leaves the best `top` so far in list and out; all threads.
// The top-th best thread maximum bounds the words that can be among the best: at most `top` threads hold one.
template <int EPT, int W, int LIST>
__device__ __forceinline__ void absorb(Shared<LIST>& sm, const float (&x)[EPT], int64_t e0, int V, int top, int tid) {
    const unsigned long long bound = sm.bound;
    unsigned long long best = 0;
    auto key = [&](int i) {
        const int64_t word = e0 + (int64_t)(i / W) * NT * W + i % W;
        return word >= 0 && word < V ? key_of(x[i], (int)word) : 0ull;
    };
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
        const unsigned long long k = key(i);
        if (k > bound && k > best) best = k;
    }
    sm.best[tid] = best;
    __syncthreads();
    unsigned long long tau = 1;               // every warp finds it for itself
    for (int w = 0; w < NW; ++w) {
        const unsigned long long k = sm.best[w * 32 + (tid & 31)];
        const unsigned mine = __ballot_sync(0xFFFFFFFFu, k && keys_above(sm.best, NT, k) == top - 1);
        if (mine) tau = __shfl_sync(0xFFFFFFFFu, k, __ffs(mine) - 1);
    }
    if (best >= tau) {
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const unsigned long long k = key(i);
            if (k >= tau && k > bound) sm.list[atomicAdd(&sm.count, 1)] = k;
        }
    }
    __syncthreads();
    rank_list(sm, top, tid);
    if (tid < sm.found) sm.list[tid] = sm.out[tid];
    if (tid == 0) sm.count = sm.found;
    __syncthreads();
}

// CLUSTER: a row's parts lie on several CTAs.  A kernel of its own, since the code that joins them costs the loop registers where
// nothing is joined (2,048 rows of 131,072 words 127 us against 119).
template <typename T, bool TOP, bool ENTROPY, bool CLUSTER>
__global__ void __launch_bounds__(NT, 8) kda_logprobs_kernel(LogprobParams p, int clusters) {
    using E = Elems<T>;
    constexpr int W = E::W, EPT = E::EPT, CHUNK = E::CHUNK;
    __shared__ Shared<TOP ? E::LIST : 1> sm;
    __shared__ uint4 ring[STAGES][LOADS][NT];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cluster = CLUSTER ? clusters : 1;
    const int64_t row = blockIdx.x / cluster;
    const int part = blockIdx.x % cluster;
    const T* x0 = static_cast<const T*>(p.logits) + row * p.row_stride;
    const int off = (int)(reinterpret_cast<uintptr_t>(x0) / sizeof(T) % W);
    const int chunks = (int)(((int64_t)p.V + off + CHUNK - 1) / CHUNK);
    const int c0 = (int)((int64_t)chunks * part / cluster), c1 = (int)((int64_t)chunks * (part + 1) / cluster);
    if (tid == 0) sm.count = 0, sm.found = 0, sm.bound = 0;
    __syncthreads();

    // Chunks come in through a ring that is STAGES deep: every thread copies its own vectors and takes them out again, so that
    // nobody waits for anybody.
    auto first = [&](int c) { return (int64_t)c * CHUNK + tid * W - off; };
    // chunks that lie in the row as a whole need no look at its ends
    const uint4* in = reinterpret_cast<const uint4*>(x0 - off) + tid;
    const int inner = off ? 1 : 0, outer = min((int)(((int64_t)p.V + off) / CHUNK), c1);
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(&ring[0][0][tid]);
    auto load = [&](int c, int stage) {
        if (c >= inner && c < outer) {
#pragma unroll
            for (int j = 0; j < LOADS; ++j)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(ring_at + (stage * LOADS + j) * (NT * 16)),
                             "l"(in + (int64_t)c * (LOADS * NT) + j * NT)
                             : "memory");
        } else if (c < c1) {
#pragma unroll 1
            for (int j = 0; j < LOADS; ++j) ring[stage][j][tid] = load_vec(x0, first(c) + j * (NT * W), p.V);
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    auto take = [&](float* x, int stage) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(STAGES - 1) : "memory");
#pragma unroll
        for (int j = 0; j < LOADS; ++j) unpack(ring[stage][j][tid], x + j * W, T());
    };
    float m = -INFINITY, r = 0.f, t = 0.f, least = -INFINITY, so_far = -INFINITY;    // m: of the warp
    int from = c0;                            // chunk that the bound is from
    bool own = false;                         // this lane holds the word that has m and stays out of r
#pragma unroll
    for (int i = 0; i < STAGES; ++i) load(c0 + i, i);
    for (int c = c0, stage = 0; c < c1; ++c, stage = stage + 1 == STAGES ? 0 : stage + 1) {
        float x[EPT];
        take(x, stage);
        load(c + STAGES, stage);
        float most[LOADS];
#pragma unroll
        for (int j = 0; j < LOADS; ++j) {
            most[j] = fmaxf(x[j * W], x[j * W + 1]);
#pragma unroll
            for (int i = 2; i < W; i += 2) most[j] = max3(most[j], x[j * W + i], x[j * W + i + 1]);
        }
        const float top_x = fmaxf(most[0], most[1]);
        if constexpr (TOP) {
            // The bound: the top-th best of the maxima of 64 groups of threads, so far; anew after 4, 16, 64 .. chunks, so that the
            // vectors written down grow with the logarithm of a row's length.  (All warps meet for it: 2,048 rows of 131,072
            // words 114 us, after 1, 2, 4 and 8 118; 400 rows of 260,000 fp32 words with top 32 91 us, with no later ones 677, since the
            // list ran over.)
            so_far = fmaxf(so_far, top_x);
            const uint32_t seen = (uint32_t)(c - c0) + 1;
            if ((seen & (seen - 1)) == 0 && (seen & 0x55555555u)) {
                float group = so_far;
#pragma unroll
                for (int o = 1; o < NT / GROUPS; o <<= 1) group = fmaxf(group, __shfl_xor_sync(0xFFFFFFFFu, group, o));
                if (tid % (NT / GROUPS) == 0) sm.most[tid / (NT / GROUPS)] = group;
                __syncthreads();
                if (warp == 0) {              // the smallest maximum with fewer than `top` above it
                    const float a = sm.most[lane], b = sm.most[lane + 32];
                    int above_a = 0, above_b = 0;
#pragma unroll 4
                    for (int j = 0; j < GROUPS / 4; ++j) {
                        const float4 y = reinterpret_cast<const float4*>(sm.most)[j];
                        above_a += (y.x > a) + (y.y > a) + (y.z > a) + (y.w > a);
                        above_b += (y.x > b) + (y.y > b) + (y.z > b) + (y.w > b);
                    }
                    float l = fminf(above_a < p.top ? a : INFINITY, above_b < p.top ? b : INFINITY);
#pragma unroll
                    for (int o = 16; o; o >>= 1) l = fminf(l, __shfl_xor_sync(0xFFFFFFFFu, l, o));
                    if (lane == 0) sm.least = l;
                }
                __syncthreads();
                least = sm.least;
                from = c;
            }
            // A word that equals the bound counts while the chunk that set it may hold it; in later chunks it is behind at
            // least `top` others.  (A NaN counts as -inf, which may be the bound.)
            if (c == from ? !(top_x < least) : top_x > least) {
#pragma unroll
                for (int j = 0; j < LOADS; ++j)
                    if (c == from ? !(most[j] < least) : most[j] > least) {
                        const int at = atomicAdd(&sm.count, 1);
                        if (at < E::VECTORS) sm.vectors[at] = (c * LOADS + j) * NT + tid;
                    }
            }
        }
        if (__any_sync(0xFFFFFFFFu, top_x > m)) {
            float all = top_x;
#pragma unroll
            for (int o = 16; o; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xFFFFFFFFu, all, o));
            if (m != -INFINITY) {
                const float d = (m - all) * LOG2E, f = exp2_approx(d), sum = r + (own ? 1.f : 0.f);
                if constexpr (ENTROPY) t = f > 0.f ? f * (t + sum * d) : 0.f;
                r = sum * f;
            }
            m = all;
            own = lane == __ffs(__ballot_sync(0xFFFFFFFFu, top_x == all)) - 1;
            if (own) {
                bool out = false;
#pragma unroll
                for (int i = 0; i < EPT; ++i)
                    if (!out && x[i] == all) {
                        x[i] = -INFINITY;
                        out = true;
                    }
            }
        }
        const float base = m == -INFINITY ? 0.f : m;
        Pair r2 = pair_of(0.f, 0.f), t2 = r2;
        const Pair minus = pair_of(-base, -base), by = pair_of(LOG2E, LOG2E);
#pragma unroll
        for (int i = 0; i < EPT; i += 2) {
            Pair y = mul2(add2(pair_of(x[i], x[i + 1]), minus), by);
            float2 v = both(y);
            if constexpr (ENTROPY) {          // 0 * -inf must not be met
                v = make_float2(max_nan(v.x, -1000.f), max_nan(v.y, -1000.f));
                y = pair_of(v.x, v.y);
            }
            const Pair e = pair_of(exp2_approx(v.x), exp2_approx(v.y));
            r2 = add2(r2, e);
            if constexpr (ENTROPY) t2 = fma2(e, y, t2);
        }
        r += both(r2).x + both(r2).y;
        if constexpr (ENTROPY) t += both(t2).x + both(t2).y;
    }

    bool given = false;                       // the row has a word to score
    float x_y = 0.f;
    if (tid == 0 && part == 0) {
        const int y = __ldg(p.tokens + row);
        if (y < -1 || y >= p.V) atomicOr(p.err, KDA_DEVERR_TOKEN);
        given = y >= 0 && y < p.V;
        if (given) x_y = (float)x0[y];        // (used at the end)
    }

    // ---- the warp's sums (its lanes have one m), the CTA's ----
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        r += __shfl_xor_sync(0xFFFFFFFFu, r, o);
        if constexpr (ENTROPY) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    }
    if (lane == 0) sm.sums[warp] = Sums{m, r, t};
    __syncthreads();
    if constexpr (TOP) {
        // the vectors written down, once more: their words from the bound up
        const int n = sm.count;
        __syncthreads();
        if (tid == 0) sm.count = 0;
        __syncthreads();
        if (n <= E::VECTORS) {
#pragma unroll 1
            for (int i = tid; i < n; i += NT) {
                const int64_t e = (int64_t)sm.vectors[i] * W - off;
                float x[W];
                unpack(load_vec(x0, e, p.V), x, T());
#pragma unroll
                for (int k = 0; k < W; ++k)
                    if (!(x[k] < least) && e + k >= 0 && e + k < p.V) {
                        const int at = atomicAdd(&sm.count, 1);
                        if (at < E::LIST) sm.list[at] = key_of(x[k], (int)(e + k));
                    }
            }
        }
        __syncthreads();
        if (n > E::VECTORS || sm.count > E::LIST || (c0 < c1 && sm.count < p.top)) {
            // Too many (words in order, equal logits), or NaNs where a bound was looked for: every chunk once more, the bound
            // brought up to date after each.
            __syncthreads();
            if (tid == 0) sm.count = 0, sm.found = 0, sm.bound = 0;
            __syncthreads();
            for (int c = c0; c < c1; ++c) {
                float x[EPT];
#pragma unroll
                for (int j = 0; j < LOADS; ++j) unpack(load_vec(x0, first(c) + j * (NT * W), p.V), x + j * W, T());
                absorb<EPT, W>(sm, x, first(c), p.V, p.top, tid);
            }
        } else {
            rank_list(sm, p.top, tid);
        }
    }
    if (tid == 0) {
        Sums s = sm.sums[0];
        for (int w = 1; w < NW; ++w) s = join(s, sm.sums[w]);
        sm.cta = s;
    }
    __syncthreads();

    // ---- the row's ----
    Sums s = sm.cta;
    if constexpr (CLUSTER) {
        cg::cluster_group group = cg::this_cluster();
        group.sync();
        if (part == 0) {
            // every warp fetches all CTAs' sums at once and joins them in their order
            const Sums theirs = *group.map_shared_rank(&sm.cta, lane < cluster ? lane : 0);
            for (int i = 1; i < cluster; ++i)
                s = join(s, Sums{__shfl_sync(0xFFFFFFFFu, theirs.m, i), __shfl_sync(0xFFFFFFFFu, theirs.r, i), __shfl_sync(0xFFFFFFFFu, theirs.t, i)});
            if constexpr (TOP) {
                const int n = cluster * p.top;                // `top` places of each CTA, 0 in those that it does not fill
                for (int x = tid; x < n; x += NT) {
                    const int i = x / p.top, e = x - i * p.top;
                    sm.best[x] = e < *group.map_shared_rank(&sm.found, i) ? group.map_shared_rank(sm.out, i)[e] : 0ull;
                }
                __syncthreads();
                for (int x = tid; x < n; x += NT) {
                    const unsigned long long k = sm.best[x];
                    const int rank = k ? keys_above(sm.best, n, k) : MAX_TOP;
                    if (rank < p.top) sm.list[rank] = k;
                }
                __syncthreads();
                if (tid < p.top) sm.out[tid] = sm.list[tid];
                __syncthreads();
            }
        }
        group.sync();
        if (part) return;
    }
    const float log_r = log1pf(s.r);
    const bool bad = s.r != s.r || s.m == INFINITY, empty = s.m == -INFINITY && !bad;
    const float nan = __int_as_float(0x7FC00000);
    auto log_p = [&](float x) { return bad ? nan : empty ? -INFINITY : (x - s.m) - log_r; };
    if (tid == 0) {
        p.logp[row] = given ? log_p(x_y) : 0.f;
        if (p.lse) p.lse[row] = bad ? nan : empty ? -INFINITY : s.m + log_r;
        if constexpr (ENTROPY) p.entropy[row] = bad ? nan : empty ? 0.f : log_r - LN2 * s.t / (1.f + s.r);
    }
    if constexpr (TOP) {
        if (tid < p.top) {
            const unsigned long long k = sm.out[tid];
            p.top_logp[row * p.top + tid] = log_p(key_value(k));
            p.top_token[row * p.top + tid] = key_word(k);
        }
    }
}

template <typename T, bool TOP, bool ENTROPY>
cudaError_t launch_forward(const LogprobParams& p, cudaStream_t s) {
    using E = Elems<T>;
    static DeviceSetup done;
    int sms = 0;
    cudaError_t e = device_setup(done, nullptr, 0, &sms);
    if (e != cudaSuccess) return e;
    // A row's parts go to a cluster where the rows alone would leave SMs idle and a part still has a chunk: up to two CTAs an SM.
    // 131,072 bf16 words with top 8, 77, 153, 304 and 400 rows: 20.4, 26.6, 28.6 and 34.6 us, with up to six CTAs an SM 18.0, 24.4,
    // 30.1 and 39.0; fp32 without top, 153 and 304 rows: 29.6 and 33.7, with six 17.1 and 28.4.
    int cluster = 1;
    while (cluster < MAX_CLUSTER && (int64_t)p.T * cluster * 2 <= 2 * sms && (int64_t)E::CHUNK * cluster < p.V) cluster *= 2;
    if (cluster == 1) {
        kda_logprobs_kernel<T, TOP, ENTROPY, false><<<(unsigned)p.T, NT, 0, s>>>(p, 1);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)(p.T * cluster));
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kda_logprobs_kernel<T, TOP, ENTROPY, true>, p, cluster);
}

template <typename T>
cudaError_t launch_any(const LogprobParams& p, cudaStream_t s) {
    if (p.top > 0) return p.entropy ? launch_forward<T, true, true>(p, s) : launch_forward<T, true, false>(p, s);
    return p.entropy ? launch_forward<T, false, true>(p, s) : launch_forward<T, false, false>(p, s);
}

// ------------------------------------------------------------------------------------------------
// the gradient
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ void store(float* p, float x) { *p = x; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ uint4 pack(const float* x, __nv_bfloat16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const float* x, float) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

constexpr int BACK = 4;
// A row's lse in fp32 is off by up to 2^-24 of its size, and p by that: beyond this size (6e-5) the row is summed up again.
constexpr float FAR_LSE = 1024.f;

// The gradient at W words whose logits x are taken against lse: -p (h (log p + H) + g), two words at a time; log p is held
// above -200, where p is 0, so that 0 * inf is not met.  The given word, `at` places into them, has g on top.
template <int W>
__device__ __forceinline__ void gradient(float (&x)[W], float lse, float g, float h, float H, int64_t at, bool given) {
    const Pair minus = pair_of(-lse, -lse), by = pair_of(LOG2E, LOG2E), h2 = pair_of(h, h), rest = pair_of(fmaf(h, H, g), fmaf(h, H, g));
#pragma unroll
    for (int i = 0; i < W; i += 2) {
        const float2 l = both(add2(pair_of(x[i], x[i + 1]), minus));
        const Pair lp = pair_of(max_nan(l.x, -200.f), max_nan(l.y, -200.f));
        const float2 z = both(mul2(lp, by));
        const float2 v = both(mul2(pair_of(-exp2_approx(z.x), -exp2_approx(z.y)), fma2(h2, lp, rest)));
        x[i] = v.x, x[i + 1] = v.y;
    }
    if (given && at >= 0 && at < W) {
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = i == at ? x[i] + g : x[i];
    }
}
template <typename T, int W>
__device__ __forceinline__ void store_vec(T* g0, int64_t e, int V, const float (&x)[W], bool together) {
    if (together && e >= 0 && e + W <= V) {
        __stcs(reinterpret_cast<uint4*>(g0 + e), pack(x, T()));
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
            if (e + i >= 0 && e + i < V) store(g0 + e + i, x[i]);
    }
}

// A whole row by one CTA: its maximum, its sum, its gradient, so that no rounding of lse matters.  (2,048 such rows of 131,072 bf16
// words take 454 us instead of 157.)
template <typename T>
__device__ __noinline__ void backward_row(const T* x0, T* g0, int V, int y, float g, float h, float H) {
    constexpr int W = Elems<T>::W;
    __shared__ float part[2][NW];
    const int tid = threadIdx.x, off = (int)(reinterpret_cast<uintptr_t>(x0) / sizeof(T) % W);
    const bool together = reinterpret_cast<uintptr_t>(x0) % 16 == reinterpret_cast<uintptr_t>(g0) % 16;
    float m = -INFINITY, sum = 0.f, x[W];
    for (int64_t e = (int64_t)tid * W - off; e < V; e += NT * W) {
        unpack(load_vec(x0, e, V), x, T());
#pragma unroll
        for (int i = 0; i < W; ++i) m = fmaxf(m, x[i]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (tid % 32 == 0) part[0][tid / 32] = m;
    __syncthreads();
    for (int w = 0; w < NW; ++w) m = fmaxf(m, part[0][w]);
    for (int64_t e = (int64_t)tid * W - off; e < V; e += NT * W) {
        unpack(load_vec(x0, e, V), x, T());
        float some = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) some += exp2_approx((x[i] - m) * LOG2E);
        sum += some;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (tid % 32 == 0) part[1][tid / 32] = sum;
    __syncthreads();
    sum = 0.f;
    for (int w = 0; w < NW; ++w) sum += part[1][w];
    const float log_sum = logf(sum);
    for (int64_t e = (int64_t)tid * W - off; e < V; e += NT * W) {
        unpack(load_vec(x0, e, V), x, T());
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] -= m;
        gradient(x, log_sum, g, h, H, y - e, y >= 0);
        store_vec(g0, e, V, x, together);
    }
}

// BACK vectors a thread, one chunk of a row a CTA.  Each vector is read before it is written, by the same thread, so the
// gradient may take the logits' place.  DRAM bounds it: 2,048 rows of 131,072 bf16 words 157 us (6.8 TB/s), with four as with eight
// vectors.
template <typename T>
__global__ void __launch_bounds__(NT) kda_logprobs_backward_kernel(LogprobGradParams p, int chunks) {
    using E = Elems<T>;
    constexpr int W = E::W;
    const int64_t row = blockIdx.x / chunks;
    const int c = blockIdx.x % chunks;
    const T* x0 = static_cast<const T*>(p.logits) + row * p.row_stride;
    T* g0 = static_cast<T*>(p.grad) + row * p.grad_stride;
    const int off = (int)(reinterpret_cast<uintptr_t>(x0) / sizeof(T) % W);
    const bool together = reinterpret_cast<uintptr_t>(x0) % 16 == reinterpret_cast<uintptr_t>(g0) % 16;
    const int64_t e0 = (int64_t)c * (BACK * NT * W) + threadIdx.x * W - off;
    uint4 raw[BACK];
#pragma unroll
    for (int j = 0; j < BACK; ++j) raw[j] = load_vec(x0, e0 + j * (NT * W), p.V);
    const int y0 = __ldg(p.tokens + row), y = y0 >= 0 && y0 < p.V ? y0 : -1;
    const float lse = __ldg(p.lse + row), g = y >= 0 ? __ldg(p.grad_logp + row) : 0.f;
    const float h = p.grad_entropy ? __ldg(p.grad_entropy + row) : 0.f, H = p.grad_entropy ? __ldg(p.entropy + row) : 0.f;
    if (fabsf(lse) > FAR_LSE && fabsf(lse) < INFINITY) {       // by the row's first CTA: the gradient may take the logits' place
        if (c == 0) backward_row(x0, g0, p.V, y, g, h, H);
        return;
    }
    const bool empty = lse == -INFINITY;      // a row with nothing above -inf has no gradient
#pragma unroll
    for (int j = 0; j < BACK; ++j) {
        const int64_t e = e0 + j * (NT * W);
        if (e >= p.V) break;
        float x[W];
        unpack(raw[j], x, T());
        gradient(x, lse, g, h, H, y - e, y >= 0);
        if (empty) {
#pragma unroll
            for (int i = 0; i < W; ++i) x[i] = 0.f;
        }
        store_vec(g0, e, p.V, x, together);
    }
}

template <typename T>
int64_t backward_chunks(int32_t V) {
    return ((int64_t)V + Elems<T>::W - 2 + BACK * NT * Elems<T>::W) / (BACK * NT * Elems<T>::W);
}

template <typename T>
cudaError_t launch_backward(const LogprobGradParams& p, cudaStream_t s) {
    const int64_t chunks = backward_chunks<T>(p.V);
    kda_logprobs_backward_kernel<T><<<(unsigned)(p.T * chunks), NT, 0, s>>>(p, (int)chunks);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobParams& p, kda_dtype dt, cudaStream_t s) {
    return dt == KDA_DTYPE_BF16 ? launch_any<__nv_bfloat16>(p, s) : launch_any<float>(p, s);
}

int64_t logprobs_backward_chunks(int32_t V, kda_dtype dt) {
    return dt == KDA_DTYPE_BF16 ? backward_chunks<__nv_bfloat16>(V) : backward_chunks<float>(V);
}

cudaError_t launch_token_logprobs_backward(const LogprobGradParams& p, kda_dtype dt, cudaStream_t s) {
    return dt == KDA_DTYPE_BF16 ? launch_backward<__nv_bfloat16>(p, s) : launch_backward<float>(p, s);
}

}  // namespace kda
