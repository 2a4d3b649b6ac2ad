// A beam search's selection over beams and vocabulary.
//
//   s(b, v) = beam_scores[b] + (x_bv - lse_b),   lse_b = m_b + log sum_v exp(x_bv - m_b)
//
// and of the K * V continuations of a group the K best, the lowest b * V + v first among equal scores.
//
// The logits are read once.  s is a monotone function of x within a row, so a part of a row contributes
// its K + 1 largest logits, its maximum and its sum of exponentials without knowing lse; a second kernel
// puts each row's lse together, scores what the parts offer and takes the K best of the group.  Two logits
// that differ can round to one score, and then the lower place wins whatever its logit.  Whether that can concern
// anything that a part left out is seen from its list (best_left_out), and then (rarely: where neighbouring logits
// fall together at the last score that is chosen) the group's logits are searched for the places with exactly that
// score.  Rows that offer nothing (finished, no score) are not read.
//
// What it costs: 410 of 512 rows of 131,072 bf16 words (107 MB) take 27.5 us, of which the read at DRAM's rate
// would be 16.  Issue slots are the rest (8 instructions a logit; a plain stream of loads, exponentials and
// sums needs 4 and runs at DRAM's rate: the bound, the lists and the barriers around them make up the others), and 5 us
// of the second kernel, a chain of loads and small steps for each group.  As many fp32 rows (215 MB) take 42 us.  What
// costs more: rows in which more words reach the first chunk's bound than the lists hold (behind a finite mask that
// leaves a few words in all, 180 us), and the search for places, one CTA per group, up to 0.15 ms for each row of 131,072.

#include <cmath>

#include "kda_serve.cuh"

namespace kda {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int BT = 256;                       // threads
constexpr int BW = BT / 32;
constexpr int GROUPS = BT / 4;                // groups of threads whose maxima bound the K-th logit, at most
constexpr int FEW = 15;                       // beams up to which half as many groups bound it as well
constexpr int CAP = 512;                      // logits kept until they are compared with one another,
constexpr int WARP_CAP = CAP / BW;            // so many by each warp
constexpr int THREAD_BYTES = 64;              // of logits in a thread's registers
constexpr int CTAS_PER_SM = 3;
constexpr int STAGES = 4;                     // chunks of a warp in shared memory or on their way there
static_assert(KDA_BEAM_MAX_K + 1 <= WARP_CAP, "the best of all warps' go on in the first one's place");
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

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float exp_of(float x) { return exp2_approx(x * LOG2E); }

// The next value above x (-inf included) or below a finite x in the logits' type.
__device__ __forceinline__ float above(float x, float) {
    const unsigned u = __float_as_uint(x + 0.f);
    return __uint_as_float(u & 0x80000000u ? u - 1u : u + 1u);
}
__device__ __forceinline__ float above(float x, __nv_bfloat16) {
    const unsigned u = __float_as_uint(x + 0.f) >> 16;
    return __uint_as_float((u & 0x8000u ? u - 1u : u + 1u) << 16);
}
__device__ __forceinline__ float below(float x, float) {
    const unsigned u = __float_as_uint(x + 0.f);
    return __uint_as_float(u == 0u ? 0x80000001u : u & 0x80000000u ? u + 1u : u - 1u);
}
__device__ __forceinline__ float below(float x, __nv_bfloat16) {
    const unsigned u = __float_as_uint(x + 0.f) >> 16;
    return __uint_as_float((u == 0u ? 0x8001u : u & 0x8000u ? u + 1u : u - 1u) << 16);
}

template <typename T>
constexpr int CHUNK = BT * THREAD_BYTES / (int)sizeof(T);        // logits of a CTA at a time

template <typename T>
struct Workspace {
    float2* stats;               // [N * K][parts] t, and the sum of exp(x - t)
    unsigned long long* list;    // [N * K][parts][K + 1] largest logits, in order; 0: none
};
template <typename T>
__host__ __device__ inline Workspace<T> workspace(const BeamParams& p, int parts) {
    Workspace<T> w;
    w.stats = reinterpret_cast<float2*>(p.workspace);
    w.list = reinterpret_cast<unsigned long long*>(w.stats + (size_t)p.N * p.K * parts);
    return w;
}

// A row that is read: a beam that goes on and has a score.
__device__ __forceinline__ bool live(const BeamParams& p, int64_t row) {
    const float bs = p.beam_scores[row];
    return !(p.finished && p.finished[row]) && bs == bs && bs != -INFINITY;
}

// A pair of floats as the packed arithmetic takes them (two lanes of one instruction).
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t c;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(c) : "l"(a), "l"(b));
    return c;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t c;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(c) : "l"(a), "l"(b));
    return c;
}
__device__ __forceinline__ float lo_of(uint64_t a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float hi_of(uint64_t a) { return __uint_as_float((uint32_t)(a >> 32)); }

// 16 bytes from global to shared memory; zeros, and no read, where `read` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// A thread's logits of a chunk: vector j of thread t holds the elements (j * BT + t) * PER .. + PER - 1, wherever
// the row starts, so that equal rows give equal sums.
//
// A row may start `off` elements past a 16-byte boundary.  Its vectors are copied as they lie between
// boundaries, 33 for the 32 of a warp, and put into place on the way to the registers; so a warp needs
// nothing that another one copies.
template <typename T>
struct Logits {
    static constexpr int PER = 16 / (int)sizeof(T), NV = THREAD_BYTES / 16;
    static constexpr int WARP_BYTES = NV * 33 * 16;    // of a chunk
    uint32_t w[4 * NV];

    // The copies of chunk `chunk` of a row of V logits at v (rounded down to the boundary).
    __device__ static void copy(uint32_t ring, const uint4* v, int chunk, int off, int V, int tid) {
        const int lane = tid & 31;
        if ((int64_t)(chunk + 1) * CHUNK<T> + PER <= V) {              // not the row's end
            const uint4* from = v + chunk * (NV * BT) + tid;
            const uint32_t to = ring + lane * 16;
#pragma unroll
            for (int j = 0; j < NV; ++j) copy16(to + j * (33 * 16), from + j * BT, true);
            if (off && lane == 0) {
#pragma unroll
                for (int j = 0; j < NV; ++j) copy16(to + j * (33 * 16) + 32 * 16, from + j * BT + 32, true);
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int at = (chunk * NV + j) * BT + tid;
            copy16(ring + (j * 33 + lane) * 16, v + at, at * PER - off < V);
            if (off && lane == 0) copy16(ring + (j * 33 + 32) * 16, v + at + 32, (at + 32) * PER - off < V);
        }
    }
    // ... and to the registers; `count` elements of the chunk exist
    __device__ void take(uint32_t ring, int off, int count, int tid) {
        const int lane = tid & 31, words = off * (int)sizeof(T) / 4;
        const bool half = off * (int)sizeof(T) % 4 != 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const uint4 a = shared16(ring + (j * 33 + lane) * 16);
            w[4 * j] = a.x; w[4 * j + 1] = a.y; w[4 * j + 2] = a.z; w[4 * j + 3] = a.w;
        }
        if (off) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const uint4 b = shared16(ring + (j * 33 + lane + 1) * 16);
                uint32_t u[9] = {w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3], b.x, b.y, b.z, b.w, 0};
                if (words & 1) {
#pragma unroll
                    for (int e = 0; e < 7; ++e) u[e] = u[e + 1];
                }
                if (words & 2) {
#pragma unroll
                    for (int e = 0; e < 5; ++e) u[e] = u[e + 2];
                }
                if (half) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) u[e] = __funnelshift_r(u[e], u[e + 1], 16);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) w[4 * j + e] = u[e];
            }
        }
        if (count < CHUNK<T>) {
#pragma unroll
            for (int i = 0; i < 4 * NV; ++i) {
                const int at = (i / 4 * BT + tid) * PER + i % 4 * (4 / (int)sizeof(T));
                if constexpr (sizeof(T) == 4) {
                    if (at >= count) w[i] = 0xFF800000u;
                } else {
                    if (at >= count) w[i] = (w[i] & 0xFFFF0000u) | 0xFF80u;
                    if (at + 1 >= count) w[i] = (w[i] & 0xFFFFu) | 0xFF800000u;
                }
            }
        }
    }
    // element i of thread `owner` of this warp, from shared memory
    __device__ static float element(uint32_t ring, int off, int owner, int i) {
        const uint32_t at = ring + (i / PER * 33 + owner) * 16 + (i % PER + off) * (int)sizeof(T);
        if constexpr (sizeof(T) == 4) {
            float x;
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
            return x;
        } else {
            unsigned short x;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at) : "memory");
            return __uint_as_float((uint32_t)x << 16);
        }
    }
    __device__ float max() const {
        if constexpr (sizeof(T) == 4) {
            float m = __uint_as_float(w[0]);
#pragma unroll
            for (int i = 1; i < 4 * NV; ++i) m = fmaxf(m, __uint_as_float(w[i]));
            return m;
        } else {
            const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(w);
            __nv_bfloat162 m = h[0];
#pragma unroll
            for (int i = 1; i < 4 * NV; ++i) m = __hmax2(m, h[i]);
            return fmaxf(__low2float(m), __high2float(m));
        }
    }
    // sum of exp(x - t): the difference first, so that neither large logits nor large masks lose anything
    __device__ float sum_exp(float t) const {
        const uint64_t scale = pair(LOG2E, LOG2E), off = pair(-t, -t);
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < 4 * NV / (sizeof(T) == 4 ? 2 : 1); ++i) {
            uint64_t x;
            if constexpr (sizeof(T) == 4) x = (uint64_t)w[2 * i + 1] << 32 | w[2 * i];
            else x = (uint64_t)(w[i] & 0xFFFF0000u) << 32 | (w[i] << 16);
            x = mul2(add2(x, off), scale);
            sum = add2(sum, pair(exp2_approx(lo_of(x)), exp2_approx(hi_of(x))));
        }
        return lo_of(sum) + hi_of(sum);
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

// The best score (or more) among the logits that a part left out of its list and that may have to be chosen all the same.
// Such a logit has at most K - 1 others before it, so two at least of the K + 1 listed ones come after it: with its
// score, at higher places, and listed only since they are larger.  It is below the list's last logit x, or equals it;
// the latter only where two listed logits above x share x's score.  (Equal logits alone are no such case.)
template <typename T>
__device__ float best_left_out(const unsigned long long* list, int K, unsigned long long last, float bs, float lse) {
    const float x = candidate_value(last), s = beam_score(bs, x, lse), under = beam_score(bs, below(x, T()), lse);
    if (under < s && beam_score(bs, above(x, T()), lse) == s) {
        int i = K - 1;
        while (i >= 0 && candidate_value(list[i]) == x) --i;
        if (i >= 1 && beam_score(bs, candidate_value(list[i - 1]), lse) == s) return s;
    }
    return under;
}

// The L largest of n candidates, in order, to best[0 .. L); 0 where there are fewer.
__device__ __forceinline__ void rank_candidates(const unsigned long long* cand, int n, int L, unsigned long long* best) {
    for (int i = threadIdx.x; i < n; i += BT) {
        const unsigned long long c = cand[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) rank += cand[j] > c;
        if (rank < L) best[rank] = c;
    }
    for (int i = n + threadIdx.x; i < L; i += BT) best[i] = 0;
}

// One part of a row, chunk by chunk.  The first chunk gives a bound that at least L of its logits reach; from
// then on only logits above it are looked at one by one (later ones lose to equal ones), each warp with a list of
// its own, and the bound moves up to the L-th best after the second chunk, the fourth, the eighth and so on.
// So about L logits are looked at between two such steps (without them about L in every chunk: 38 us instead of 28
// for 512 rows of 131,072), and the other chunks need no barrier.  If a warp's list runs over, the L-th best of
// those kept is a better bound, and the part is searched again with it.  Where too many reach that as well (a row in
// rising order, or behind a masked stretch), the bound is found digit by digit, eight bits of a candidate at a time: ten
// more reads of the part at most, whatever the row (320 rising rows of 400,000 bf16 words 2.5 ms; with
// one bound after another from the lists 91).
//
// The sum is that of exp(x - t), t the first chunk's maximum; a thread that meets a logit 64 above moves its own t
// up.
template <typename T>
__global__ void __launch_bounds__(BT, CTAS_PER_SM) kda_beam_part_kernel(BeamParams p, int parts) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float warp_top[BW], warp_sum[BW], chunk_top, bound;
    __shared__ int found, kept[BW];
    __shared__ __align__(16) unsigned long long cand[CAP], all[CAP], best[KDA_BEAM_MAX_K + 1];
    float* thread_max = reinterpret_cast<float*>(all);   // until the lists are put together
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / (unsigned)parts;
    const int part = blockIdx.x % (unsigned)parts, L = p.K + 1;
    if (!live(p, row)) return;
    const int chunks = (p.V + CHUNK<T> - 1) / CHUNK<T>;
    const int first = (int)((int64_t)part * chunks / parts), last = (int)((int64_t)(part + 1) * chunks / parts);
    using X = Logits<T>;
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(ring_bytes) + warp * (STAGES * X::WARP_BYTES);
    const uintptr_t start = reinterpret_cast<uintptr_t>(static_cast<const T*>(p.logits) + row * p.row_stride);
    const int off = (int)(start % 16 / sizeof(T));
    const uint4* v = reinterpret_cast<const uint4*>(start - start % 16);

    float t = -INFINITY, limit = -INFINITY, sum = 0.f;   // limit: logits above it move t
    float least = -INFINITY;                             // logits from it on are looked at
    int mine_kept = 0;                                   // in this warp's list (more than WARP_CAP: some are lost)
    // All warps' lists as one, all[0 .. n); a barrier before and one inside.
    auto gather = [&](bool& lost) -> int {
        if (lane == 0) kept[warp] = mine_kept;
        __syncthreads();
        int before = 0, n = 0;
#pragma unroll
        for (int w = 0; w < BW; ++w) {
            const int c = kept[w];
            lost |= c > WARP_CAP;
            if (w < warp) before += min(c, WARP_CAP);
            n += min(c, WARP_CAP);
        }
        for (int i = lane; i < min(mine_kept, WARP_CAP); i += 32) all[before + i] = cand[warp * WARP_CAP + i];
        __syncthreads();
        return n;
    };
    int ahead = first, in = 0, out = 0;                  // the next chunk to copy, stages
    auto copy_next = [&]() {
        if (ahead < last) X::copy(ring + in * X::WARP_BYTES, v, ahead, off, p.V, tid);
        ++ahead;
        in = in + 1 == STAGES ? 0 : in + 1;
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < STAGES - 1; ++i) copy_next();
    // ---- the first chunk's maximum, and a bound that L of its logits reach ----
    {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(STAGES - 2) : "memory");
        __syncwarp();
        X x;
        x.take(ring, off, min(p.V - first * CHUNK<T>, CHUNK<T>), tid);
        const float mine = x.max();
        // 64 groups of threads, or 32: for an L of 16 at most they let about as few through.  A group's threads lie
        // 64 or 32 apart, so that a row of few words still has some in most groups.
        thread_max[tid] = mine;
        __syncthreads();
        if (warp == 0) {
            const bool few = p.K <= FEW;
            float g = -INFINITY, h = -INFINITY;     // of groups `lane` and `lane` + 32
#pragma unroll
            for (int i = 0; i < BW; ++i) {
                const float y = thread_max[i * 32 + lane];
                if (few || i % 2 == 0) g = fmaxf(g, y);
                else h = fmaxf(h, y);
            }
            int rank_g = 0, rank_h = 0;
            if (few) {
                thread_max[lane] = g;               // read above by this warp alone
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 y = *reinterpret_cast<const float4*>(thread_max + j);
                    rank_g += (y.x > g || (y.x == g && j < lane)) + (y.y > g || (y.y == g && j + 1 < lane)) +
                              (y.z > g || (y.z == g && j + 2 < lane)) + (y.w > g || (y.w == g && j + 3 < lane));
                }
                rank_h = L;
            } else {
#pragma unroll 8
                for (int j = 0; j < 32; ++j) {
                    const float y = __shfl_sync(0xFFFFFFFFu, g, j), z = __shfl_sync(0xFFFFFFFFu, h, j);
                    rank_g += (y > g || (y == g && j < lane)) + (z > g);
                    rank_h += (y >= h) + (z > h || (z == h && j < lane));
                }
            }
            if (rank_g == L - 1) bound = g;
            else if (rank_h == L - 1) bound = h;
            g = fmaxf(g, h);
#pragma unroll
            for (int o = 16; o; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xFFFFFFFFu, g, o));
            if (lane == 0) chunk_top = g;
        }
        __syncthreads();
        t = chunk_top;
        limit = t + 64.f;
        least = bound == -INFINITY ? above(bound, T()) : bound;
    }
    bool lost = false;
#pragma unroll 1
    for (int chunk = first; chunk < last; ++chunk) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(STAGES - 2) : "memory");
        __syncwarp();                                    // the warp's copies are there, its reads of the next stage over
        const uint32_t stage = ring + out * X::WARP_BYTES;
        out = out + 1 == STAGES ? 0 : out + 1;
        copy_next();
        X x;
        x.take(stage, off, min(p.V - chunk * CHUNK<T>, CHUNK<T>), tid);
        const float mine = x.max();
        const unsigned owners = __ballot_sync(0xFFFFFFFFu, mine >= least);
        if (owners) {
            // the few threads with such a logit: theirs are read again, a lane per element
            for (unsigned rest = owners; rest; rest &= rest - 1) {
                const int owner = __ffs(rest) - 1;
#pragma unroll
                for (int e = 0; e < X::NV * X::PER; e += 32) {
                    const int i = e + lane;
                    const int place = chunk * CHUNK<T> + (i / X::PER * BT + tid - lane + owner) * X::PER + i % X::PER;
                    const bool there = i < X::NV * X::PER && place < p.V;
                    const float y = there ? X::element(stage, off, owner, i) : -INFINITY;
                    const unsigned hits = __ballot_sync(0xFFFFFFFFu, there && y >= least);
                    const int at = mine_kept + __popc(hits & ((1u << lane) - 1));
                    if (hits >> lane & 1 && at < WARP_CAP) cand[warp * WARP_CAP + at] = candidate(y, (unsigned)place);
                    mine_kept += __popc(hits);
                }
            }
        }
        if (mine > limit) {                             // whatever the bound: behind masks it may be far above t
            if (sum != 0.f) sum *= exp_of(t - mine);
            t = mine;
            limit = mine + 64.f;
        }
        sum += x.sum_exp(t == -INFINITY ? 0.f : t);
        if (chunk == first && bound != -INFINITY) least = above(bound, T());
        const int done = chunk - first + 1;
        if (done >= 2 && (done & (done - 1)) == 0 && chunk + 1 < last) {
            const int n = gather(lost);                  // the L-th best of those kept is a bound even if some were lost
            if (n >= L) {
                rank_candidates(all, n, L, best);
                __syncthreads();
                if (tid < L) cand[tid] = best[tid];
                mine_kept = warp == 0 ? L : 0;
                least = fmaxf(least, above(candidate_value(best[L - 1]), T()));
            }
        }
    }
    int n = gather(lost);
    if (lost) {
        const T* logits = static_cast<const T*>(p.logits) + row * p.row_stride;
        const int stop = min(p.V, last * CHUNK<T>);
        // every candidate of the part, eight of a thread on their way at a time
        auto each = [&](auto use) {
            constexpr int BATCH = 8;
            for (int i0 = first * CHUNK<T> + tid; i0 < stop; i0 += BATCH * BT) {
                float y[BATCH];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) y[k] = i0 + k * BT < stop ? to_float(logits[i0 + k * BT]) : -INFINITY;
#pragma unroll
                for (int k = 0; k < BATCH; ++k)
                    if (y[k] > -INFINITY) use(candidate(y[k], (unsigned)(i0 + k * BT)));
            }
        };
        // those from `from` on to the list, the first CAP that come
        auto search = [&](unsigned long long from) {
            if (tid == 0) found = 0;
            __syncthreads();
            each([&](unsigned long long c) {
                if (c < from) return;
                const int at = atomicAdd(&found, 1);
                if (at < CAP) all[at] = c;
            });
            __syncthreads();
            n = found;
        };
        rank_candidates(all, n, L, best);
        __syncthreads();
        search(best[L - 1]);
        if (n > CAP) {
            // the L-th best of the part, its highest digits first, until CAP at most share them or are better
            unsigned long long from = 0;
            int over = 0;                                // better than all that share the digits found
            int* digits = reinterpret_cast<int*>(cand);  // how many have each
            static_assert(BT == 256 && sizeof(cand) >= 256 * sizeof(int), "a thread per digit");
            for (int shift = 56; n > CAP; shift -= 8) {
                digits[tid] = 0;
                __syncthreads();
                each([&](unsigned long long c) {
                    if (c >> shift >> 8 == from >> shift >> 8) atomicAdd(&digits[c >> shift & 255], 1);
                });
                __syncthreads();
                int better = over;
                for (int d = tid + 1; d < 256; ++d) better += digits[d];
                if (better < L && better + digits[tid] >= L) {           // in one thread
                    kept[0] = tid;
                    kept[1] = better;
                    kept[2] = better + digits[tid];
                }
                __syncthreads();
                from |= (unsigned long long)kept[0] << shift;
                over = kept[1];
                n = kept[2];                             // L in the end: no two candidates are equal
            }
            search(from);
        }
    }

    const Workspace<T> w = workspace<T>(p, parts);
    rank_candidates(all, n, L, w.list + (row * parts + part) * L);
    float top = t;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (lane == 0) warp_top[warp] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < BW; ++i) top = fmaxf(top, warp_top[i]);
    if (t != top) sum = sum == 0.f ? 0.f : sum * exp_of(t - top);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == 0) warp_sum[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < BW; ++i) sum += warp_sum[i];
        w.stats[row * parts + part] = make_float2(top, sum);
    }
}

template <typename T>
__global__ void __launch_bounds__(BT) kda_beam_join_kernel(BeamParams p, int parts) {
    constexpr int KEPT = 2048;                         // scored entries in shared memory; more of them in their place
    __shared__ float bs[KDA_BEAM_MAX_K], lse[KDA_BEAM_MAX_K], warp_left[BW];
    __shared__ unsigned char fin[KDA_BEAM_MAX_K], alive[KDA_BEAM_MAX_K];
    __shared__ unsigned long long kept[KEPT], best[KDA_BEAM_MAX_K], red[2][BW], group_max[GROUPS], cand[CAP], bound;
    __shared__ int found, counts[BW];
    const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = p.K, L = K + 1;
    const Workspace<T> w = workspace<T>(p, parts);
    const float2* stats = w.stats + (int64_t)n * K * parts;
    unsigned long long* list = w.list + (int64_t)n * K * parts * L;
    const int per_row = parts * L, entries = K * per_row;
    unsigned long long* scored = entries <= KEPT ? kept : list;
    if (tid == 0) found = 0;
    // the inputs are there since before the parts' kernel began
    float score = warp < K ? p.beam_scores[n * K + warp] : 0.f;
    bool done = warp < K && p.finished && p.finished[n * K + warp];
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // a warp per row: its lse, and its entries as scores with their places in the group
    unsigned long long mine = 0;
    float left_out = -INFINITY;                        // the best of what the parts' lists left out, or more
    for (int b = warp; b < K; b += BW) {
        const unsigned long long* from = list + b * per_row;
        unsigned long long* to = scored + b * per_row;
        constexpr int AHEAD = 4;                       // entries of a lane on their way (of a row that is not read: unused)
        unsigned long long c[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) c[i] = lane + 32 * i < per_row ? from[lane + 32 * i] : 0;
        const unsigned long long head = lane < parts ? from[lane * L] : 0, tail = lane < parts ? from[lane * L + K] : 0;
        const float2 stat = lane < parts ? stats[b * parts + lane] : make_float2(0.f, 0.f);
        bool is_alive = false;
        float log_sum = 0.f;
        if (!done && score == score && score != -INFINITY) {
            // the row's largest logit stands first in one of the lists
            float top = head ? candidate_value(head) : -INFINITY, sum = 0.f;
            for (int i = lane + 32; i < parts; i += 32)
                if (from[i * L]) top = fmaxf(top, candidate_value(from[i * L]));
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            if (lane < parts && stat.y != 0.f) sum = stat.y * exp_of(stat.x - top);
            for (int i = lane + 32; i < parts; i += 32) {
                const float2 s = stats[b * parts + i];
                if (s.y != 0.f) sum += s.y * exp_of(s.x - top);
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            is_alive = top != -INFINITY && sum == sum;               // else every score of the row is -inf
            log_sum = top + logf(sum);
            if (is_alive) {
                if (tail) left_out = fmaxf(left_out, best_left_out<T>(from + lane * L, K, tail, score, log_sum));
                for (int i = lane + 32; i < parts; i += 32) {
                    const unsigned long long last = from[i * L + K];
                    if (last) left_out = fmaxf(left_out, best_left_out<T>(from + i * L, K, last, score, log_sum));
                }
            }
            __syncwarp();                                            // scores may take the lists' place
            for (int e0 = lane; e0 < per_row; e0 += 32 * AHEAD) {
                unsigned long long after[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const int e = e0 + 32 * (AHEAD + i);
                    after[i] = e < per_row ? from[e] : 0;
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const int e = e0 + 32 * i;
                    unsigned long long d = 0;
                    if (is_alive && c[i]) {
                        const float x = candidate_value(c[i]), s = beam_score(score, x, log_sum);
                        if (s != -INFINITY) d = candidate(s, (unsigned)b * p.V + candidate_place(c[i]));
                    }
                    if (e < per_row) to[e] = d;
                    mine = d > mine ? d : mine;
                    c[i] = after[i];
                }
            }
        } else {
            for (int e = lane; e < per_row; e += 32) to[e] = 0;
            __syncwarp();
            if (lane == 0 && done && score == score && score != -INFINITY) {      // a finished beam's one word
                const unsigned long long d = candidate(score, (unsigned)b * p.V + (unsigned)p.eos);
                to[0] = d;
                mine = d > mine ? d : mine;
            }
        }
        if (lane == 0) {
            bs[b] = score;
            fin[b] = done;
            lse[b] = log_sum;
            alive[b] = is_alive;
        }
        if (b + BW < K) {
            score = p.beam_scores[n * K + b + BW];
            done = p.finished && p.finished[n * K + b + BW];
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) left_out = fmaxf(left_out, __shfl_xor_sync(0xFFFFFFFFu, left_out, o));
    if (lane == 0) warp_left[warp] = left_out;
    // as in a part: the K-th largest of the groups' maxima bounds the K-th score from below
    const bool few = K <= FEW;
    unsigned long long g = mine;
#pragma unroll
    for (int o = 1; o < 8; o *= 2) {
        if (o == 4 && !few) break;
        const unsigned long long other = __shfl_xor_sync(0xFFFFFFFFu, g, o);
        g = other > g ? other : g;
    }
    const int members = few ? 8 : 4, groups = BT / members;
    if (lane % members == 0) group_max[tid / members] = g;
    __syncthreads();
    if (tid < groups) {
        g = group_max[tid];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < groups; ++j) rank += group_max[j] > g || (group_max[j] == g && j < tid);
        if (rank == K - 1) bound = g;
    }
    __syncthreads();
    const unsigned long long least = bound;
#pragma unroll 4
    for (int e = tid; e < entries; e += BT) {
        const unsigned long long c = scored[e];
        if (c && c >= least) {
            const int at = atomicAdd(&found, 1);
            if (at < CAP) cand[at] = c;
        }
    }
    __syncthreads();
    int chosen = min(found, K);                        // continuations with a score
    if (found <= CAP) {
        for (int i = tid; i < found; i += BT) {
            const unsigned long long c = cand[i];
            int rank = 0;
            for (int j = 0; j < found; ++j) rank += cand[j] > c;
            if (rank < K) best[rank] = c;
        }
    } else {
        unsigned long long last = ~0ull;               // the best left, K times
        for (int k = 0; k < K; ++k) {
            unsigned long long c = 0;
            for (int e = tid; e < entries; e += BT) {
                const unsigned long long d = scored[e];
                if (d < last && d > c) c = d;
            }
            c = warp_max(c);
            if (lane == 0) red[k & 1][warp] = c;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < BW; ++i) c = red[k & 1][i] > c ? red[k & 1][i] : c;
            if (tid == 0) best[k] = c;
            last = c;
        }
    }
    __syncthreads();

    auto score_at = [&](int b, int v) -> float {
        if (fin[b]) return v == p.eos && bs[b] == bs[b] ? bs[b] : -INFINITY;
        if (!alive[b]) return -INFINITY;
        return beam_score(bs[b], to_float(static_cast<const T*>(p.logits)[((int64_t)n * K + b) * p.row_stride + v]), lse[b]);
    };
    if (chosen == K) {
        // could a logit that a part left out share the last score?
        const float worst = candidate_value(best[K - 1]);
        bool doubt = false;
#pragma unroll
        for (int i = 0; i < BW; ++i) doubt |= warp_left[i] >= worst;
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

// Parts of a row: so many that there are two CTAs per SM, as far as a row has chunks.  Each has its bound, its list and
// its joining on top of its chunks, so more of them pay only where the GPU would stay empty: 64 rows of 200,000 fp32
// words (16 groups of 4) take 17.7 us in 5 parts a row, 19.4 in 8 and 20.8 in 15.  The GPU's size is
// taken as 152 SMs, so that the workspace's size needs no device.
template <typename T>
int part_count(const int64_t rows, int V) {
    const int64_t chunks = (V + CHUNK<T> - 1) / CHUNK<T>, wanted = (2 * 152 + rows - 1) / rows;
    return (int)(wanted < chunks ? wanted : chunks);
}

template <typename T>
cudaError_t launch(const BeamParams& p, cudaStream_t s) {
    const int parts = part_count<T>((int64_t)p.N * p.K, p.V);
    constexpr int ring = BW * STAGES * Logits<T>::WARP_BYTES;
    static_assert(CTAS_PER_SM * (ring + 9728) <= 233472, "the rings, the kept logits and the system's 1 KB");
    static DeviceSetup done;
    int sms = 0;
    cudaError_t e = device_setup(done, reinterpret_cast<const void*>(kda_beam_part_kernel<T>), ring, &sms);
    if (e != cudaSuccess) return e;
    kda_beam_part_kernel<T><<<(unsigned)p.N * p.K * parts, BT, ring, s>>>(p, parts);
    e = cudaGetLastError();
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
    return cudaLaunchKernelEx(&cfg, kda_beam_join_kernel<T>, p, parts);
}

}  // namespace

size_t beam_workspace(int32_t N, int32_t K, int32_t V, kda_dtype dt) {
    const int64_t rows = (int64_t)N * K;
    const size_t parts = dt == KDA_DTYPE_BF16 ? part_count<__nv_bfloat16>(rows, V) : part_count<float>(rows, V);
    return (size_t)rows * parts * (sizeof(float2) + (K + 1) * sizeof(unsigned long long));
}

cudaError_t launch_beam_select(const BeamParams& p, kda_dtype dt, cudaStream_t s) {
    return dt == KDA_DTYPE_BF16 ? launch<__nv_bfloat16>(p, s) : launch<float>(p, s);
}

}  // namespace kda
