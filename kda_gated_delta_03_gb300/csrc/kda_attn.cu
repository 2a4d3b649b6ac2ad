// Attention of one new token per sequence over a paged key-value cache.
//
//   s_t = scale * q . k_t,   o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),   m = max_t s_t
//
// in one pass: the running maximum and sum of the softmax, the sum over the values rescaled whenever the
// maximum grows.  Exponents are taken in base 2 (scale * log2 e folded into the scores).  Every key and
// value is read once and meets the g = H_q / H_kv query heads that share it, 4 g flop for 2 elements.
//
// The visible tokens of all rows and heads are numbered tile after tile and cut into equal contiguous shares,
// one per CTA (two to four CTAs per SM), so that one long sequence, many short ones and anything between fill
// the GPU alike.  The shares are worked out on the device from seq_lens; the host never sees them (but it
// sees when every row must be short, and then a CTA does a unit whole).  Inside a CTA each warp takes every
// fourth sub-tile of TS tokens through its own ring of asynchronous copies (cp.async, no barrier with other
// warps) and keeps its own maximum, sum and accumulator; the four are joined in shared memory where a (row,
// head) unit ends.  A unit that a share's border cuts leaves partial results in the workspace, which a second
// kernel joins in the order of the CTAs: no atomics, the same bits on every call.
//
// What bounds it is DRAM, once there is enough to read: one row of 1,048,573 tokens with 8 heads of 128 takes
// 580 us (7.4 TB/s of reads), 64 rows of 213,000 tokens in all with 8 key-value heads 134 us (6.5 TB/s, the rest
// is the first loads' latency, the joins and the second kernel, together about 12 us whatever the size).  With few
// bytes that latency is all: 4.2 us for a row of 37 tokens whose table holds no more pages, 6.0 in a table of 1,024
// pages, where the shares are searched and the second kernel is launched all the same.  With more query heads a key
// the products begin to show: 32 rows of 8,192 tokens and two key-value heads (260 MB) take 47.9 us with 8 heads a key,
// 50.5 with 16 and 68.1 with 32 (3.8 TB/s); above 32 the cache is read once for each block of 32.
//
// The products: with the tokens as the 16 rows of mma.m16n8k16 and the query heads as its 8 columns, both
// products take the cache as the A operand straight from shared memory (K by ldmatrix, V by ldmatrix.trans)
// and leave no padding at 8 heads.  tcgen05 could take 128 tokens as its rows and the heads as its columns just as
// well, with the scores and weights on a round trip through tensor memory.  There is little to gain up to 16 heads a key
// (the tensor pipe is busy for 14 % of the time at 4 heads, 25 % at 16, and the kernel waits for loads); at 32 and more
// (36 %, with the second product done twice for the weights' two halves) it would be the way on, and is not built.  fp32
// caches take the same path with FFMA (two products in one instruction), since TF32's 11 bits would not keep fp32's
// precision; at 4 heads a key they are read at 6.5 TB/s, 16 heads a key on one key-value head run at 2.0.

#include <cmath>
#include <type_traits>

#include "kda_serve.cuh"

namespace kda {
namespace {

constexpr int NW = 4;                         // warps of a CTA
constexpr int AT = NW * 32;
constexpr int MAX_CTAS = 640;                 // of the main kernel, whatever the GPU (bounds the workspace)
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 16 bytes from global to shared memory; zeros, and no read, where `read` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two fp32 products and sums in one instruction.
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n.reg .b64 a, b, d;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 d, {%0, %1};\n"
        "fma.rn.f32x2 d, a, b, d;\nmov.b64 {%0, %1}, d;\n}\n"
        : "+f"(d0), "+f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// ---- which tokens a row's tiles hold ----
struct Row {
    int len;
    int tiles;                   // tiles with a visible token
    int lead;                    // the first `lead` of them start at token 0,
    int skip;                    // the others at tile lead + skip (between sinks and window)
    int from;                    // first token of the window
    int solid;                   // tokens below it come from the cache (the new one does not)
};

template <int TILE>
__device__ __forceinline__ Row row_of(const AttnParams& p, int len) {
    Row r;
    r.len = len < 0 || len > p.max_pages * p.page_size ? 0 : len;
    const int all = (r.len + TILE - 1) / TILE;
    r.from = p.window > 0 && r.len > p.window ? r.len - p.window : 0;
    r.lead = r.skip = 0;
    r.tiles = all;
    r.solid = p.k_new ? r.len - 1 : r.len;
    const int sink_tiles = (min(p.sinks, r.from) + TILE - 1) / TILE, first = r.from / TILE;
    if (first > sink_tiles) {
        r.lead = sink_tiles;
        r.skip = first - sink_tiles;
        r.tiles = all - r.skip;
    }
    return r;
}

// A place in the CTA's share: tile `tile` of key-value head kvh and head block hb of row b.
struct Place {
    int b, kvh, hb, tile;
    Row row;
};

template <typename T, int D, int NH>
struct Core;

// bf16: tokens are the rows and heads the columns of the tensor core's tile.
template <int D, int NH>
struct Core<__nv_bfloat16, D, NH> {
    static constexpr int MT = D == 128 ? 1 : D == 64 ? 2 : 4;        // blocks of 16 tokens that share a maximum's update
    static constexpr int TS = 16 * MT;                  // tokens of a warp's sub-tile
    static constexpr int CPR = D / 8;                   // 16-byte chunks of a token
    static constexpr int NT = NH / 8, KT = D / 16;
    static constexpr int SLOTS = 2 * NT;                // heads that a lane has columns of
    static constexpr int ACC = NT * KT * 4;
    static constexpr int QP = D * 2 + 16;               // bytes from head to head of q (conflict-free fragments)
    static constexpr int P_BYTES = 0;

    static constexpr bool Q_KEPT = NT == 1;             // q's fragments in registers; else fetched each time
    uint32_t qf[Q_KEPT ? KT : 1][2];
    uint32_t qa;
    float acc[ACC], m[SLOTS], l[SLOTS];

    __device__ static int swizzle(int row, int chunk) { return D >= 64 ? chunk ^ (row & 7) : chunk; }
    __device__ static int head_of_slot(int s, int lane) { return (s >> 1) * 8 + 2 * (lane & 3) + (s & 1); }
    __device__ static int slot_of(int i) { return i / (KT * 4) * 2 + (i & 1); }
    __device__ static int dim_of(int i, int lane) { return (i / 4 % KT) * 16 + (lane >> 2) + 8 * ((i >> 1) & 1); }
    __device__ static bool owns_output(int) { return true; }
    __device__ static bool writes_stats(int lane) { return lane < 4; }

    __device__ void begin(const unsigned char* q, int lane) {
        // as the B operand: heads 0-7, columns 0-7 and 8-15, then heads 8-15
        qa = smem_addr(q) + ((lane >> 4) * 8 + (lane & 7)) * QP + ((lane >> 3) & 1) * 16;
        if constexpr (Q_KEPT) {
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    qf[k][h] = *reinterpret_cast<const uint32_t*>(q + (lane >> 2) * QP + (k * 16 + 2 * (lane & 3) + 8 * h) * 2);
        }
#pragma unroll
        for (int i = 0; i < ACC; ++i) acc[i] = 0.f;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            m[s] = -INFINITY;
            l[s] = 0.f;
        }
    }

    // One sub-tile; sees(t): token t of it is visible (a token that is not lies in shared memory as zeros), `all`: every
    // one is.  Rows of shared memory: chunk c of row r at c ^ (r & 7), so that a fragment's address is one XOR away
    // from the lane's own (the sub-tiles start on 2 KB boundaries).
    template <typename Sees>
    __device__ void step(uint32_t ks, uint32_t vs, bool all, Sees sees, float scale2, unsigned char*, int lane) {
        constexpr int SW = D >= 64 ? 7 : 0;
        const int i8 = lane >> 3, r8 = lane & 7;
        float s[MT][NT][4];
        const uint32_t ka = ks + ((i8 & 1) * 8 + r8) * (D * 2) + (((i8 >> 1) ^ (r8 & SW)) << 4);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float s1[NT][4];                            // two chains of products
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mt][n][e] = s1[n][e] = 0.f;
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                uint32_t a[4];
                ldsm4((ka ^ (k << 5)) + mt * (16 * D * 2), a);
                if constexpr (Q_KEPT) {
                    mma_bf16(k & 1 ? s1[0] : s[mt][0], a, qf[k][0], qf[k][1]);
                } else {
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t b[4];
                        ldsm4(qa + n * 8 * QP + k * 32, b);
                        mma_bf16(k & 1 ? s1[n] : s[mt][n], a, b[0], b[1]);
                        mma_bf16(k & 1 ? s1[n + 1] : s[mt][n + 1], a, b[2], b[3]);
                    }
                }
            }
            if (KT > 1) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[mt][n][e] += s1[n][e];
            }
            if (!all) {
                const bool lo = sees(mt * 16 + (lane >> 2)), hi = sees(mt * 16 + (lane >> 2) + 8);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!(e < 2 ? lo : hi)) s[mt][n][e] = -INFINITY;
            }
        }
        float base[SLOTS];
        bool grown = false;
#pragma unroll
        for (int c = 0; c < SLOTS; ++c) {
            float x = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) x = fmaxf(x, fmaxf(s[mt][c / 2][c & 1], s[mt][c / 2][(c & 1) + 2]));
#pragma unroll
            for (int o = 4; o < 32; o *= 2) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
            x = fmaxf(m[c], x * scale2);
            grown |= x != m[c];
            base[c] = x;
        }
        if (__any_sync(0xFFFFFFFFu, grown)) {           // the maximum of some head: rescale to it
            float keep[SLOTS];
#pragma unroll
            for (int c = 0; c < SLOTS; ++c) {
                keep[c] = exp2_approx(m[c] - (base[c] == -INFINITY ? 0.f : base[c]));
                m[c] = base[c];
                l[c] *= keep[c];
            }
#pragma unroll
            for (int i = 0; i < ACC; ++i) acc[i] *= keep[slot_of(i)];
        }
        // The weights go to the tensor core as bf16 pairs hi + lo (16 bits together): rounded to bf16 alone
        // they would add 1.1e-3 of relative error to an output that is itself rounded to 1.7e-3.
        const uint32_t va = vs + ((i8 >> 1) * 8 + r8) * (D * 2) + (((i8 & 1) ^ (r8 & SW)) << 4);
#pragma unroll
        for (int c = 0; c < SLOTS; ++c) base[c] = base[c] == -INFINITY ? 0.f : base[c];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float x = exp2_approx(fmaf(s[mt][n][2 * h], scale2, -base[2 * n]));
                    const float y = exp2_approx(fmaf(s[mt][n][2 * h + 1], scale2, -base[2 * n + 1]));
                    l[2 * n] += x;
                    l[2 * n + 1] += y;
                    const uint32_t hi = pack_bf16(x, y);
                    const uint32_t lo = pack_bf16(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xFFFF0000u));
                    ph[n][h] = transpose8x8(hi);
                    pl[n][h] = transpose8x8(lo);
                }
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                uint32_t a[4];
                ldsm4_trans((va ^ (k << 5)) + mt * (16 * D * 2), a);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float(&o)[4] = *reinterpret_cast<float(*)[4]>(&acc[(n * KT + k) * 4]);
                    mma_bf16(o, a, ph[n][0], ph[n][1]);
                    mma_bf16(o, a, pl[n][0], pl[n][1]);
                }
            }
        }
    }

    __device__ void sum_lanes() {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
#pragma unroll
            for (int o = 4; o < 32; o *= 2) l[s] += __shfl_xor_sync(0xFFFFFFFFu, l[s], o);
    }
};

// fp32: four lanes per token for the scores, then D / 32 output columns per lane.
template <int D, int NH>
struct Core<float, D, NH> {
    static constexpr int MT = D == 128 ? 1 : D == 64 ? 2 : 4;        // tokens of a lane
    static constexpr int TS = 8 * MT;
    static constexpr int CPR = D / 4;
    static constexpr int E = D >= 32 ? D / 32 : 1;      // columns of a lane (d = 16: lanes 16-31 repeat 0-15)
    static constexpr int SLOTS = NH;
    static constexpr int ACC = NH * E;
    static constexpr int QP = D * 4;
    static constexpr int P_BYTES = TS * NH * 4;         // the weights, from the token's lanes to all of them

    const unsigned char* q;
    float acc[ACC], m[SLOTS], l[SLOTS];

    __device__ static int swizzle(int row, int chunk) { return D >= 64 ? chunk ^ ((row & 1) << 2) : chunk; }
    __device__ static int head_of_slot(int s, int) { return s; }
    __device__ static int slot_of(int i) { return i / E; }
    __device__ static int dim_of(int i, int lane) { return (lane * E + i % E) % D; }
    __device__ static bool owns_output(int lane) { return lane * E < D; }
    __device__ static bool writes_stats(int lane) { return lane == 0; }

    __device__ void begin(const unsigned char* qbuf, int) {
        q = qbuf;
#pragma unroll
        for (int i = 0; i < ACC; ++i) acc[i] = 0.f;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            m[s] = -INFINITY;
            l[s] = 0.f;
        }
    }

    template <typename Sees>
    __device__ void step(uint32_t ks, uint32_t vs, bool all, Sees sees, float scale2, unsigned char* pbuf, int lane) {
        const int r = lane >> 2, c = lane & 3;          // tokens r, r + 8, ...
        float s[MT][NH], s1[MT][NH];                    // even and odd columns
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < NH; ++h) s[mt][h] = s1[mt][h] = 0.f;
#pragma unroll
        for (int j = 0; j < CPR / 4; ++j) {
            const int chunk = c + 4 * j;
            float4 k[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(k[mt].x), "=f"(k[mt].y), "=f"(k[mt].z), "=f"(k[mt].w)
                             : "r"(ks + (r + 8 * mt) * (D * 4) + swizzle(r, chunk) * 16) : "memory");
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const float4 x = *reinterpret_cast<const float4*>(q + h * QP + chunk * 16);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    fma2(s[mt][h], s1[mt][h], x.x, x.y, k[mt].x, k[mt].y);
                    fma2(s[mt][h], s1[mt][h], x.z, x.w, k[mt].z, k[mt].w);
                }
            }
        }
        float* pw = reinterpret_cast<float*>(pbuf);
        bool grown = false, seen[MT];
        float base[NH];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) seen[mt] = all || sees(r + 8 * mt);
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            float x = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                s[mt][h] += s1[mt][h];
                s[mt][h] += __shfl_xor_sync(0xFFFFFFFFu, s[mt][h], 1);
                s[mt][h] += __shfl_xor_sync(0xFFFFFFFFu, s[mt][h], 2);
                if (!seen[mt]) s[mt][h] = -INFINITY;
                x = fmaxf(x, s[mt][h]);
            }
#pragma unroll
            for (int o = 4; o < 32; o *= 2) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
            base[h] = fmaxf(m[h], x * scale2);
            grown |= base[h] != m[h];
        }
        if (__any_sync(0xFFFFFFFFu, grown)) {           // the maximum of some head: rescale to it
            float keep[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                keep[h] = exp2_approx(m[h] - (base[h] == -INFINITY ? 0.f : base[h]));
                m[h] = base[h];
                l[h] *= keep[h];
            }
#pragma unroll
            for (int i = 0; i < ACC; ++i) acc[i] *= keep[slot_of(i)];
        }
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            const float from = base[h] == -INFINITY ? 0.f : base[h];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const float x = exp2_approx(fmaf(s[mt][h], scale2, -from));
                l[h] += x;
                if ((h & 3) == c) pw[(r + 8 * mt) * NH + h] = x;
            }
        }
        __syncwarp();
#pragma unroll
        for (int t = 0; t < TS; ++t) {
            float v[E], w[NH];
            const int d0 = (lane * E) % D;
            const uint32_t at = vs + t * (D * 4) + swizzle(t, d0 / 4) * 16 + (d0 & 3) * 4;
            if constexpr (E == 4)
                asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                             : "r"(at) : "memory");
            else if constexpr (E == 2)
                asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(at) : "memory");
            else
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[0]) : "r"(at) : "memory");
            if constexpr (NH % 4 == 0) {
#pragma unroll
                for (int h = 0; h < NH; h += 4)
                    *reinterpret_cast<float4*>(w + h) = *reinterpret_cast<const float4*>(pw + t * NH + h);
            } else {
#pragma unroll
                for (int h = 0; h < NH; ++h) w[h] = pw[t * NH + h];
            }
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                if constexpr (E == 1) {
                    acc[h] += w[h] * v[0];
                } else {
#pragma unroll
                    for (int e = 0; e < E; e += 2) fma2(acc[h * E + e], acc[h * E + e + 1], w[h], w[h], v[e], v[e + 1]);
                }
            }
        }
        __syncwarp();
    }

    __device__ void sum_lanes() {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
#pragma unroll
            for (int o = 4; o < 32; o *= 2) l[s] += __shfl_xor_sync(0xFFFFFFFFu, l[s], o);
    }
};

__host__ __device__ constexpr int piece_floats(int heads, int d) { return (heads * (d + 2) + 3) / 4 * 4; }

template <typename T, int D, int NH>
struct Layout {
    using C = Core<T, D, NH>;
    static constexpr int TILE = NW * C::TS;
    static constexpr int SUB = C::TS * D * (int)sizeof(T);        // bytes of a sub-tile's keys
    static constexpr int CTAS_PER_SM = NH == 32 || (NH == 16 && sizeof(T) == 4) ? 2 : NH == 16 || D > 16 ? 3 : 4;
    static constexpr int STAGES = D > 16 && CTAS_PER_SM == 2 ? 3 : 2;
    static constexpr int RING = STAGES * 2 * SUB;                 // of one warp
    static constexpr int Q = NW * RING;
    static constexpr int Q_BYTES = NH * C::QP;
    static constexpr int MERGE = Q + Q_BYTES;                     // part of the warps' accumulators
    static constexpr int MERGE_REGS = C::ACC < 8 ? C::ACC : D == 128 && NH == 8 && sizeof(T) == 2 ? 16 : 8;
    static constexpr int STATS = MERGE + NW * MERGE_REGS * 32 * 4;   // m, l [NW][NH], then multipliers [NW][NH], m, 1 / l [NH]
    static constexpr int PW = STATS + (3 * NW + 2) * NH * 4;
    static constexpr int MISC = PW + NW * C::P_BYTES;
    static constexpr int BYTES = MISC + 32;
    static_assert(CTAS_PER_SM * (BYTES + 1024) <= 233472, "shared memory of the CTAs of an SM");
    // workspace: a record per CTA, then its two partial results of o[NH][D], m[NH], l[NH]
    static constexpr int PIECE = piece_floats(NH, D);
};

// Partial results of a unit that starts in one CTA's share and goes on in others'.  Records lie at the unit's
// place where the units are no more than the CTAs, else at its first CTA's (which has one at most).
struct Record {
    int b, unit;                 // -1: none
    int first, last;             // the CTAs with its pieces
    int slot;                    // of the first piece; the others lie in slot 0
    int pad[3];
};

template <typename T, int D, int NH>
__global__ void __launch_bounds__(AT, Layout<T, D, NH>::CTAS_PER_SM) kda_attn_kernel(AttnParams p, int head_blocks, int grid) {
    using C = Core<T, D, NH>;
    using L = Layout<T, D, NH>;
    constexpr int TS = C::TS, TILE = L::TILE, CPR = C::CPR;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    const int group = p.Hq / p.Hkv, units = p.Hkv * head_blocks;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- this CTA's share ----
    int* misc = reinterpret_cast<int*>(sm + L::MISC);
    int64_t* split = reinterpret_cast<int64_t*>(sm + L::MISC + 16);
    int64_t* sums = reinterpret_cast<int64_t*>(sm + L::MERGE);
    // tiles of the rows b0 .. b0 + AT - 1: this thread's row's, those before it, and in all
    auto scan_rows = [&](int b0, int& mine, int64_t& before, int64_t& all) {
        mine = b0 + tid < p.B ? row_of<TILE>(p, __ldg(p.lens + b0 + tid)).tiles : 0;
        int64_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) sums[warp] = inc;
        __syncthreads();
        before = inc - mine;
        all = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) before += sums[w];
            all += sums[w];
        }
    };
    int left = 0;                                       // tiles of this CTA's share
    Place at{};
    if (p.whole) {                                      // one unit, uncut
        at.b = cta / units;
        at.kvh = (cta - at.b * units) / head_blocks;
        at.hb = cta % head_blocks;
        at.row = row_of<TILE>(p, __ldg(p.lens + at.b));
        left = at.row.tiles;
    } else {
        int mine;
        int64_t before, total;                              // of the first AT rows, then of all
        scan_rows(0, mine, before, total);
        for (int b0 = AT; b0 < p.B; b0 += AT) {
            int m;
            int64_t unused, all;
            __syncthreads();
            scan_rows(b0, m, unused, all);
            total += all;
        }
        // no more shares than tiles: none of them is empty, so a unit's pieces lie in consecutive CTAs
        const int64_t flat = total * units, shares = flat < grid ? flat : grid;
        const int64_t begin = cta < shares ? cta * flat / shares : flat;
        const int64_t end = cta < shares ? (cta + 1) * flat / shares : flat;
        left = (int)(end - begin);
        if (tid == 0) {                                 // for its records, later
            split[0] = flat;
            split[1] = end;
            misc[3] = (int)shares;
        }
        if (left > 0) {
            int64_t base = 0;                               // tiles of the rows before b0
            for (int b0 = 0; b0 < p.B; b0 += AT) {
                int64_t all = total;
                if (p.B > AT) {
                    __syncthreads();
                    scan_rows(b0, mine, before, all);
                }
                const int64_t lo = (base + before) * units, hi = lo + (int64_t)mine * units;
                if (mine > 0 && begin >= lo && begin < hi) {
                    const int64_t in = begin - lo;
                    misc[0] = b0 + tid;
                    misc[1] = (int)(in / mine);
                    misc[2] = (int)(in % mine);
                }
                base += all;
                if (begin < base * units) break;
            }
            __syncthreads();
            at.b = misc[0];
            at.kvh = misc[1] / head_blocks;
            at.hb = misc[1] - at.kvh * head_blocks;
            at.tile = misc[2];
            at.row = row_of<TILE>(p, __ldg(p.lens + at.b));
        }
    }

    auto next_unit = [&](Place& x) {                    // only called while the share goes on
        x.tile = 0;
        if (++x.hb < head_blocks) return;
        x.hb = 0;
        if (++x.kvh < p.Hkv) return;
        x.kvh = 0;
        while (x.b + 1 < p.B) {
            x.row = row_of<TILE>(p, __ldg(p.lens + ++x.b));
            if (x.row.tiles > 0) break;
        }
    };
    // this warp's sub-tile of a tile: its first token
    auto sub_tile = [&](const Row& row, int tile) -> int {
        return (tile + (tile < row.lead ? 0 : row.skip)) * TILE + warp * TS;
    };
    auto any_seen = [&](const Row& row, int first) {
        return first < row.len && (first + TS > row.from || first < p.sinks);
    };
    auto all_seen = [&](const Row& row, int first) { return first >= row.from && first + TS <= row.len; };
    auto is_seen = [&](const Row& row, int t) { return t < row.len && (t >= row.from || t < p.sinks); };
    const T* kp = static_cast<const T*>(p.k_pages);
    const T* vp = static_cast<const T*>(p.v_pages);
    const uint32_t ring = smem_addr(sm) + warp * L::RING;
    auto page_of = [&](int t) -> int { return p.page_magic ? (int)(__umulhi(t, p.page_magic) >> p.page_shift) : t; };
    auto checked = [&](int page) -> int {
        if ((unsigned)page < (unsigned)p.num_pages) return page;
        atomicOr(p.err, KDA_DEVERR_PAGES);
        return 0;
    };

    // ---- copies of this warp's next visible sub-tile into the ring ----
    Place ahead = at;
    int ahead_left = left, stage_in = 0;
    constexpr int RUN = TS / C::MT;                     // tokens copied as one run of memory,
    const bool whole_runs = p.page_size % RUN == 0;     // which then never crosses a page
    auto issue = [&]() {
        int first = 0;
        while (ahead_left > 0) {
            first = sub_tile(ahead.row, ahead.tile);
            if (any_seen(ahead.row, first)) break;
            if (--ahead_left > 0 && ++ahead.tile == ahead.row.tiles) next_unit(ahead);
        }
        if (ahead_left > 0) {
            const uint32_t dst = ring + stage_in * (2 * L::SUB);
            stage_in = stage_in + 1 == L::STAGES ? 0 : stage_in + 1;
            const int32_t* table = p.table + (int64_t)ahead.b * p.max_pages;
            if (whole_runs && first >= ahead.row.from && first + TS <= ahead.row.solid) {
                int page[C::MT];
#pragma unroll
                for (int m = 0; m < C::MT; ++m) page[m] = __ldg(table + page_of(first + m * RUN));
#pragma unroll
                for (int m = 0; m < C::MT; ++m) {
                    const int t = first + m * RUN, in_page = t - page_of(t) * p.page_size, pg = checked(page[m]);
                    const int64_t off = ((int64_t)ahead.kvh * p.page_size + in_page) * D;
                    const char* k = reinterpret_cast<const char*>(kp + pg * p.k_stride + off) + lane * 16;
                    const char* v = reinterpret_cast<const char*>(vp + pg * p.v_stride + off) + lane * 16;
#pragma unroll
                    for (int i = 0; i < (RUN * CPR + 31) / 32; ++i) {
                        const int id = lane + 32 * i, r = m * RUN + id / CPR, c = id % CPR;
                        const uint32_t to = dst + r * (CPR * 16) + C::swizzle(r, c) * 16;
                        if (RUN * CPR % 32 == 0 || id < RUN * CPR) {
                            copy16(to, k + i * 512, true);
                            copy16(to + L::SUB, v + i * 512, true);
                        }
                    }
                }
            } else {
                // each lane with its token's own place: several lanes a token, or several tokens a lane
                constexpr int LPT = TS < 32 ? 32 / TS : 1, TPL = TS < 32 ? 1 : TS / 32;
#pragma unroll
                for (int j = 0; j < TPL; ++j) {
                    const int r = lane / LPT + 32 * j, t = first + r;
                    const bool read = is_seen(ahead.row, t);
                    const T* k = kp;
                    const T* v = vp;
                    if (read && t >= ahead.row.solid) {
                        const int64_t off = ((int64_t)ahead.b * p.Hkv + ahead.kvh) * D;
                        k = static_cast<const T*>(p.k_new) + off;
                        v = static_cast<const T*>(p.v_new) + off;
                    } else if (read) {
                        const int slot = page_of(t), page = checked(__ldg(table + slot));
                        const int64_t off = ((int64_t)ahead.kvh * p.page_size + t - slot * p.page_size) * D;
                        k += page * p.k_stride + off;
                        v += page * p.v_stride + off;
                    }
#pragma unroll
                    for (int i = 0; i < CPR / LPT; ++i) {
                        const int c = i * LPT + lane % LPT;
                        const uint32_t to = dst + r * (CPR * 16) + C::swizzle(r, c) * 16;
                        copy16(to, reinterpret_cast<const char*>(k) + c * 16, read);
                        copy16(to + L::SUB, reinterpret_cast<const char*>(v) + c * 16, read);
                    }
                }
            }
            if (--ahead_left > 0 && ++ahead.tile == ahead.row.tiles) next_unit(ahead);
        }
        copy_commit();
    };
#pragma unroll 1
    for (int i = 0; i < L::STAGES - 1; ++i) issue();

    // ---- q of a unit: fetched to registers while the unit before it runs, then to shared memory ----
    constexpr int QV = NH * D * (int)sizeof(T) / 16, QPT = (QV + AT - 1) / AT, QC = D * (int)sizeof(T) / 16;
    uint4 qnext[QPT];
    const uint32_t flip = p.scale < 0.f ? (sizeof(T) == 2 ? 0x80008000u : 0x80000000u) : 0u;   // q carries the scale's sign
    auto fetch_q = [&](int b, int kvh, int hb) {
        const int h0 = hb * NH;
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            const int id = tid + i * AT, h = id / QC, c = id % QC;
            qnext[i] = make_uint4(0, 0, 0, 0);
            if (id < QV && h0 + h < group)
                qnext[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) +
                                                                ((int64_t)b * p.Hq + kvh * group + h0 + h) * D) + c);
        }
    };
    auto store_q = [&]() {
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            const int id = tid + i * AT, h = id / QC, c = id % QC;
            const uint4 x = qnext[i];
            if (id < QV)
                *reinterpret_cast<uint4*>(sm + L::Q + h * C::QP + c * 16) =
                    make_uint4(x.x ^ flip, x.y ^ flip, x.z ^ flip, x.w ^ flip);
        }
    };

    Record* records = reinterpret_cast<Record*>(p.workspace);
    const bool by_unit = !p.whole && (int64_t)p.B * units <= grid;
    float* pieces = reinterpret_cast<float*>(p.workspace + MAX_CTAS * sizeof(Record)) + (int64_t)cta * 2 * L::PIECE;
    float* sm_m = reinterpret_cast<float*>(sm + L::STATS);
    float* sm_l = sm_m + NW * NH;
    float* sm_mult = sm_l + NW * NH;
    float* sm_inv = sm_mult + NW * NH;
    float* merge = reinterpret_cast<float*>(sm + L::MERGE);
    const float scale2 = fmaxf(fabsf(p.scale) * LOG2E, 1e-38f);      // above 0: a masked score stays at -inf
    bool first_unit = true, recorded = false;
    int stage = 0;
    if (left > 0) {
        fetch_q(at.b, at.kvh, at.hb);
        store_q();
        __syncthreads();
    }
    C core;
    while (left > 0) {
        // ---- one unit, or this share's part of it ----
        const int b = at.b, t0 = at.tile, count = min(left, at.row.tiles - t0);
        const bool starts = t0 == 0, ends = t0 + count == at.row.tiles;
        const Row row = at.row;
        core.begin(sm + L::Q, lane);
        Place after = at;
        if (left > count) {
            next_unit(after);
            fetch_q(after.b, after.kvh, after.hb);
        }
        for (int tile = t0; tile < t0 + count; ++tile) {
            const int first = sub_tile(row, tile);
            if (!any_seen(row, first)) continue;
            copy_wait<L::STAGES - 2>();
            __syncwarp();
            issue();
            const uint32_t ks = ring + stage * (2 * L::SUB), vs = ks + L::SUB;
            core.step(ks, vs, all_seen(row, first), [&](int t) { return is_seen(row, first + t); }, scale2,
                      sm + L::PW + warp * C::P_BYTES, lane);
            if (first + TS > row.solid && p.k_new && at.hb == 0 && row.solid >= first) {
                // the new token's key and value into the cache, from the copy in shared memory
                const int t = row.solid, r = t - first, slot = page_of(t);
                const int page = __ldg(p.table + (int64_t)b * p.max_pages + slot);
                if (page >= 0 && page < p.num_pages) {
                    const int64_t off = ((int64_t)at.kvh * p.page_size + (t - slot * p.page_size)) * D;
                    for (int c = lane; c < 2 * CPR; c += 32) {
                        const bool is_k = c < CPR;
                        const int chunk = is_k ? c : c - CPR;
                        uint4 x;
                        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                                     : "r"((is_k ? ks : vs) + r * (CPR * 16) + C::swizzle(r, chunk) * 16) : "memory");
                        T* to = is_k ? static_cast<T*>(p.k_pages) + page * p.k_stride
                                     : static_cast<T*>(p.v_pages) + page * p.v_stride;
                        reinterpret_cast<uint4*>(to + off)[chunk] = x;
                    }
                } else if (lane == 0) {
                    atomicOr(p.err, KDA_DEVERR_PAGES);  // nobody may have read that page: not stored, and told
                }
            }
            stage = stage + 1 == L::STAGES ? 0 : stage + 1;
        }

        // ---- join the warps: their accumulators through shared memory, a few registers at a time ----
        core.sum_lanes();
        if (C::writes_stats(lane)) {
#pragma unroll
            for (int i = 0; i < C::SLOTS; ++i) {
                sm_m[warp * NH + C::head_of_slot(i, lane)] = core.m[i];
                sm_l[warp * NH + C::head_of_slot(i, lane)] = core.l[i];
            }
        }
        const int kvh = at.kvh, h0 = at.hb * NH;
        const bool complete = starts && ends;
        float* piece = pieces + (first_unit ? 0 : L::PIECE);
#pragma unroll
        for (int r0 = 0; r0 < C::ACC; r0 += L::MERGE_REGS) {
#pragma unroll
            for (int i = 0; i < L::MERGE_REGS; ++i)
                if (r0 + i < C::ACC) merge[(warp * L::MERGE_REGS + i) * 32 + lane] = core.acc[r0 + i];
            __syncthreads();
            if (r0 == 0) {
                if (left > count) store_q();            // every warp is done with this unit's
                if (tid < NH) {
                    float top = -INFINITY, sum = 0.f;
#pragma unroll
                    for (int w = 0; w < NW; ++w) top = fmaxf(top, sm_m[w * NH + tid]);
                    const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        const float x = exp2_approx(sm_m[w * NH + tid] - base);
                        sm_mult[w * NH + tid] = x;
                        sum += sm_l[w * NH + tid] * x;
                    }
                    sm_inv[tid] = sum == 0.f ? 0.f : 1.f / sum;
                    if (!complete) {
                        piece[NH * D + tid] = top;
                        piece[NH * D + NH + tid] = sum;
                    } else if (p.lse && h0 + tid < group) {
                        p.lse[(int64_t)b * p.Hq + kvh * group + h0 + tid] =
                            sum == 0.f ? -INFINITY : (top + log2f(sum)) * LN2;
                    }
                }
                __syncthreads();
            }
#pragma unroll
            for (int k = 0; k < (L::MERGE_REGS + NW - 1) / NW; ++k) {
                const int j = warp + NW * k, i = r0 + j;                 // register i of every warp
                if (j >= L::MERGE_REGS || i >= C::ACC) break;
                const int h = C::head_of_slot(C::slot_of(i), lane), d = C::dim_of(i, lane);
                float o = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) o += merge[(w * L::MERGE_REGS + j) * 32 + lane] * sm_mult[w * NH + h];
                if (!C::owns_output(lane)) continue;
                if (!complete)
                    piece[h * D + d] = o;
                else if (h0 + h < group)
                    store_from_float(static_cast<T*>(p.o), ((int64_t)b * p.Hq + kvh * group + h0 + h) * D + d, o * sm_inv[h]);
            }
            __syncthreads();
        }
        if (tid == 0 && starts) {
            const int unit = kvh * head_blocks + at.hb;
            if (!ends) {
                const int64_t x = split[1] - left + row.tiles;          // flat tiles up to the unit's last
                records[by_unit ? b * units + unit : cta] =
                    Record{b, unit, cta, (int)((x * misc[3] - 1) / split[0]), first_unit ? 0 : 1, {0, 0, 0}};
                recorded = true;
            } else if (by_unit) {
                records[b * units + unit].b = -1;
            }
        }
        left -= count;
        first_unit = false;
        if (left > 0) at = after;
    }
    if (tid == 0 && !recorded && !by_unit && !p.whole) records[cta].b = -1;
    // rows without a visible token
    for (int b = cta; b < p.B; b += grid) {
        const int len = p.lens[b];
        if (tid == 0 && (len < 0 || len > p.max_pages * p.page_size)) atomicOr(p.err, KDA_DEVERR_PAGES);
        if (row_of<TILE>(p, len).tiles) continue;
        if (by_unit)
            for (int u = tid; u < units; u += AT) records[b * units + u].b = -1;
        T* o = static_cast<T*>(p.o) + (int64_t)b * p.Hq * D;
        for (int i = tid; i < p.Hq * D; i += AT) store_from_float(o, i, 0.f);
        if (p.lse)
            for (int h = tid; h < p.Hq; h += AT) p.lse[(int64_t)b * p.Hq + h] = -INFINITY;
    }
}

// Joins the pieces of a unit, one CTA per record and head.
template <typename T, int D, int NH>
__global__ void __launch_bounds__(AT) kda_attn_join_kernel(AttnParams p, int head_blocks) {
    using L = Layout<T, D, NH>;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Record r = reinterpret_cast<const Record*>(p.workspace)[blockIdx.x];
    const int group = p.Hq / p.Hkv, h = blockIdx.y;
    if (r.b < 0 || r.unit % head_blocks * NH + h >= group) return;
    const int first = r.first, n = r.last - first + 1, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float* pieces = reinterpret_cast<const float*>(p.workspace + MAX_CTAS * sizeof(Record)) + (int64_t)first * 2 * L::PIECE;
    __shared__ float weight[MAX_CTAS], red[NW], part[AT * 4];
    auto piece = [&](int i) { return pieces + (int64_t)i * 2 * L::PIECE + (i == 0 ? r.slot * L::PIECE : 0); };
    float top = -INFINITY;
    for (int i = tid; i < n; i += AT) top = fmaxf(top, weight[i] = piece(i)[NH * D + h]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (lane == 0) red[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, red[w]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int i = tid; i < n; i += AT) {
        const float w = exp2_approx(weight[i] - base);
        weight[i] = w;
        sum += w * piece(i)[NH * D + NH + h];
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    __syncthreads();
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += red[w];
    constexpr int V = D / 4, G = AT / V;                // lanes of a piece, pieces at a time
    const int g = tid / V, c = tid % V;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = g; i < n; i += G) {
        const float4 x = *reinterpret_cast<const float4*>(piece(i) + h * D + 4 * c);
        const float w = weight[i];
        o.x += w * x.x;
        o.y += w * x.y;
        o.z += w * x.z;
        o.w += w * x.w;
    }
    reinterpret_cast<float4*>(part)[tid] = o;
    __syncthreads();
    const int64_t row = (int64_t)r.b * p.Hq + r.unit / head_blocks * group + r.unit % head_blocks * NH + h;
    for (int d = tid; d < D; d += AT) {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < G; ++k) x += part[k * D + d];
        store_from_float(static_cast<T*>(p.o), row * D + d, sum == 0.f ? 0.f : x / sum);
    }
    if (p.lse && tid == 0) p.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * LN2;
}


// No row has more tiles with a visible token, whatever its length: as many as its table's pages hold, or as the
// window and the first tokens touch.
int64_t most_tiles(const AttnParams& p, int tile) {
    const int64_t all = ((int64_t)p.max_pages * p.page_size + tile - 1) / tile;
    if (p.window == 0) return all;
    const int64_t seen = (p.sinks + (int64_t)tile - 1) / tile + (p.window + (int64_t)tile - 1) / tile + 1;
    return seen < all ? seen : all;
}

// Whether each unit is done by one CTA, however long: no search for the shares, no pieces, no second kernel.  It is
// decided from what the table and the window can hold, which the host knows, not from the lengths, which it does not: a
// table allocated for longer rows takes the other way (64 rows of 128 tokens 15.9 us instead of 12.4).  That
// pays where rows are short beside those: always up to four tiles (a row of 64 tokens 4.2 us instead of 6.0, of 256
// 6.9 instead of 7.4, 48 rows of 256 with 8 heads 12.9 instead of 18.0), and up to eight where the units fill a
// quarter of the GPU (48 rows of 512: 19.9 instead of 24.9, of 1 to 512: 10.3 instead of 12.0; but one row of 512: 9.7
// instead of 7.7).  With many units for each CTA that could be resident, each one's start shows instead: 1,024 units
// of 64 tokens 14.0 us instead of 14.3, 4,096 of them 42.8 instead of 35.8.
bool done_whole(int64_t units, int64_t tiles, int grid) {
    return units <= 3 * (int64_t)grid && (tiles <= 4 || (tiles <= 8 && 4 * units >= grid));
}

template <typename T, int D, int NH>
cudaError_t launch_core(AttnParams p, cudaStream_t s) {
    using L = Layout<T, D, NH>;
    static DeviceSetup done;
    int sms = 0;
    cudaError_t e = device_setup(done, reinterpret_cast<const void*>(kda_attn_kernel<T, D, NH>), L::BYTES, &sms);
    if (e != cudaSuccess) return e;
    // floor(2^(32 + shift) / page_size) + 1 with 2^shift < page_size <= 2^(shift + 1): exact for 31-bit tokens
    p.page_shift = 0;
    while ((2ll << p.page_shift) < p.page_size) ++p.page_shift;
    p.page_magic = p.page_size == 1 ? 0u : (uint32_t)((1ull << (32 + p.page_shift)) / p.page_size + 1);
    const int group = p.Hq / p.Hkv, head_blocks = (group + NH - 1) / NH;
    const int64_t all_units = (int64_t)p.B * p.Hkv * head_blocks;
    int grid = sms * L::CTAS_PER_SM < MAX_CTAS ? sms * L::CTAS_PER_SM : MAX_CTAS;
    p.whole = done_whole(all_units, most_tiles(p, L::TILE), grid);
    if (p.whole) grid = (int)all_units;
    kda_attn_kernel<T, D, NH><<<grid, AT, L::BYTES, s>>>(p, head_blocks, grid);
    e = cudaGetLastError();
    if (e != cudaSuccess || p.whole) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(all_units < grid ? (unsigned)all_units : grid, group < NH ? group : NH);
    cfg.blockDim = dim3(AT);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kda_attn_join_kernel<T, D, NH>, p, head_blocks);
}

template <typename T, int NH>
cudaError_t launch_d(const AttnParams& p, cudaStream_t s) {
    if (p.d == 16) return launch_core<T, 16, NH>(p, s);
    if (p.d == 64) return launch_core<T, 64, NH>(p, s);
    return launch_core<T, 128, NH>(p, s);
}

// Query heads that meet a key at once: the smallest variant that holds the group, else blocks of the largest.
int block_heads(int group, kda_dtype dt) {
    if (dt == KDA_DTYPE_BF16) return group <= 8 ? 8 : group <= 16 ? 16 : 32;
    return group == 1 ? 1 : group <= 4 ? 4 : group <= 8 ? 8 : 16;
}

}  // namespace

size_t attn_workspace(int32_t, int32_t Hq, int32_t Hkv, int32_t d, kda_dtype dt) {
    return MAX_CTAS * (sizeof(Record) + 2 * (size_t)piece_floats(block_heads(Hq / Hkv, dt), d) * sizeof(float));
}

cudaError_t launch_attention_decode(const AttnParams& p, kda_dtype dt, cudaStream_t s) {
    const int nh = block_heads(p.Hq / p.Hkv, dt);
    if (dt == KDA_DTYPE_BF16)
        return nh == 8 ? launch_d<__nv_bfloat16, 8>(p, s) : nh == 16 ? launch_d<__nv_bfloat16, 16>(p, s)
                                                                      : launch_d<__nv_bfloat16, 32>(p, s);
    if (nh == 1) return launch_d<float, 1>(p, s);
    if (nh == 4) return launch_d<float, 4>(p, s);
    if (nh == 8) return launch_d<float, 8>(p, s);
    return launch_d<float, 16>(p, s);
}

}  // namespace kda
