// How the work of attention over chunks of new tokens is cut into shares, for its kernels.
//
// The G = H_q / H_kv query heads of a key-value head read the same keys, so the rows of a product are (token, head)
// pairs: row r of a sequence's key-value head is token r / G with head r % G.  BM of them are a unit; its work is the
// tiles of BN tokens of the cache that any of its rows sees.  All units' tiles, numbered one after the other (all units
// of a head, then the next head), are cut into equal shares, one per CTA, so that one long prompt, many short ones
// and a few tokens behind a long context fill the GPU alike.  Every CTA works its own share out from cu_seqlens and
// seq_lens on the device: nothing launched for it, nothing for the host to know.  It takes 3 us for a few sequences as for 64,
// and grows with their number, since a warp steps through its sequences one at a time: 700 of one token 23 us in the slowest
// CTA (of a call of 255 us), 4,096 130 us (of 1,297).  (A unit's own cost, `extra` tiles, counts: without it the CTAs
// whose units are short were done 50 us after the others of a 455 us prompt.)
// A unit that a border between shares cuts leaves pieces (maximum, sums and unscaled outputs), which a second
// kernel joins in the order of the CTAs: no atomics, the same bits on every call.
#pragma once

#include "kda_prompt.cuh"

namespace kda {
namespace {

struct ChunkPlan {
    int32_t group;               // query heads of a key-value head
    int32_t BM;                  // rows of a unit, a power of two
    int32_t BN;                  // tokens of a tile
    int32_t extra;               // what a unit costs beside its tiles, in tiles
    int32_t whole;               // CTA i does unit i, and nothing is left to join
    Divisor by_page, by_group, by_tile;
};
inline ChunkPlan chunk_plan(const ChunkParams& p, int32_t BM, int32_t BN, int32_t extra) {
    const int32_t group = p.Hq / p.Hkv;
    return ChunkPlan{group, BM, BN, extra, 0, divisor(p.page_size), divisor(group), divisor(BN)};
}

// One sequence of the batch: its new tokens and its length, 0 where they are not valid.
struct Seq {
    int32_t start, n, len;
    bool bad_cu, bad_len;
};
__device__ __forceinline__ Seq seq_of(const ChunkParams& p, int b) {
    const int a = __ldg(p.cu + b), e = __ldg(p.cu + b + 1), len = __ldg(p.lens + b);
    Seq s;
    s.bad_cu = a < 0 || e < a || e > p.T || (b == 0 && a != 0);
    s.bad_len = len < 0 || (int64_t)len > (int64_t)p.max_pages * p.page_size;
    s.start = a;
    s.n = s.bad_cu ? 0 : e - a;
    s.len = s.bad_len ? 0 : len;
    s.bad_len = s.bad_len || s.n > s.len;     // new tokens before the first place: they see nothing
    return s;
}
__device__ __forceinline__ int units_of(const ChunkPlan& f, const Seq& s) {
    return (int)(((unsigned)(s.n * f.group) + f.BM - 1) / f.BM);          // rows are numbered in 31 bits, BM is a power of two
}

// A unit's rows and tiles.  Tile i < near covers tokens from i * BN, a later one from (i + skip) * BN.
struct Unit {
    int32_t rows;                // of BM
    int32_t pos0;                // position of the first row's token
    int32_t end;                 // tokens that any row sees end here
    int32_t near, skip, tiles;   // at least one tile, also where no row sees anything
};
// The first token that any row of a unit sees, but for the first ones of all (p.sinks).
__device__ __forceinline__ int seen_from(const ChunkParams& p, int pos0) {
    return p.window > 0 && pos0 >= p.window ? pos0 + 1 - p.window : 0;
}
__device__ __forceinline__ Unit unit_of(const ChunkParams& p, const ChunkPlan& f, const Seq& s, int m) {
    Unit u;
    const int row0 = m * f.BM, all = s.n * f.group;
    u.rows = all - row0 < f.BM ? all - row0 : f.BM;
    const int t0 = over(row0, f.by_group), t1 = over(row0 + u.rows - 1, f.by_group);
    u.pos0 = s.len - s.n + t0;
    const int last = s.len - s.n + t1;
    u.end = last < 0 ? 0 : last + 1;
    const int all_tiles = over(u.end + f.BN - 1, f.by_tile);
    u.near = 0, u.skip = 0;
    if (p.window > 0) {
        const int w0 = over(seen_from(p, u.pos0), f.by_tile);
        const int sinks = p.sinks < u.end ? p.sinks : u.end;
        u.near = sinks > 0 ? over(sinks - 1, f.by_tile) + 1 : 0;
        if (u.near > w0) u.near = w0;
        u.skip = w0 - u.near;
    }
    u.tiles = all_tiles - u.skip;
    if (u.tiles < 1) u.tiles = 1;
    return u;
}
__device__ __forceinline__ int tile_start(const ChunkPlan& f, const Unit& u, int i) {
    return (i < u.near ? i : i + u.skip) * f.BN;
}
__device__ __forceinline__ int64_t cost_of(const ChunkParams& p, const ChunkPlan& f, const Seq& s, int m) {
    return f.whole ? 1 : f.extra + unit_of(p, f, s, m).tiles;
}

// What a CTA does: `left` places from place `at` of unit m of sequence b and key-value head h on.  A unit has `extra` places
// for what it costs beside its tiles, and then one a tile (with whole shares, one in all).
struct Share {
    int64_t left;
    int64_t start;               // flat number of the first place
    int64_t all;                 // places of all shares
    int32_t ctas;                // shares
    int32_t h, b, m, at;
};

constexpr int MIN_SHARE = 2;                  // tiles: pieces of one would cost more to join than they save

// Works the CTA's share out; all its NW warps.  `sums` holds NW numbers, `out` the result, both in shared memory.
template <int NW>
__device__ __forceinline__ void plan_share(const ChunkParams& p, const ChunkPlan& f, int64_t* sums, Share* out, int cta, int grid) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned all = 0xFFFFFFFFu;
    const int b0 = (int)((int64_t)p.B * warp / NW), b1 = (int)((int64_t)p.B * (warp + 1) / NW);
    auto add = [&](int64_t x) {
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(all, x, o);
        return x;
    };
    // 32 sequences at a time: a lane sums a sequence's units where they are few, the warp one sequence after the other else
    int64_t mine = 0;
    for (int g = b0; g < b1; g += 32) {
        Seq s{0, 0, 0, false, false};
        if (g + lane < b1) s = seq_of(p, g + lane);
        if (cta == 0 && (s.bad_cu || s.bad_len))
            atomicOr(p.err, (s.bad_cu ? KDA_DEVERR_CU_SEQLENS : 0u) | (s.bad_len ? KDA_DEVERR_PAGES : 0u));
        const int units = units_of(f, s);
        if (!__any_sync(all, units > 32)) {
            for (int m = 0; m < units; ++m) mine += cost_of(p, f, s, m);
        } else {
            for (int i = 0; i < 32 && g + i < b1; ++i) {
                Seq x{__shfl_sync(all, s.start, i), __shfl_sync(all, s.n, i), __shfl_sync(all, s.len, i), false, false};
                const int n = units_of(f, x);
                for (int m = lane; m < n; m += 32) mine += cost_of(p, f, x, m);
            }
        }
    }
    mine = add(mine);
    if (lane == 0) sums[warp] = mine;
    if (tid == 0) out->left = 0;
    __syncthreads();
    int64_t head = 0, before = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < warp) before += sums[w];
        head += sums[w];
    }
    const int64_t total = head * p.Hkv;
    const int64_t least = MIN_SHARE + f.extra, most = f.whole ? total : (total + least - 1) / least;
    const int ctas = (int)(most < grid ? most : grid);
    if (cta >= ctas) {                        // (no work at all: ctas = 0)
        __syncthreads();
        return;
    }
    const int64_t x0 = total * cta / ctas, x1 = total * (cta + 1) / ctas;
    const int h = (int)(x0 / head);
    int64_t at = x0 - h * head - before;      // tiles of this warp's sequences before the share
    if (at >= 0 && at < sums[warp]) {
        bool found = false;
        for (int g = b0; g < b1 && !found; g += 32) {
            Seq s{0, 0, 0, false, false};
            if (g + lane < b1) s = seq_of(p, g + lane);
            for (int i = 0; i < 32 && g + i < b1 && !found; ++i) {
                Seq x{__shfl_sync(all, s.start, i), __shfl_sync(all, s.n, i), __shfl_sync(all, s.len, i), false, false};
                const int n = units_of(f, x);
                for (int m = 0; m < n && !found; m += 32) {
                    const int64_t c = m + lane < n ? cost_of(p, f, x, m + lane) : 0;
                    int64_t to = c;           // tiles up to and with this lane's unit
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int64_t y = __shfl_up_sync(all, to, o);
                        if (lane >= o) to += y;
                    }
                    const int64_t batch = __shfl_sync(all, to, 31);
                    if (at < batch) {
                        found = true;
                        if (at >= to - c && at < to)
                            *out = Share{x1 - x0, x0, total, ctas, h, g + i, m + lane, (int)(at - (to - c))};
                    } else {
                        at -= batch;
                    }
                }
            }
        }
    }
    __syncthreads();
}

// Steps through the units of a share; every warp that takes part has its own.
struct Walk {
    int32_t h, b, m;
    Seq s;
    Unit u;
    __device__ __forceinline__ void begin(const ChunkParams& p, const ChunkPlan& f, const Share& share) {
        h = share.h, b = share.b, m = share.m;
        s = seq_of(p, b);
        u = unit_of(p, f, s, m);
    }
    __device__ __forceinline__ void next(const ChunkParams& p, const ChunkPlan& f) {
        if (++m >= units_of(f, s)) {
            m = 0;
            do {
                if (++b == p.B) b = 0, ++h;
                s = seq_of(p, b);
            } while (units_of(f, s) == 0);
        }
        u = unit_of(p, f, s, m);
    }
};

// A run: the share's tiles of one unit.
struct Runs {
    Walk w;
    int64_t left;                // places of the share, from the run's first on
    int32_t at;                  // the run's first place in its unit
    int32_t tile, count, run;    // its first tile and how many; its number
    uint32_t before = 0;         // tiles of the runs before it
    __device__ __forceinline__ Runs(const ChunkParams& p, const ChunkPlan& f, const Share& share) : left(share.left), at(share.at), run(0) {
        w.begin(p, f, share);
        measure(f);
    }
    __device__ __forceinline__ void measure(const ChunkPlan& f) {
        if (f.whole) {
            tile = 0, count = w.u.tiles;
            return;
        }
        const int all = f.extra + w.u.tiles, end = left < all - at ? at + (int)left : all;
        tile = at > f.extra ? at - f.extra : 0;
        count = (end > f.extra ? end - f.extra : 0) - tile;
    }
    __device__ __forceinline__ bool next(const ChunkParams& p, const ChunkPlan& f) {
        left -= f.whole ? 1 : f.extra + w.u.tiles - at;
        if (left <= 0) return false;
        ++run;
        before += count;
        at = 0;
        w.next(p, f);
        measure(f);
        return count > 0;        // a share may end among the places before a unit's first tile: that unit is the next one's
    }
    // Flat number of the unit's end.
    __device__ __forceinline__ int64_t end(const ChunkPlan& f, const Share& share) const {
        return share.start + share.left - left + (f.extra + w.u.tiles - at);
    }
};

// A unit whose first tiles are in CTA `first`'s share and whose last ones in `last`'s; b = -1: none.
struct ChunkRecord {
    int32_t b, m, h, first, last, slot, pad[2];
};
// The share that flat tile x - 1 lies in.
__device__ __forceinline__ int cta_before(const Share& s, int64_t x) { return (int)((x * s.ctas - 1) / s.all); }

__host__ __device__ constexpr int64_t piece_floats(int BM, int D) { return (int64_t)BM * (D + 3); }

__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr int JOIN_WARPS = 4, JOIN_ROWS = 2;  // of a CTA, and of a warp at a time

template <int N>
struct alignas(4 * N) Floats {
    float x[N];
};

// Joins the pieces of a unit.  A piece is [BM][D] sums, then [BM] maxima (base 2), [BM] sums of the weights and [BM] sums of them
// as they were multiplied, which the outputs are divided by.  A lane works out the weight
// of one piece for each of the warp's rows; then all of them add the pieces up, a few columns each, with the next pieces'
// loads under way.
template <typename T, int D>
__global__ void __launch_bounds__(JOIN_WARPS * 32) kda_chunk_join_kernel(ChunkParams p, ChunkPlan f, int max_ctas) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const ChunkRecord r = reinterpret_cast<const ChunkRecord*>(p.workspace)[blockIdx.x];
    if (r.b < 0) return;
    const unsigned all = 0xFFFFFFFFu;
    const int lane = threadIdx.x & 31, row0 = (blockIdx.y * JOIN_WARPS + (threadIdx.x >> 5)) * JOIN_ROWS;
    const Seq s = seq_of(p, r.b);
    const int flat0 = r.m * f.BM + row0, rows = s.n * f.group - flat0;    // of the unit from the warp's first on
    if (rows <= 0) return;
    const int64_t size = piece_floats(f.BM, D);
    const float* pieces = reinterpret_cast<const float*>(p.workspace + max_ctas * sizeof(ChunkRecord));
    const int n = r.last - r.first + 1;
    auto piece = [&](int i) { return pieces + ((int64_t)(r.first + i) * 2 + (i == 0 ? r.slot : 0)) * size; };
    constexpr int PER = D / 32 > 0 ? D / 32 : 1;                          // columns of a lane
    const int col = lane * PER;
    float top[JOIN_ROWS], sum[JOIN_ROWS], by[JOIN_ROWS];
    Floats<PER> o[JOIN_ROWS];
#pragma unroll
    for (int k = 0; k < JOIN_ROWS; ++k) {
        top[k] = -INFINITY, sum[k] = by[k] = 0.f;
        for (int i = lane; i < n; i += 32) top[k] = fmaxf(top[k], piece(i)[(int64_t)f.BM * D + row0 + k]);
#pragma unroll
        for (int x = 16; x; x >>= 1) top[k] = fmaxf(top[k], __shfl_xor_sync(all, top[k], x));
#pragma unroll
        for (int c = 0; c < PER; ++c) o[k].x[c] = 0.f;
    }
    for (int i0 = 0; i0 < n; i0 += 32) {
        float w[JOIN_ROWS];
#pragma unroll
        for (int k = 0; k < JOIN_ROWS; ++k) {
            w[k] = 0.f;
            if (i0 + lane < n && k < rows) {
                const float* x = piece(i0 + lane) + row0 + k;
                w[k] = ex2_approx(x[(int64_t)f.BM * D] - (top[k] == -INFINITY ? 0.f : top[k]));
                sum[k] = fmaf(w[k], x[(int64_t)f.BM * (D + 1)], sum[k]);
                by[k] = fmaf(w[k], x[(int64_t)f.BM * (D + 2)], by[k]);
            }
        }
        const int count = n - i0 < 32 ? n - i0 : 32;
#pragma unroll 4
        for (int i = 0; i < count; ++i) {
            const float* x = piece(i0 + i) + (int64_t)row0 * D + col;
#pragma unroll
            for (int k = 0; k < JOIN_ROWS; ++k) {
                const float y = __shfl_sync(all, w[k], i);
                if (k >= rows || col >= D) continue;
                const Floats<PER> v = *reinterpret_cast<const Floats<PER>*>(x + k * D);
#pragma unroll
                for (int c = 0; c < PER; ++c) o[k].x[c] = fmaf(y, v.x[c], o[k].x[c]);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < JOIN_ROWS; ++k) {
#pragma unroll
        for (int x = 16; x; x >>= 1) sum[k] += __shfl_xor_sync(all, sum[k], x), by[k] += __shfl_xor_sync(all, by[k], x);
        if (k >= rows) continue;
        const int t = over(flat0 + k, f.by_group), head = r.h * f.group + flat0 + k - t * f.group;
        const int64_t at = (int64_t)(s.start + t) * p.Hq + head;
        if (col < D) {
#pragma unroll
            for (int c = 0; c < PER; ++c) put(static_cast<T*>(p.o) + at * D + col + c, sum[k] == 0.f ? 0.f : o[k].x[c] / by[k]);
        }
        if (p.lse && lane == 0) p.lse[at] = sum[k] == 0.f ? -INFINITY : (top[k] + log2f(sum[k])) * 0.6931471805599453f;
    }
}

template <typename T, int D>
cudaError_t launch_join(const ChunkParams& p, const ChunkPlan& f, int grid, int max_ctas, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(grid, f.BM / (JOIN_WARPS * JOIN_ROWS));
    cfg.blockDim = dim3(JOIN_WARPS * 32);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kda_chunk_join_kernel<T, D>, p, f, max_ctas);
}

// Tiles of a unit, whatever the lengths: as many as its table's pages hold, or as the window and the first tokens touch.
inline int64_t most_tiles(const ChunkParams& p, const ChunkPlan& f) {
    const int64_t all = ((int64_t)p.max_pages * p.page_size + f.BN - 1) / f.BN;
    if (p.window == 0) return all > 1 ? all : 1;
    const int64_t seen = ((int64_t)p.sinks + f.BN - 1) / f.BN + ((int64_t)p.window + (f.BM - 1) / f.group + f.BN - 1) / f.BN + 1;
    return seen < all ? seen : all > 1 ? all : 1;
}
inline int64_t most_units(const ChunkParams& p, const ChunkPlan& f) {
    return ((int64_t)p.T * f.group / f.BM + (p.B < p.T ? p.B : p.T)) * p.Hkv;
}

}  // namespace
}  // namespace kda
