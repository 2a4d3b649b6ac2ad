// Attention of chunks of new tokens over a paged key-value cache, on the tensor cores (bf16, d = 64 and 128).
//
//   s_tj = scale * q_t . k_j over the visible j,   o_t = sum_j exp(s_tj - m_t) v_j / sum_j exp(s_tj - m_t)
//
// One persistent CTA per SM.  A unit is 256 (token, head) rows of a sequence and key-value head, as two blocks of 128: the
// rows of tcgen05 products S = Q K^T (operands in shared memory) and O += P V (P in tensor memory, where S was).  Two
// groups of four warps hold a row a thread: while one group takes the exponentials of its block, the tensor core works for
// the other.  One warp issues the products, one brings the pages in by TMA (boxes of the largest run of tokens that divides
// a page and fits the tile, through a table lookup each), and one looks after tiles that some row sees in part.
//
// Exponents are in base 2.  The reference that they are taken against only moves when a row's maximum has grown by
// more than 2^8, which rescales O in tensor memory; weights up to 256 lose nothing in bf16.  Weights are rounded to bf16
// for the second product, by half a step (2^-8 of a value) at most, and the outputs are divided by the sum of the rounded ones,
// so that an error that many weights share (keys of the same score) drops out and those of different ones are left: n weights of
// a size bring 1.1e-3 / sqrt(n) of a value.  Divided by the sum of the unrounded ones, 4,000 equal keys behind a higher
// one were off by 3.7e-3.  The sum before rounding, in fp32, gives lse.
//
// What is masked must not be multiplied: its weight is 0, and 0 * inf would be a NaN.  In tiles that are not open to every
// row the helper warp clears the values behind the last token, and takes values that are not finite out of the tile; the
// rows that see them add them when the unit is done, one by one.
//
// Every wait is bounded (KDA_DEVERR_TIMEOUT on expiry).
#include "kda_tc_util.cuh"

#include "kda_chunk_plan.cuh"

namespace kda {
namespace {

constexpr int TILE = 128;                     // rows of a block and of a tile
constexpr int UNIT = 2 * TILE;
constexpr int WARPS = 12, THREADS = WARPS * 32;
constexpr int MMA_WARP = 8, LOAD_WARP = 9, HELP_WARP = 10, QUERY_WARP = 11;
constexpr int TC_MAX_CTAS = 160;              // of the main kernel, whatever the GPU (bounds the workspace)
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr int EXTRA = 1;                      // tiles' time that a unit's queries and outputs take
constexpr float SLACK = 8.f;                  // the reference moves when the maximum has grown by 2^SLACK

// Tokens of a tile whose value is not finite, taken out of it.  A unit of 256 rows has at most eleven tiles that some row sees
// in part: tiles hold 65 tokens or more (box_of), the rows' own tokens touch 5 of them, the lower borders of their windows 5,
// the border of the first tokens 1.
constexpr int MAX_ODD = 11;
struct OddTiles {
    int32_t n;
    int32_t start[MAX_ODD];
    uint32_t rows[MAX_ODD][4];
};

constexpr int RING = 8;                       // runs whose lists are kept: the helper is at most 6 ahead of a reader

struct Barriers {
    uint64_t full[8], empty[8];               // of stages
    uint64_t fixed[8];                        // a stage's partly seen tile of V is ready for the product
    uint64_t q, q_empty;                      // a run's queries in shared memory, and read for the last time
    uint64_t s[2], p[2][2];                   // of row blocks: scores, the weights' two halves
    uint64_t first;                           // a run's products for the first block done
    uint64_t run, ack;                        // a run's products done, and the second block's group has seen that
    uint64_t done;                            // all products done
};

struct Misc {
    Barriers bar;
    OddTiles odd[RING];
    int64_t sums[WARPS];
    Share share;
    uint32_t tmem_base;
    uint32_t issued;                          // stages whose copies have been issued
    float zero;
};

template <int D>
struct TcLayout {
    static constexpr int HALVES = D / 64;                      // 128-byte columns of a tile
    static constexpr int HALF = TILE * 128;                    // bytes of one
    static constexpr int BLOCK = HALVES * HALF;                // bytes of a block of Q, K or V
    static constexpr int STAGES = D == 128 ? 5 : 8;            // K and V in turn
    static constexpr int Q = 0, KV = 2 * BLOCK, MISC = KV + STAGES * BLOCK, BYTES = MISC + (int)sizeof(Misc);
    static_assert(BYTES <= 227 * 1024, "shared memory of a CTA");
    static constexpr uint32_t S = 0, O = 2 * TILE;             // columns of tensor memory: S0, S1, O0, O1
};

__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t mbar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(done)
                 : "r"(mbar), "r"(parity)
                 : "memory");
    return done;
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint32_t mbar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(mbar)
        : "memory");
}
// The product with its A operand in tensor memory.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc));
}
// Descriptor of 16 tokens (K) by D columns (N) of a V tile: N contiguous, 128-byte swizzle, 64 columns HALF bytes from the
// next ones, 8 tokens 1 KiB from the next ones.
__device__ __forceinline__ uint64_t desc_v(uint32_t addr, uint32_t half) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((half >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024u >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// 32 columns of this thread's lane of tensor memory, on their way until tmem_wait32 has been called for them.
__device__ __forceinline__ void tmem_fetch32(uint32_t taddr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait32(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                   "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]),
                   "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]),
                   "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 x) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr) : "memory");
    return x;
}

// Tiles that are open: every row of the unit sees every token of them.  Among the first `near` ones (first tokens behind a
// window) those below a, else those from b to below c.
struct Open {
    int32_t near, a, b, c;
    __device__ __forceinline__ Open(const ChunkParams& p, const ChunkPlan& f, const Walk& w) {
        const int below = max(w.u.pos0 + 1, 0);                // tokens that the first row sees end here
        const int last = w.s.len - w.s.n + over(w.m * UNIT + w.u.rows - 1, f.by_group);
        near = w.u.near;
        a = over(min(p.sinks, below), f.by_tile);
        b = p.window > 0 && last >= p.window ? over(last - p.window, f.by_tile) + 1 - w.u.skip : 0;
        c = over(below, f.by_tile) - w.u.skip;
    }
    __device__ __forceinline__ bool operator()(int it) const { return it < near ? it < a : it >= b && it < c; }
};

// Adds the two weights of a packed pair to their sum.
__device__ __forceinline__ void add_bf16x2(float& sum, uint32_t x) {
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %1;\nadd.rn.f32.bf16 %0, l, %0;\nadd.rn.f32.bf16 %0, h, %0;\n}\n" : "+f"(sum) : "r"(x));
}

// 64 bytes of a row: whole 32-byte sectors at a time where the address allows it, since each lane has a row of its own.
__device__ __forceinline__ void store64(void* to, const uint32_t (&x)[16], bool wide) {
    uint32_t* p = static_cast<uint32_t*>(to);
    if (wide) {
#pragma unroll
        for (int i = 0; i < 16; i += 8)
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p + i), "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]),
                         "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 16; i += 4) *reinterpret_cast<uint4*>(p + i) = make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    }
}

// Reports a lane's boxes of tokens from j, j + 32 box, .. on that have no page, if some row sees a token of one.
__device__ __noinline__ void tell_bad_pages(const ChunkParams& p, bool a, bool b, bool c, bool d, int j, int box, int from) {
    auto seen = [&](int x) { return x + box > from || x < p.sinks; };
    if ((a && seen(j)) || (b && seen(j + 32 * box)) || (c && seen(j + 64 * box)) || (d && seen(j + 96 * box))) atomicOr(p.err, KDA_DEVERR_PAGES);
}

// Adds the tokens that were taken out of a run's tiles to a row that sees them; a whole warp.
template <int D>
__device__ __noinline__ void add_odd(const ChunkParams& p, const ChunkPlan& f, const OddTiles& list, int b, int h, int pos,
                                     const __nv_bfloat16* q, uint32_t t_o, float scale2, float base) {
    for (int e = 0; e < list.n; ++e)
        for (int x = 0; x < TILE; ++x) {
            if (!(list.rows[e][x >> 5] >> (x & 31) & 1u)) continue;
            const int j = list.start[e] + x, slot = over(j, f.by_page), page = __ldg(p.table + (int64_t)b * p.max_pages + slot);
            const int64_t off = ((int64_t)h * p.page_size + (j - slot * p.page_size)) * D;
            const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.k_pages) + page * p.k_stride + off;
            const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(p.v_pages) + page * p.v_stride + off;
            const bool seen = j <= pos && (p.window == 0 || j > pos - p.window || j < p.sinks);
            float s = 0.f;
            for (int c = 0; seen && c < D; ++c) s = fmaf(__bfloat162float(q[c]), __bfloat162float(k[c]), s);
            const float y = ex2_approx(s * scale2 - base);
            for (int c = 0; c < D; c += 16) {
                float o[16];
                __syncwarp();
                tmem_ld16(t_o + c, o);
                for (int i = 0; i < 16; ++i)
                    if (seen) o[i] = fmaf(y, __bfloat162float(v[c + i]), o[i]);
                tmem_st16(t_o + c, o);
                tmem_wait_st();
            }
        }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
kda_chunk_tc_kernel(ChunkParams p, ChunkPlan f, int box, int q_boxes, const __grid_constant__ CUtensorMap q_map,
                    const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using L = TcLayout<D>;
    extern __shared__ __align__(1024) unsigned char sm[];
    Misc& misc = *reinterpret_cast<Misc*>(sm + L::MISC);
    Barriers& bar = misc.bar;
    OddTiles* const odd = misc.odd;
    Share& share = misc.share;
    volatile uint32_t& issued = misc.issued;
    const uint32_t sm_q = saddr(sm) + L::Q, sm_kv = saddr(sm) + L::KV;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x, grid = gridDim.x;
    ChunkRecord* records = reinterpret_cast<ChunkRecord*>(p.workspace);

    if (tid == 0) {
        auto init = [](uint64_t* b, int n) { asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(n) : "memory"); };
        for (int i = 0; i < L::STAGES; ++i) init(&bar.full[i], 1), init(&bar.empty[i], 1);
        for (int i = 0; i < 8; ++i) init(&bar.fixed[i], 1);
        for (int i = 0; i < 2; ++i) init(&bar.s[i], 1), init(&bar.p[i][0], 4), init(&bar.p[i][1], 4);
        init(&bar.q, 1), init(&bar.q_empty, 1), init(&bar.first, 1), init(&bar.run, 1), init(&bar.ack, 4), init(&bar.done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        issued = 0;
        misc.zero = 0.f;
        if (!f.whole) records[cta].b = -1;
    }
    if (warp == MMA_WARP) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&misc.tmem_base)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (f.BN < TILE) {                        // rows that no copy ever fills
        for (int i = tid; i < L::STAGES * (L::BLOCK / 16); i += THREADS) st_shared16(sm_kv + i * 16, make_uint4(0, 0, 0, 0));
        fence_async_smem();
    }
    plan_share<WARPS>(p, f, misc.sums, &share, cta, grid);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc.tmem_base;
    auto wait_at = [&](uint32_t b, uint32_t parity) {          // each role that gives up leaves the others to give up, too
        if (mbar_test(b, parity & 1u) || mbar_wait(b, parity & 1u)) return true;
        atomicOr(p.err, KDA_DEVERR_TIMEOUT);
        return false;
    };
    auto wait = [&](uint64_t* b, uint32_t parity) { return wait_at(saddr(b), parity); };
    // every role steps through the same runs
    const bool work = share.left > 0 && Runs(p, f, share).count > 0;
    // Registers go from the warps that move data to those that hold rows: 2 x 192 + 120 = 3 x 168, what the launch has.
    if (warp < MMA_WARP) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        if (work) {
        // ---------------- softmax: a row a thread ----------------
        const int blk = warp >> 2, r = tid;   // rows 0..127 and 128..255 of the unit
        const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
        const uint32_t t_s = tmem + lanes + L::S + blk * TILE, t_o = tmem + lanes + L::O + blk * D;
        const float scale2 = fmaxf(p.scale * LOG2E, 1e-37f);               // above 0: 0 * -inf must not be met
        uint32_t ns = 0;                      // tiles of this block so far
        bool ok = true, first_unit = true;
        Runs runs(p, f, share);
        do {
            const Walk& w = runs.w;
            const int count = runs.count, tile = runs.tile, run = runs.run;
            const bool active = blk * TILE < w.u.rows;
            // The thread that tells the loader of free stages, when the scores of the last block are there: the products' thread
            // has no time for it (a commit behind products holds it up until they are done).
            const bool releases = lane == 0 && warp == (w.u.rows > TILE ? 4 : 0);
            float ref = -INFINITY, l = 0.f, lw = 0.f;      // lw: of the rounded weights
            bool part = false;                // the helper has looked at a tile of this run
            if (active) {
                const Open is_open(p, f, w);
                const int pos = r < w.u.rows ? max(w.s.len - w.s.n + over(w.m * UNIT + r, f.by_group), -1) : -1;
                for (int it = tile; it < tile + count; ++it, ++ns) {
                    const int j0 = tile_start(f, w.u, it);
                    const bool open = is_open(it);
                    part = part || !open;
                    ok = wait(&bar.s[blk], ns);
                    if (!ok) break;
                    tc_fence_after();
                    if (releases) {           // K of this tile and V of the one before have been read for the last time
                        const uint32_t n = 2 * (runs.before + it - tile);
                        arrive(&bar.empty[n % L::STAGES]);
                        if (it > tile) arrive(&bar.empty[(n - 1) % L::STAGES]);
                    }
                    __syncwarp();
                    float s[4][32], top[4];
                    auto top_of = [&](int c) {
                        top[c] = max3(s[c][0], s[c][1], s[c][2]);
#pragma unroll
                        for (int i = 3; i < 31; i += 2) top[c] = max3(top[c], s[c][i], s[c][i + 1]);
                        top[c] = fmaxf(top[c], s[c][31]);
                    };
                    tmem_fetch32(t_s, s[0]);
                    tmem_fetch32(t_s + 32, s[1]);
                    tmem_wait32(s[0]);
                    tmem_wait32(s[1]);
                    tmem_fetch32(t_s + 64, s[2]);
                    tmem_fetch32(t_s + 96, s[3]);
                    top_of(0);                // (in vain where something is masked)
                    top_of(1);
                    tmem_wait32(s[2]);
                    tmem_wait32(s[3]);
                    if (!open || f.BN < TILE) {
                        const int hi = min(pos - j0, f.BN - 1);
                        if (p.window == 0) {
#pragma unroll
                            for (int c = 0; c < TILE; ++c) s[c / 32][c % 32] = c <= hi ? s[c / 32][c % 32] : -INFINITY;
                        } else {
                            const int lo = max(pos - p.window, j0 - 1) - j0, near = p.sinks - j0;
#pragma unroll
                            for (int c = 0; c < TILE; ++c)
                                s[c / 32][c % 32] = c <= hi && (c > lo || c < near) ? s[c / 32][c % 32] : -INFINITY;
                        }
                        top_of(0);
                        top_of(1);
                    }
                    top_of(2);
                    top_of(3);
                    const float m = fmaxf(max3(top[0], top[1], top[2]), top[3]);
                    const bool move = (m - ref) * scale2 > SLACK;          // (NaN with nothing seen so far: no)
                    if (__any_sync(0xFFFFFFFFu, move)) {
                        const float to = move ? m : ref;
                        const float by = !move ? 1.f : ref == -INFINITY ? 0.f : ex2_approx((ref - to) * scale2);
                        l *= by, lw *= by;
                        if (it > tile) {      // the scores' barrier tells of the products issued before them, too
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                float o[16];
                                tmem_ld16(t_o + c, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] *= by;
                                tmem_st16(t_o + c, o);
                            }
                        }
                        ref = to;
                    }
                    const float base = ref == -INFINITY ? 0.f : ref * scale2;
                    const Pair by2 = pair_of(scale2, scale2), minus = pair_of(-base, -base);
                    Pair sum[2] = {pair_of(0.f, 0.f), pair_of(0.f, 0.f)};
                    float x[4][16];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 y = both(fma2(pair_of(s[c][2 * i], s[c][2 * i + 1]), by2, minus));
                            const float a = ex2_approx(y.x), b = ex2_approx(y.y);
                            x[c][i] = __uint_as_float(pack_bf16x2(a, b));
                            sum[i & 1] = add2(sum[i & 1], pair_of(a, b));
                        }
                        tmem_st16(t_s + 16 * c, x[c]);
                        if (c % 2 == 1) {     // half of the weights: the product may begin
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) arrive(&bar.p[blk][c / 2]);
                        }
                    }
                    const float2 sums2 = both(add2(sum[0], sum[1]));
                    l += sums2.x + sums2.y;
                    // The rounded weights' sum, behind their hand-over, one at a time, so that it leaves the other block the pipes:
                    // it begins with a zero that is read there, so that no compiler brings it forward.  (The prompt of 8,192
                    // tokens 442 us, without it 383; two and four chains 446 and 451, among the exponentials 452, with the halves
                    // taken apart by shifts 490 to 508, as a product on the old matrix path 500.)
                    float zero;
                    asm volatile("ld.volatile.shared.f32 %0, [%1];" : "=f"(zero) : "r"(saddr(&misc.zero)) : "memory");
                    lw += zero;
#pragma unroll
                    for (int i = 0; i < 64; ++i) add_bf16x2(lw, __float_as_uint(x[i / 16][i % 16]));
                }
            }
            // The second block waits for the whole run also where it has no rows, and says so, so that neither side gets
            // ahead by more than a run (a barrier's phases are told apart by one bit).
            if (ok) ok = blk == 0 ? wait(&bar.first, run) : wait(&bar.run, run);
            if (!ok) break;
            if (releases) arrive(&bar.empty[(2 * (runs.before + count) - 1) % L::STAGES]);
            __syncwarp();
            if (blk == 1 && lane == 0) arrive(&bar.ack);
            // ---- outputs, or a piece of them ----
            const bool starts = tile == 0, ends = tile + count == w.u.tiles, complete = starts && ends;
            if (active) {
                tc_fence_after();
                __syncwarp();
                const bool mine = r < w.u.rows;
                const int flat = w.m * UNIT + (mine ? r : 0), t = over(flat, f.by_group);
                const int64_t at = (int64_t)(w.s.start + t) * p.Hq + w.h * f.group + flat - t * f.group;
                const float base = ref == -INFINITY ? 0.f : ref * scale2;
                if (part && *const_cast<const volatile int32_t*>(&odd[run % RING].n) > 0)
                    add_odd<D>(p, f, odd[run % RING], w.b, w.h, mine ? w.s.len - w.s.n + t : -1,
                               static_cast<const __nv_bfloat16*>(p.q) + at * D, t_o, scale2, base);
                if (complete) {
                    const float inv = l == 0.f ? 0.f : 1.f / lw;
                    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.o) + at * D;
                    const bool wide = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float o[32];
                        tmem_ld32(t_o + c, o);
                        uint32_t x[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = l == 0.f ? 0u : pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
                        if (mine) store64(to + c, x, wide);
                    }
                    if (mine && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (base + log2f(l)) * LN2;
                } else {
                    float* piece = reinterpret_cast<float*>(p.workspace + TC_MAX_CTAS * sizeof(ChunkRecord)) +
                                   ((int64_t)cta * 2 + (first_unit ? 0 : 1)) * piece_floats(UNIT, D);
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float o[32];
                        tmem_ld32(t_o + c, o);
                        if (mine) {
#pragma unroll
                            for (int i = 0; i < 32; i += 16) store64(piece + r * D + c + i, reinterpret_cast<const uint32_t(&)[16]>(o[i]), true);
                        }
                    }
                    if (mine) piece[UNIT * D + r] = ref == -INFINITY ? -INFINITY : base, piece[UNIT * (D + 1) + r] = l, piece[UNIT * (D + 2) + r] = lw;
                }
                tc_fence_before();            // the next run's products overwrite O
            }
            if (tid == 0 && starts && !ends) {
                records[cta] = ChunkRecord{w.b, w.m, w.h, cta, cta_before(share, runs.end(f, share)), first_unit ? 0 : 1, {0, 0}};
            }
            first_unit = false;
            if (!runs.next(p, f)) break;
        } while (true);
    }
    } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    if (warp == LOAD_WARP && work) {
        // ---------------- pages ----------------
        // Lane x has the boxes x, x + 32, ..; the next tile's page numbers are on their way while this one is copied.
        uint32_t n = 0, st = 0, turn = 1;     // stages filled; the next one, and the phase of `empty` to wait for
        const int boxes = f.BN / box;
        bool ok = true;
        Runs runs(p, f, share);
        do {
            const Walk& w = runs.w;
            const int end = runs.tile + runs.count;
            const int32_t* table = p.table + (int64_t)w.b * p.max_pages;
            int next[4], next_row[4];
            auto look_up = [&](int it) {
                const int j0 = tile_start(f, w.u, it);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int x = lane + 32 * i, j = j0 + x * box;
                    next[i] = INT32_MIN;      // no box
                    if (32 * i < boxes && x < boxes && j < w.u.end) {
                        const int slot = over(j, f.by_page);
                        next_row[i] = j - slot * p.page_size;
                        next[i] = max(__ldg(table + slot), -1);
                    }
                }
            };
            look_up(runs.tile);
            for (int it = runs.tile; it < end && ok; ++it) {
                int page[4], row[4], found = 0;
                bool bad = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    page[i] = next[i], row[i] = next_row[i];
                    if (32 * i < boxes) {
                        if (page[i] >= p.num_pages) page[i] = -1;
                        bad = bad || page[i] == -1;
                        found += __popc(__ballot_sync(0xFFFFFFFFu, page[i] >= 0));
                    }
                }
                if (it + 1 < end) look_up(it + 1);
                const bool zeros = __any_sync(0xFFFFFFFFu, bad);
                if (zeros) {
                    const int j = tile_start(f, w.u, it) + lane * box;
                    tell_bad_pages(p, page[0] == -1, page[1] == -1, page[2] == -1, page[3] == -1, j, box, seen_from(p, w.u.pos0));
                }
                for (int v = 0; v < 2; ++v, ++n) {
                    ok = wait(&bar.empty[st], turn);
                    if (!ok) break;
                    const uint32_t to = sm_kv + st * L::BLOCK, full = saddr(&bar.full[st]);
                    if (zeros) {              // no such page
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (page[i] == -1)
                                for (int h = 0; h < L::HALVES; ++h)
                                    for (int y = 0; y < box * 8; ++y)
                                        st_shared16(to + h * L::HALF + (lane + 32 * i) * box * 128 + y * 16, make_uint4(0, 0, 0, 0));
                        fence_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_expect_tx(full, (uint32_t)(found * box * D * 2));
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (page[i] >= 0)
#pragma unroll
                            for (int h = 0; h < L::HALVES; ++h)
                                tma_load_4d(to + h * L::HALF + (lane + 32 * i) * box * 128, v ? &v_map : &k_map, h * 64, row[i], w.h, page[i], full);
                    if (lane == 0) issued = n + 1;
                    if (++st == L::STAGES) st = 0, turn ^= 1;
                }
            }
            if (!ok || !runs.next(p, f)) break;
        } while (true);
        // no copy is left in flight
        for (uint32_t i = n > L::STAGES ? n - L::STAGES : 0; i < n; ++i) mbar_wait(saddr(&bar.full[i % L::STAGES]), (i / L::STAGES) & 1u);
    } else if (warp == QUERY_WARP && work) {
        // ---------------- queries ----------------
        // Boxes of the heads that share a key and the tokens that fill a block, where the heads divide it; else row by row.
        bool ok = true;
        uint32_t boxed = 0;                   // runs whose queries came in boxes
        Runs runs(p, f, share);
        do {
            const Walk& w = runs.w;
            const int run = runs.run, row0 = w.m * UNIT;
            if (run > 0) ok = wait(&bar.q_empty, run - 1);
            if (!ok) break;
            if (q_boxes) {
                const int blocks = w.u.rows > TILE ? 2 : 1, t0 = w.s.start + over(row0, f.by_group), step = over(TILE, f.by_group);
                if (lane == 0) {
                    mbar_expect_tx(saddr(&bar.q), (uint32_t)(blocks * L::BLOCK));
                    for (int i = 0; i < blocks; ++i)
#pragma unroll
                        for (int h = 0; h < L::HALVES; ++h)
                            tma_load_3d(sm_q + i * L::BLOCK + h * L::HALF, &q_map, h * 64, w.h * f.group, t0 + i * step, saddr(&bar.q));
                }
                __syncwarp();
                ++boxed;
                if (!runs.next(p, f)) break;
                continue;
            }
            constexpr int PER = D / 8;        // 16-byte columns of a row
            const int c = lane % PER;
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + ((int64_t)w.s.start * p.Hq + w.h * f.group) * D + c * 8;
#pragma unroll 4
            for (int r = lane / PER; r < w.u.rows; r += 32 / PER) {        // rows behind the unit's last hold anything
                const int t = over(row0 + r, f.by_group), g = row0 + r - t * f.group;
                const uint32_t to = sm_q + (r >> 7) * L::BLOCK + (c >> 3) * L::HALF + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(q + ((int64_t)t * p.Hq + g) * D) : "memory");
            }
            cp_async_commit();
            cp_async_wait_all();
            fence_async_smem();
            __syncwarp();
            if (lane == 0) arrive(&bar.q);
            if (!runs.next(p, f)) break;
        } while (true);
        if (boxed) mbar_wait(saddr(&bar.q), (boxed - 1) & 1u);  // no copy is left in flight
    } else if (warp == HELP_WARP && work) {
        // ---------------- tiles that some row sees in part ----------------
        bool ok = true;
        Runs runs(p, f, share);
        do {
            const Walk& w = runs.w;
            const int count = runs.count, tile = runs.tile, run = runs.run;
            const Open is_open(p, f, w);
            OddTiles& list = odd[run % RING];
            bool begun = false;
            for (int it = tile; it < tile + count; ++it) {
                if (is_open(it)) continue;
                const int j0 = tile_start(f, w.u, it);
                if (!begun && lane == 0) list.n = 0;
                begun = true;
                // The copy has to have been issued before its barrier's phase can be told from the one before.
                const uint32_t n = 2 * (runs.before + it - tile) + 1, st = n % L::STAGES;
                const long long t0 = clock64();
                while (issued <= n && (ok = clock64() - t0 < kWaitLimit)) {}
                ok = ok && wait(&bar.full[st], n / L::STAGES);
                if (!ok) break;
                __syncwarp();
                {
                    const uint32_t at = sm_kv + st * L::BLOCK;
                    const int real = w.u.end - j0 < f.BN ? w.u.end - j0 : f.BN;     // may be less than 1: nothing is seen
                    // Tokens up to the first row's are hidden from nobody where there is no window.  A lane has rows
                    // 32 g + lane; eight lanes at a time read eight different 16-byte columns.
                    const int first = p.window == 0 ? max(w.u.pos0 + 1 - j0, 0) : 0;
                    uint32_t any = 0, bad[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int r = 32 * g + lane;
                        const uint32_t row = at + r * 128;
                        const bool look = r >= first && r < real;
                        uint32_t hit = 0;     // an exponent of all ones carries into the sign's place
                        if (__any_sync(0xFFFFFFFFu, look)) {
#pragma unroll
                            for (int c = 0; c < D / 8; ++c) {
                                const uint4 x = ld_shared16(row + (c >> 3) * L::HALF + (((c & 7) ^ (r & 7)) << 4));
                                hit |= ((x.x & 0x7F807F80u) + 0x00800080u) | ((x.y & 0x7F807F80u) + 0x00800080u) |
                                       ((x.z & 0x7F807F80u) + 0x00800080u) | ((x.w & 0x7F807F80u) + 0x00800080u);
                            }
                        }
                        const bool out = look && (hit & 0x80008000u);
                        bad[g] = __ballot_sync(0xFFFFFFFFu, out);
                        any |= bad[g];
                        if (out || r >= real) {
#pragma unroll
                            for (int c = 0; c < D / 8; ++c)
                                st_shared16(row + (c >> 3) * L::HALF + (((c & 7) ^ (r & 7)) << 4), make_uint4(0, 0, 0, 0));
                        }
                    }
                    if (any && lane == 0 && list.n < MAX_ODD) {
                        list.start[list.n] = j0;
#pragma unroll
                        for (int g = 0; g < 4; ++g) list.rows[list.n][g] = bad[g];
                        ++list.n;
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive(&bar.fixed[st]);
                }
            }
            if (!ok || !runs.next(p, f)) break;
        } while (true);
    } else if (warp == MMA_WARP && work) {
        // ---------------- products: one thread ----------------
        if (elect_one()) {
            const uint32_t id_s = idesc_bf16(TILE, TILE), id_o = idesc_bf16(TILE, D) | (1u << 16);  // V's columns are contiguous
            const uint64_t dq = desc_sw128(sm_q), dk = desc_sw128(sm_kv), dv = desc_v(sm_kv, L::HALF);
            constexpr uint32_t STEP = L::BLOCK >> 4;           // descriptors count in 16 bytes
            constexpr uint32_t S = L::STAGES;
            // The tensor core takes few products ahead, and every hundred cycles between two batches of them beyond that it
            // stands still.  So what the next tile needs is done while the products of P V run that were issued last.
            uint32_t st = 0, phase = 0, n0 = 0, n1 = 0, fixed = 0;         // next stage; tiles of each block; phases of `fixed`, a bit a stage
            bool ok = true;
            const uint32_t full = saddr(bar.full), p_full = saddr(&bar.p[0][0]), s_full = saddr(bar.s), q_empty = saddr(&bar.q_empty);
            auto filled = [&](uint32_t x, uint32_t ph) { ok = ok && wait_at(full + 8 * x, ph); };
            auto step = [&]() {
                if (++st == S) st = 0, phase ^= 1;
            };
            auto scores = [&](int i, uint64_t b) {             // S_i = Q_i K^T
                const uint64_t a = dq + i * STEP;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t o = ((ks / 4) * L::HALF + (ks % 4) * 32) >> 4;
                    umma_bf16_1(tmem + L::S + i * TILE, a + o, b + o, id_s, ks > 0);
                }
                umma_commit(s_full + 8 * i);
            };
            auto product = [&](int i, int half, uint64_t b, bool first) {      // O_i += P_i V, half of the tokens
#pragma unroll
                for (int ks = half * (TILE / 32); ks < (half + 1) * (TILE / 32); ++ks)
                    umma_bf16_ts(tmem + L::O + i * D, tmem + L::S + i * TILE + ks * 8, b + ks * (2048 >> 4), id_o, !first || ks > 0);
            };
            auto weights = [&](int i, int half, uint32_t n) {
                ok = ok && wait_at(p_full + 16 * i + 8 * half, n);
                if (ok) tc_fence_after();
                return ok;
            };
            // The next V: there, and looked after where some row sees it in part.
            auto values = [&](bool open) {
                filled(st, phase);
                if (!open && ok) {
                    ok = wait(&bar.fixed[st], fixed >> st);
                    fixed ^= 1u << st;
                }
                const uint64_t b = dv + st * STEP;
                step();
                return b;
            };
            Runs runs(p, f, share);
            do {
                const Walk& w = runs.w;
                int left = runs.count, it = runs.tile;         // tiles whose products are to come
                const bool two = w.u.rows > TILE;
                const Open is_open(p, f, w);
                ok = wait(&bar.q, runs.run);
                filled(st, phase);
                if (!ok) break;
                tc_fence_after();
                uint64_t k = dk + st * STEP;
                step();
                scores(0, k);
                if (two) scores(1, k);
                if (left == 1) umma_commit(q_empty);
                uint64_t v = values(is_open(it));
                bool first = true;
                if (two) {                                     // the other block's products cover the wait for a block's weights
                    while (ok) {
                        if (!weights(0, 1, n0)) break;
                        product(0, 0, v, first);
                        product(0, 1, v, first);
                        if (left > 1) {
                            filled(st, phase);
                            k = dk + st * STEP;
                            if (!ok) break;
                            scores(0, k);
                        } else {
                            umma_commit(saddr(&bar.first));
                        }
                        if (!weights(1, 1, n1)) break;
                        product(1, 0, v, first);
                        product(1, 1, v, first);
                        ++n0, ++n1;
                        if (--left == 0) break;
                        step();
                        v = values(is_open(++it));
                        first = false;
                        if (!ok) break;
                        scores(1, k);
                        if (left == 1) umma_commit(q_empty);
                    }
                } else {                                       // the first half of the weights starts the products
                    while (ok) {
                        if (!weights(0, 0, n0)) break;
                        product(0, 0, v, first);
                        if (!weights(0, 1, n0)) break;
                        product(0, 1, v, first);
                        ++n0;
                        if (--left == 0) break;
                        filled(st, phase);
                        k = dk + st * STEP;
                        step();
                        if (!ok) break;
                        scores(0, k);
                        if (left == 1) umma_commit(q_empty);
                        v = values(is_open(++it));
                        first = false;
                    }
                    umma_commit(saddr(&bar.first));
                }
                if (ok && runs.run > 0) ok = wait(&bar.ack, runs.run - 1);
                if (!ok) break;
                umma_commit(saddr(&bar.run));
            } while (runs.next(p, f));
            umma_commit(saddr(&bar.done));
        }
        __syncwarp();
        mbar_wait(saddr(&bar.done), 0);       // no product is left in flight
    }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// Tokens of a TMA box: the largest run that divides a page and of which at most 24 fill three quarters of a tile, else the
// largest of which whole ones fill more than half (one token always does).  2,048 tokens behind 6,000 (32 / 8 heads of 128), as
// many boxes that fill more against one that fills less: pages of 77, 11 of 11 302 us, one 360; of 66, 3 of 33 295, one 415; of 94,
// 64 of 2 803, one 302; of 67, 128 of one token 1,437, one 409.
int box_of(int page_size) {
    const int most = page_size < TILE ? page_size : TILE;
    for (int x = most; TILE / x <= 24; --x)
        if (page_size % x == 0 && 4 * (TILE / x * x) >= 3 * TILE) return x;
    int x = most;
    while (page_size % x || 2 * (TILE / x * x) <= TILE) --x;
    return x;
}

bool encode_pages(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const ChunkParams& p, const void* base, int64_t stride, int box) {
    const int64_t page = (int64_t)p.Hkv * p.page_size * p.d;
    const cuuint64_t dims[4] = {(cuuint64_t)p.d, (cuuint64_t)p.page_size, (cuuint64_t)p.Hkv, (cuuint64_t)p.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)p.d * 2, (cuuint64_t)p.page_size * p.d * 2, (cuuint64_t)(p.num_pages > 1 ? stride : page) * 2};
    const cuuint32_t boxes[4] = {64u, (cuuint32_t)box, 1u, 1u}, ones[4] = {1u, 1u, 1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries [T, H_q, d]: boxes of the heads that share a key and as many tokens as fill a block.
bool encode_queries(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const ChunkParams& p) {
    const int group = p.Hq / p.Hkv;
    const cuuint64_t dims[3] = {(cuuint64_t)p.d, (cuuint64_t)p.Hq, (cuuint64_t)p.T};
    const cuuint64_t strides[2] = {(cuuint64_t)p.d * 2, (cuuint64_t)p.Hq * p.d * 2};
    const cuuint32_t boxes[3] = {64u, (cuuint32_t)group, (cuuint32_t)(TILE / group)}, ones[3] = {1u, 1u, 1u};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_tc(const ChunkParams& p, cudaStream_t s) {
    static DeviceSetup done;
    int sms = 0;
    cudaError_t e = device_setup(done, reinterpret_cast<const void*>(kda_chunk_tc_kernel<D>), TcLayout<D>::BYTES, &sms);
    if (e != cudaSuccess) return e;
    const auto enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const int box = box_of(p.page_size);
    const int group = p.Hq / p.Hkv;
    const bool q_boxes = group <= TILE && TILE % group == 0;
    CUtensorMap q_map, k_map, v_map;
    if (q_boxes ? !encode_queries(enc, &q_map, p) : (std::memset(&q_map, 0, sizeof q_map), false)) return cudaErrorInvalidValue;
    if (!encode_pages(enc, &k_map, p, p.k_pages, p.k_stride, box) || !encode_pages(enc, &v_map, p, p.v_pages, p.v_stride, box))
        return cudaErrorInvalidValue;
    ChunkPlan f = chunk_plan(p, UNIT, TILE / box * box, EXTRA);
    int grid = sms < TC_MAX_CTAS ? sms : TC_MAX_CTAS;
    const int64_t units = most_units(p, f);
    // Where a unit has few tiles, whatever the lengths, pieces and a second kernel would cost more than they bring: 16 rows of one
    // token behind 100 and 400 (32 / 8 heads of 128) 9.9 and 15.5 us, in shares 19.0 and 21.4; 12 rows of 64 tokens behind 400 20.6
    // and 33.9; at the limit of units, 48 rows of one token behind 400, 45.2 and 45.0.
    f.whole = units <= 3 * (int64_t)grid && most_tiles(p, f) <= 2 * MIN_SHARE;
    if (f.whole) grid = (int)units;
    kda_chunk_tc_kernel<D><<<grid, THREADS, TcLayout<D>::BYTES, s>>>(p, f, box, q_boxes, q_map, k_map, v_map);
    e = cudaGetLastError();
    return e != cudaSuccess || f.whole ? e : launch_join<__nv_bfloat16, D>(p, f, grid, TC_MAX_CTAS, s);
}

}  // namespace

size_t chunk_tc_workspace(int32_t d) { return TC_MAX_CTAS * (sizeof(ChunkRecord) + 2 * (size_t)piece_floats(UNIT, d) * sizeof(float)); }

cudaError_t launch_attention_prefill_tc(const ChunkParams& p, cudaStream_t s) {
    return p.d == 64 ? launch_tc<64>(p, s) : launch_tc<128>(p, s);
}

}  // namespace kda
