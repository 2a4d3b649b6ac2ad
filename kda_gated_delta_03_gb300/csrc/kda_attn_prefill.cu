// Attention of chunks of new tokens over a paged key-value cache, on the CUDA cores.
//
//   s_tj = scale * q_t . k_j over the visible j,   o_t = sum_j exp(s_tj - m_t) v_j / sum_j exp(s_tj - m_t)
//
// in one pass over the keys with a running maximum and sum.  A unit is 64 (token, head) rows, a tile 64 tokens of the
// cache, taken from the pages row by row, so that any page size will do.  256 threads hold 4 x 4 scores and 4 x d / 16
// outputs each; keys and values share one buffer, and two CTAs an SM hide each other's loads.
//
// What is masked is never multiplied: a masked weight is stored as -1 and skipped, since 0 * inf would be a NaN.
#include "kda_chunk_plan.cuh"

namespace kda {

namespace {

constexpr int NT = 256, NW = NT / 32, BM = 64, BN = 64;
constexpr int EXTRA = 0;                      // a unit's queries and outputs take little beside a tile
constexpr int MAX_CTAS = 512;                 // of the main kernel, whatever the GPU (bounds the workspace)
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

template <int D>
struct Layout {
    static constexpr int LD = D + 4;                           // floats of a row of Q and K
    static constexpr int PLD = BN + 4;
    // Two CTAs an SM: at d = 128 the weights take the keys' place, and the next keys are fetched after them.
    static constexpr bool OWN_P = D < 128;
    static constexpr int Q = 0, K = BM * LD, V = K + BN * LD, P = OWN_P ? V + BN * D : K, BYTES = (V + BN * D + (OWN_P ? BM * PLD : 0)) * 4;
    static_assert((OWN_P || LD >= PLD) && BYTES <= 113 * 1024, "two CTAs an SM");
};

// Four elements from global memory, as floats.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u), __uint_as_float(x.y << 16),
                       __uint_as_float(x.y & 0xFFFF0000u));
}

template <typename T, int D>
__global__ void __launch_bounds__(NT, 2) kda_chunk_kernel(ChunkParams p, ChunkPlan f) {
    using L = Layout<D>;
    extern __shared__ float smem[];
    __shared__ int64_t sums[NW];
    __shared__ Share share;
    float *Qs = smem + L::Q, *Ks = smem + L::K, *Vs = smem + L::V, *Ps = smem + L::P;
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16, cta = blockIdx.x, grid = gridDim.x;
    ChunkRecord* records = reinterpret_cast<ChunkRecord*>(p.workspace);
    if (!f.whole && tid == 0) records[cta].b = -1;
    plan_share<NW>(p, f, sums, &share, cta, grid);
    if (share.left == 0) return;
    constexpr int CO = D / 16 < 4 ? D / 16 : 4, GO = D / 16 / CO;         // output columns of a thread: GO runs of CO
    const float scale2 = p.scale * LOG2E;
    float* pieces = f.whole ? nullptr : reinterpret_cast<float*>(p.workspace + MAX_CTAS * sizeof(ChunkRecord));
    Runs runs(p, f, share);
    bool first_unit = true;
    if (runs.count <= 0) return;
    do {
        const Walk& w = runs.w;
        const Unit& u = w.u;
        const int row0 = w.m * BM, tile = runs.tile, count = runs.count;
        // ---- the unit's queries ----
        for (int i = tid; i < BM * (D / 4); i += NT) {
            const int r = i / (D / 4), c = i % (D / 4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < u.rows) {
                const int t = over(row0 + r, f.by_group), h = row0 + r - t * f.group;
                x = load4(static_cast<const T*>(p.q) + ((int64_t)(w.s.start + t) * p.Hq + w.h * f.group + h) * D + c);
            }
            *reinterpret_cast<float4*>(Qs + r * L::LD + c) = x;
        }
        int pos[4];                                            // of this thread's rows; rows past the unit's see nothing
        float m[4], l[4], o[4][GO * CO];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            pos[i] = r < u.rows ? w.s.len - w.s.n + over(row0 + r, f.by_group) : -1;
            m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < GO * CO; ++c) o[i][c] = 0.f;
        }
        const int32_t* table = p.table + (int64_t)w.b * p.max_pages;
        // A tile's rows into shared memory: fp32 on its way until the copies of its group are waited for.
        auto fetch = [&](const void* pages, int64_t stride, int j0, float* to, int ld) {
            for (int i = tid; i < BN * (D / 4); i += NT) {
                const int r = i / (D / 4), c = i % (D / 4) * 4, j = j0 + r;
                const T* from = nullptr;
                if (j < u.end) {
                    const int slot = over(j, f.by_page), page = __ldg(table + slot);
                    if (page >= 0 && page < p.num_pages)
                        from = static_cast<const T*>(pages) + page * stride + ((int64_t)w.h * p.page_size + (j - slot * p.page_size)) * D + c;
                    else if (c == 0 && (j >= seen_from(p, u.pos0) || j < p.sinks))       // (in a tile, but seen by nobody: nothing wrong)
                        atomicOr(p.err, KDA_DEVERR_PAGES);
                }
                if constexpr (sizeof(T) == 4) {
                    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to + r * ld + c);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(from ? from : static_cast<const T*>(p.q)), "r"(from ? 16 : 0)
                                 : "memory");
                } else {
                    *reinterpret_cast<float4*>(to + r * ld + c) = from ? load4(from) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            asm volatile("cp.async.commit_group;\n" ::: "memory");
        };
        fetch(p.k_pages, p.k_stride, tile_start(f, u, tile), Ks, L::LD);
        for (int it = tile; it < tile + count; ++it) {
            const int j0 = tile_start(f, u, it);
            fetch(p.v_pages, p.v_stride, j0, Vs, D);
            asm volatile("cp.async.wait_group 1;\n" ::: "memory");         // the keys
            __syncthreads();
            float s[4][4] = {};
#pragma unroll 4
            for (int k = 0; k < D; k += 4) {
                float4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(Qs + (ty * 4 + i) * L::LD + k);
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * L::LD + k);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, s[i][j]))));
            }
            // every row of the unit sees every token of the tile: the first row's position bounds it from above, the last one's window from below
            const int last = w.s.len - w.s.n + over(row0 + u.rows - 1, f.by_group);
            const bool open = j0 + BN - 1 <= u.pos0 && (p.window == 0 || j0 > last - p.window || j0 + BN <= p.sinks);
            if (!L::OWN_P) __syncthreads();   // every thread has read the keys
            float grow[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float top = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = j0 + tx + 16 * j;
                    const bool seen = key <= pos[i] && (p.window == 0 || key > pos[i] - p.window || key < p.sinks);
                    s[i][j] = open || seen ? s[i][j] * scale2 : -INFINITY;
                    top = fmaxf(top, s[i][j]);
                }
#pragma unroll
                for (int x = 1; x < 16; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
                const float base = top == -INFINITY ? 0.f : top;
                grow[i] = ex2_approx(m[i] - base);
                m[i] = top;
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = j0 + tx + 16 * j;
                    const bool seen = key <= pos[i] && (p.window == 0 || key > pos[i] - p.window || key < p.sinks);
                    const float e = ex2_approx(s[i][j] - base);
                    sum += e;
                    Ps[(ty * 4 + i) * L::PLD + tx + 16 * j] = open || seen ? e : -1.f;
                }
#pragma unroll
                for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
                l[i] = l[i] * grow[i] + sum;
#pragma unroll
                for (int c = 0; c < GO * CO; ++c) o[i][c] *= grow[i];
            }
            asm volatile("cp.async.wait_group 0;\n" ::: "memory");         // the values
            __syncthreads();
            const bool more = it + 1 < tile + count;
            if (L::OWN_P && more) fetch(p.k_pages, p.k_stride, tile_start(f, u, it + 1), Ks, L::LD);
            auto product = [&](auto checked) {
#pragma unroll 2
                for (int j = 0; j < BN; j += 4) {
                    float e[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 x = *reinterpret_cast<const float4*>(Ps + (ty * 4 + i) * L::PLD + j);
                        e[i][0] = x.x, e[i][1] = x.y, e[i][2] = x.z, e[i][3] = x.w;
                    }
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
                        for (int g = 0; g < GO; ++g) {
                            float v[CO];
#pragma unroll
                            for (int c = 0; c < CO; ++c) v[c] = Vs[(j + jj) * D + g * 16 * CO + tx * CO + c];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int c = 0; c < CO; ++c)
                                    if (!decltype(checked)::value || e[i][jj] >= 0.f)
                                        o[i][g * CO + c] = fmaf(e[i][jj], v[c], o[i][g * CO + c]);
                        }
                }
            };
            if (open)
                product(std::false_type());
            else
                product(std::true_type());
            __syncthreads();
            if (!L::OWN_P && more) fetch(p.k_pages, p.k_stride, tile_start(f, u, it + 1), Ks, L::LD);
        }
        // ---- outputs, or a piece of them ----
        const bool starts = tile == 0, ends = tile + count == u.tiles, complete = starts && ends;
        float* piece = complete ? nullptr : pieces + ((int64_t)cta * 2 + (first_unit ? 0 : 1)) * piece_floats(BM, D);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            if (r >= u.rows) continue;
            if (complete) {
                const int t = over(row0 + r, f.by_group);
                const int64_t at = (int64_t)(w.s.start + t) * p.Hq + w.h * f.group + (row0 + r - t * f.group);
                const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
                for (int g = 0; g < GO; ++g)
#pragma unroll
                    for (int c = 0; c < CO; ++c)
                        put(static_cast<T*>(p.o) + at * D + g * 16 * CO + tx * CO + c, l[i] == 0.f ? 0.f : o[i][g * CO + c] * inv);
                if (p.lse && tx == 0) p.lse[at] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * LN2;
            } else {
#pragma unroll
                for (int g = 0; g < GO; ++g)
#pragma unroll
                    for (int c = 0; c < CO; ++c) piece[r * D + g * 16 * CO + tx * CO + c] = o[i][g * CO + c];
                if (tx == 0) piece[BM * D + r] = m[i], piece[BM * (D + 1) + r] = piece[BM * (D + 2) + r] = l[i];
            }
        }
        if (tid == 0 && starts && !ends)
            records[cta] = ChunkRecord{w.b, w.m, w.h, cta, cta_before(share, runs.end(f, share)), first_unit ? 0 : 1, {0, 0}};
        first_unit = false;
    } while (runs.next(p, f));
}

template <typename T, int D>
cudaError_t launch(const ChunkParams& p, cudaStream_t s) {
    static DeviceSetup done;
    int sms = 0;
    cudaError_t e = device_setup(done, reinterpret_cast<const void*>(kda_chunk_kernel<T, D>), Layout<D>::BYTES, &sms);
    if (e != cudaSuccess) return e;
    ChunkPlan f = chunk_plan(p, BM, BN, EXTRA);
    int grid = 2 * sms < MAX_CTAS ? 2 * sms : MAX_CTAS;
    const int64_t units = most_units(p, f);
    // Where a unit has few tiles, whatever the lengths, pieces and a second kernel would cost more than they bring: fp32, d = 64, 16
    // rows of one token behind 60 and 100 10.9 and 16.9 us, in shares 20.6 and 18.8; at the limit of tiles, 37 tokens behind 200,
    // eight rows 29.3 and 30.3, but one row 28.8 and 21.5.
    f.whole = units <= 3 * (int64_t)grid && most_tiles(p, f) <= 2 * MIN_SHARE;
    if (f.whole) grid = (int)units;
    kda_chunk_kernel<T, D><<<grid, NT, Layout<D>::BYTES, s>>>(p, f);
    e = cudaGetLastError();
    return e != cudaSuccess || f.whole ? e : launch_join<T, D>(p, f, grid, MAX_CTAS, s);
}

}  // namespace

size_t chunk_workspace(int32_t d, kda_dtype dt) {
    const size_t cores = MAX_CTAS * (sizeof(ChunkRecord) + 2 * (size_t)piece_floats(BM, d) * sizeof(float));
    const size_t tensor = dt == KDA_DTYPE_BF16 && d >= 64 ? chunk_tc_workspace(d) : 0;
    return cores > tensor ? cores : tensor;
}

// fp32 stays here: TF32's 11 bits would not keep its precision.  So do bf16 heads of 16, whose rows of 32 bytes leave a
// TMA box of an odd number of tokens off the 128-byte places it has to start at, tables without a page, and scales below
// zero, where the largest score is the smallest product.
cudaError_t launch_attention_prefill(const ChunkParams& p, kda_dtype dt, cudaStream_t s) {
    if (dt == KDA_DTYPE_BF16)
        return p.d >= 64 && p.max_pages > 0 && p.scale >= 0.f ? launch_attention_prefill_tc(p, s)
               : p.d == 16                  ? launch<__nv_bfloat16, 16>(p, s)
               : p.d == 64                  ? launch<__nv_bfloat16, 64>(p, s)
                                            : launch<__nv_bfloat16, 128>(p, s);
    return p.d == 16 ? launch<float, 16>(p, s) : p.d == 64 ? launch<float, 64>(p, s) : launch<float, 128>(p, s);
}

}  // namespace kda
