// Slots and pages: copies within pools, the fork of a batch's KDA states, and the fork and the compaction
// of a paged cache.
//
// None of this computes anything; what it costs is the bytes that have to move and the latency of the
// bookkeeping in front of them.  So the bookkeeping is one kernel on one thread-block cluster, whose CTAs
// meet at the hardware's cluster barrier between the steps that depend on one another (a chain of small
// launches would pay a launch each), and the copies are one kernel over the whole GPU that reads its work
// list from the bookkeeping.  Every list is ranked by prefix sums, never by the order in which atomics
// arrive: two calls give the same tables.

#include <climits>

#include "kda_serve.cuh"

namespace kda {
namespace {

// ---- copies ----
// What bounds a copy is DRAM, which likes long runs of reads and of writes: three CTAs per SM, each with 32 KB
// on its way, and a few pieces per CTA, so that what is moved at a time lies together, move 192 states of 2 MiB
// at 7.3 TB/s (read and written, 110 us).  Pieces of 16 KB with four vectors a thread reach 6.5 TB/s and with eight
// resident CTAs per SM 5.2; a resident CTA that strides over all pieces 6.4; one CTA a piece 5.1 (each works its list out).
constexpr int CT = 256;                       // threads of a copying CTA
constexpr int COPY_CTAS = 3;                  // of them per SM
constexpr int CV = 8;                         // 16-byte vectors that a thread has in flight
constexpr int PIECE = 32768;                  // bytes of a slot that one group of threads moves at a time
constexpr int MOST_CTAS = 32;                 // copying CTAs launched per SM, at most

// The grid's threads move all pieces of n slots within one pool; slot_pair(i, src, dst) names the i-th copy (false:
// skip it).  A slot smaller than a piece is moved by fewer threads, so that small pages still fill the CTA.  A
// group goes from piece to piece by adding, and asks for the next pair before it moves the present one's data.
template <typename Pair>
__device__ __forceinline__ void copy_pool(const kda_pool& p, int64_t n, Pair slot_pair, unsigned* err, unsigned err_bit) {
    const int vecs_in_piece = PIECE / 16;
    const int64_t vecs = p.slot_bytes / 16;
    const int pieces = (int)((vecs + vecs_in_piece - 1) / vecs_in_piece);
    const int per = (int)((vecs + pieces - 1) / pieces);                   // vectors of a piece
    int lanes = 8;
    while (lanes < CT && lanes * CV < per) lanes *= 2;
    const int groups = CT / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    // unit = (pair * layers + layer) * pieces + piece; the grid's stride in the same three digits
    const unsigned first = blockIdx.x * groups + group, stride = gridDim.x * groups;
    if (first >= n * p.layers * pieces) return;
    int piece = first % pieces, layer = first / pieces % p.layers;
    int64_t pair = first / pieces / p.layers;
    const int piece_step = stride % pieces, layer_step = stride / pieces % p.layers, pair_step = stride / pieces / p.layers;
    int src = 0, dst = 0;
    bool moves = pair < n && slot_pair(pair, src, dst);
    while (pair < n) {
        const int from_piece = piece, from_layer = layer, from_src = src, from_dst = dst;
        const bool now = moves;
        piece += piece_step;
        int carry = piece >= pieces;
        piece -= carry * pieces;
        layer += layer_step + carry;
        carry = layer >= p.layers;
        layer -= carry * p.layers;
        pair += pair_step + carry;
        if (pair < n) moves = slot_pair(pair, src, dst);
        if (!now) continue;
        if ((unsigned)from_src >= (unsigned)p.slots || (unsigned)from_dst >= (unsigned)p.slots) {
            if (lane == 0) atomicOr(err, err_bit);
            continue;
        }
        char* base = static_cast<char*>(p.data) + from_layer * p.layer_stride + (int64_t)from_piece * per * 16;
        const uint4* from = reinterpret_cast<const uint4*>(base + from_src * p.slot_stride) + lane;
        uint4* to = reinterpret_cast<uint4*>(base + from_dst * p.slot_stride) + lane;
        const int64_t rest = vecs - (int64_t)from_piece * per;
        const int end = rest < per ? (int)rest : per;
        if (per == lanes * CV && end == per) {
            uint4 x[CV];
#pragma unroll
            for (int k = 0; k < CV; ++k) x[k] = __ldcs(from + k * lanes);
#pragma unroll
            for (int k = 0; k < CV; ++k) __stcs(to + k * lanes, x[k]);
        } else {
            for (int v = lane; v < end; v += lanes * CV, from += lanes * CV, to += lanes * CV) {
                uint4 x[CV];
#pragma unroll
                for (int k = 0; k < CV; ++k)
                    if (v + k * lanes < end) x[k] = __ldcs(from + k * lanes);
#pragma unroll
                for (int k = 0; k < CV; ++k)
                    if (v + k * lanes < end) __stcs(to + k * lanes, x[k]);
            }
        }
    }
}

// Copies the pairs of a list; its length is n, or *n_dev where an earlier kernel counts it.
__global__ void __launch_bounds__(CT, COPY_CTAS) kda_copy_kernel(const __grid_constant__ PoolSet set, const int32_t* src,
                                                      const int32_t* dst, int32_t n, const int32_t* n_dev,
                                                      unsigned* err) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t count = n_dev ? *n_dev : n;
    for (int i = 0; i < set.n; ++i)
        copy_pool(set.pool[i], count,
                  [&](int64_t pair, int& s, int& d) {
                      d = dst[pair];
                      s = src ? src[pair] : (int)pair;
                      return s >= 0 && d >= 0 && s != d;
                  },
                  err, KDA_DEVERR_PAGES);
}

// ---- block-wide exclusive prefix sums ----
template <typename T, int NT>
__device__ __forceinline__ T block_scan(T x, T& total, T* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T inc = x;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const T y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();                                   // warp_sums of an earlier scan is read no more
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    T before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const T s = warp_sums[w];
        if (w < warp) before += s;
        sum += s;
    }
    total = sum;
    return before + inc - x;
}

// ---- the fork of a batch's states ----
// Every CTA works out the whole plan (a few thousand integers at most) and copies its share, so that the
// call is one launch.  At the 8,192 rows that are allowed the plan is the cost: 0.22 ms, whether rows move or not.  Shared memory: first[B], then the rows that need a copy and the free rows.
__global__ void __launch_bounds__(CT, COPY_CTAS) kda_state_fork_kernel(const __grid_constant__ PoolSet set,
                                                            const int32_t* state_idx, const int32_t* parent, int32_t B,
                                                            int32_t* out, unsigned* err) {
    extern __shared__ int32_t fork_sm[];
    __shared__ unsigned long long sums[CT / 32];
    int32_t* first = fork_sm;
    uint16_t* extra = reinterpret_cast<uint16_t*>(first + B);
    uint16_t* freed = extra + B;
    for (int i = threadIdx.x; i < B; i += CT) first[i] = INT_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < B; i += CT) {
        const int p = parent[i];
        if (p >= 0 && p < B) atomicMin(&first[p], i);
        else if (p != -1 && blockIdx.x == 0) atomicOr(err, KDA_DEVERR_PARENT);
    }
    __syncthreads();
    // ranks of the rows that need a copy (bits 0-19), of the free rows (20-39) and of the new rows (40-59)
    unsigned long long base = 0;
    for (int t = 0; t < B; t += CT) {
        const int i = t + threadIdx.x;
        const int p = i < B ? parent[i] : -1;
        const bool goes_on = p >= 0 && p < B;
        const bool is_extra = goes_on && first[p] != i, is_free = i < B && first[i] == INT_MAX;
        const unsigned long long flags = (is_extra ? 1ull : 0) | (is_free ? 1ull << 20 : 0);
        unsigned long long total;
        const unsigned long long at = base + block_scan<unsigned long long, CT>(flags, total, sums);
        if (is_extra) extra[at & 0xFFFFF] = (uint16_t)i;
        if (is_free) freed[(at >> 20) & 0xFFFFF] = (uint16_t)i;
        base += total;
    }
    __syncthreads();
    const int copies = (int)(base & 0xFFFFF);
    if (blockIdx.x == 0) {
        for (int i = threadIdx.x; i < copies; i += CT) out[extra[i]] = state_idx[freed[i]];
        int started = 0;
        for (int t = 0; t < B; t += CT) {
            const int i = t + threadIdx.x;
            const int p = i < B ? parent[i] : -1;
            const bool goes_on = p >= 0 && p < B;
            unsigned long long total;
            const unsigned long long at = block_scan<unsigned long long, CT>(i < B && !goes_on ? 1 : 0, total, sums);
            if (goes_on && first[p] == i) out[i] = state_idx[p];
            if (i < B && !goes_on) out[i] = state_idx[freed[copies + started + (int)at]];
            started += (int)total;
        }
    }
    for (int i = 0; i < set.n; ++i)
        copy_pool(set.pool[i], copies,
                  [&](int64_t pair, int& s, int& d) {
                      s = state_idx[parent[extra[pair]]];
                      d = state_idx[freed[pair]];
                      return true;
                  },
                  err, KDA_DEVERR_STATE_IDX);
}

// ---- one cluster's bookkeeping ----
// 16 CTAs of 256 threads: fewer threads meet sooner at a barrier, more CTAs read the tables faster.  256 rows of up
// to 377 pages, 96,632 pages (copies included), measured together: 32.5 us; 8 x 256: 34.1, 8 x 512: 34.8, 8 x 1024: 36.9, 16 x 512: 33.6.
constexpr int NC = 16;                        // CTAs of the cluster
constexpr int PT = 256;                       // threads of each
// Tables and copies up to so many bytes are left to the cluster's CTAs, which saves a launch (2 us of the host's time).
// 4 rows of 32 KB pages, two pools: 4 layers (1 MB at most) 10.8 us against 11.0 in two launches, 16 layers 12.9
// against 11.6, 32 layers 16.9 against 12.0.
constexpr int64_t WHOLE_BYTES = 1 << 20;
static_assert(PT == CT, "the cluster's threads move pages as the copying kernels' do");

// Everything that the cluster's threads wrote before is seen by all of them after.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// What the bookkeeping of a fork leaves for the kernel that writes the tables and copies the pages.
struct RowPlan {
    int parent;                  // -1: none
    int shared;                  // pages taken over from the parent
    int need;                    // pages in all
    int fresh_at;                // rank of the first page of its own
};
struct ForkScratch {
    RowPlan* plan;               // [rows_out]
    int32_t* listed;             // [num_pages] each CTA's free pages, at its own part of the pages
    int32_t* fresh;              // [num_pages] the pages handed out, in order
    int32_t* src;                // [rows_out] the copies
    int32_t* dst;
    int32_t* totals;             // [NC] free pages listed per CTA; then pages handed out, copies
};

size_t pad(size_t ints) { return (ints + 63) / 64 * 64; }

ForkScratch fork_scratch(int32_t* w, int32_t rows_out, int32_t num_pages, size_t* ints) {
    ForkScratch s;
    size_t at = 0;
    auto take = [&](size_t n) { int32_t* p = w ? w + at : nullptr; at += pad(n); return p; };
    s.totals = take(NC + 2);
    s.plan = reinterpret_cast<RowPlan*>(take(4 * (size_t)rows_out));
    s.src = take(rows_out);
    s.dst = take(rows_out);
    s.listed = take(num_pages);
    s.fresh = take(num_pages);
    if (ints) *ints = at;
    return s;
}

__device__ __forceinline__ int pages_of(int len, int page_size) { return len / page_size + (len % page_size != 0); }

__device__ __forceinline__ int old_length(const ForkParams& p, int row) {
    const int len = p.lens[row];
    return len < 0 || len > p.max_pages * p.page_size ? 0 : len;
}

// The new rows' tables, a warp per row, and the copies of their pages.
__device__ __forceinline__ void fork_finish(const ForkParams p, const ForkScratch s, const PoolSet& set) {
    const int lane = threadIdx.x & 31, handed = s.totals[NC], copies = s.totals[NC + 1];
    for (int i = blockIdx.x * (CT / 32) + (threadIdx.x >> 5); i < p.rows_out; i += gridDim.x * (CT / 32)) {
        const RowPlan r = s.plan[i];
        const int32_t* from = p.table + (int64_t)r.parent * p.max_pages;
        int32_t* to = p.table_out + (int64_t)i * p.max_pages;
        constexpr int BATCH = 4;
        for (int j0 = lane; j0 < p.max_pages; j0 += 32 * BATCH) {
            int page[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int j = j0 + 32 * k, rank = r.fresh_at + j - r.shared;
                page[k] = j < r.shared ? from[j] : j < r.need && rank < handed ? s.fresh[rank] : -1;
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int j = j0 + 32 * k;
                if (j >= p.max_pages) break;
                if (j < r.shared && (page[k] < 0 || page[k] >= p.num_pages)) {
                    atomicOr(p.err, KDA_DEVERR_PAGES);
                    page[k] = -1;
                }
                to[j] = page[k];
            }
        }
    }
    for (int i = 0; i < set.n; ++i)
        copy_pool(set.pool[i], copies,
                  [&](int64_t pair, int& from, int& to) {
                      from = s.src[pair];
                      to = s.dst[pair];
                      return from >= 0;
                  },
                  p.err, KDA_DEVERR_PAGES);
}

// The bookkeeping: which pages every new row takes over and how many it needs of its own, the counts, and the
// lowest free pages, in order.  Every CTA works out all rows' plans in its own shared memory (first, count
// [rows_in], fresh_at, copy_at [rows_out]), which costs less than one more meeting of the cluster; counts and
// pages are divided among the CTAs.  WHOLE: the cluster also writes the tables and moves the pages.
template <bool WHOLE>
__global__ void __launch_bounds__(PT) kda_cache_fork_kernel(ForkParams p, ForkScratch s,
                                                            const __grid_constant__ PoolSet set) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ int32_t fork_sm[];
    __shared__ unsigned long long sums[PT / 32];
    const int cta = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const int gt = cta * PT + tid, gw = gt >> 5;
    constexpr int GT = NC * PT, GW = GT / 32;
    int32_t* first = fork_sm;
    int32_t* count = first + p.rows_in;
    int32_t* fresh_at = count + p.rows_in;
    int32_t* copy_at = fresh_at + p.rows_out;                    // -1: no copy
    const int cap = p.max_pages * p.page_size;

    if (p.ref_out != p.ref) {
        constexpr int BATCH = 16;                                // on their way together
        for (int i0 = gt; i0 < p.num_pages; i0 += BATCH * GT) {
            int ref[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
                if (i0 + k * GT < p.num_pages) ref[k] = p.ref[i0 + k * GT];
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
                if (i0 + k * GT < p.num_pages) p.ref_out[i0 + k * GT] = ref[k];
        }
    }
    for (int i = tid; i < p.rows_in; i += PT) {
        first[i] = INT_MAX;
        count[i] = 0;
    }
    __syncthreads();
    for (int i = tid; i < p.rows_out; i += PT) {
        const int q = p.parent[i];
        if (q >= 0 && q < p.rows_in) {
            atomicMin(&first[q], i);
            atomicAdd(&count[q], 1);
        } else if (q != -1 && cta == 0) {
            atomicOr(p.err, KDA_DEVERR_PARENT);
        }
    }
    __syncthreads();
    unsigned long long base = 0;                       // pages of their own (bits 0-31) and copies (32-63) so far
    for (int t = 0; t < p.rows_out; t += PT) {
        const int i = t + tid;
        unsigned long long mine = 0;
        RowPlan r;
        int len = 0;
        bool copy = false;
        if (i < p.rows_out) {
            r.parent = p.parent[i];
            if (r.parent < 0 || r.parent >= p.rows_in) r.parent = -1;
            len = r.parent < 0 ? 0 : old_length(p, r.parent);
            const int full = len / p.page_size;
            copy = len > full * p.page_size && first[r.parent] != i;
            r.shared = copy ? full : pages_of(len, p.page_size);
            int grow = p.grow ? p.grow[i] : 0;
            if (grow < 0 || grow > cap - len) {
                if (cta == 0) atomicOr(p.err, KDA_DEVERR_PAGES);
                grow = grow < 0 ? 0 : cap - len;
            }
            len += grow;
            r.need = pages_of(len, p.page_size);
            mine = (unsigned)(r.need - r.shared) | (copy ? 1ull << 32 : 0ull);
        }
        unsigned long long total;
        const unsigned long long at = base + block_scan<unsigned long long, PT>(mine, total, sums);
        if (i < p.rows_out) {
            r.fresh_at = fresh_at[i] = (int)(at & 0xFFFFFFFFu);
            copy_at[i] = copy ? (int)(at >> 32) : -1;
            if (i % NC == cta) s.plan[i] = r;
        }
        base += total;
    }
    const int wanted = (int)(base & 0xFFFFFFFFu), copies = (int)(base >> 32);
    cluster_sync();                                    // the counts' copy is complete

    // a row continued c times names its whole pages c times instead of once, and its last, partly filled one once
    // if anybody continues it
    for (int i = gw; i < p.rows_in; i += GW) {
        const int c = count[i], length = p.lens[i];
        if (lane == 0 && (length < 0 || length > cap)) atomicOr(p.err, KDA_DEVERR_PAGES);
        if (c == 1) continue;
        const int len = old_length(p, i), full = len / p.page_size, pages = full + (len % p.page_size != 0);
        const int32_t* row = p.table + (int64_t)i * p.max_pages;
        constexpr int BATCH = 12;
        for (int j0 = lane; j0 < pages; j0 += 32 * BATCH) {
            int page[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) page[k] = j0 + 32 * k < pages ? row[j0 + 32 * k] : 0;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int j = j0 + 32 * k, change = j < full ? c - 1 : c > 0 ? 0 : -1;
                if (j >= pages) break;
                if (page[k] < 0 || page[k] >= p.num_pages) atomicOr(p.err, KDA_DEVERR_PAGES);
                else if (change) atomicAdd(&p.ref_out[page[k]], change);
            }
        }
    }
    int available = 0, before = 0, mine = 0;           // free pages listed in all, before this CTA's, by it
    const int seg = (p.num_pages + NC - 1) / NC, p0 = min(cta * seg, p.num_pages), p1 = min(p0 + seg, p.num_pages);
    if (wanted > 0) {
        cluster_sync();                                // the counts are final
        // this CTA's lowest free pages, as many as all rows want together
        constexpr int BATCH = 4;
        for (int t = p0; t < p1 && mine < wanted; t += BATCH * PT) {
            int ref[BATCH], n = 0;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int i = t + tid * BATCH + k;
                ref[k] = i < p1 ? p.ref_out[i] : 1;
                n += ref[k] == 0;
            }
            unsigned long long found;
            int rank = mine + (int)block_scan<unsigned long long, PT>((unsigned long long)n, found, sums);
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
                if (ref[k] == 0) s.listed[p0 + rank++] = t + tid * BATCH + k;
            mine += (int)found;
        }
        if (tid == 0) s.totals[cta] = mine;
        cluster_sync();
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int n = s.totals[c];
            if (c < cta) before += n;
            available += n;
        }
        for (int r = tid; r < mine && before + r < wanted; r += PT) {
            const int page = s.listed[p0 + r];
            s.fresh[before + r] = page;
            p.ref_out[page] = 1;
        }
    }
    if (gt == 0) {
        s.totals[NC] = min(available, wanted);
        s.totals[NC + 1] = copies;
    }
    for (int i = gt; i < p.rows_out; i += GT) {
        int q = p.parent[i];
        if (q < 0 || q >= p.rows_in) q = -1;
        int len = q < 0 ? 0 : old_length(p, q);
        const int full = len / p.page_size, at = fresh_at[i];
        const int next = i + 1 < p.rows_out ? fresh_at[i + 1] : wanted;
        const bool copy = copy_at[i] >= 0;
        const int shared = copy ? full : pages_of(len, p.page_size);
        len += p.grow ? max(0, min(p.grow[i], cap - len)) : 0;
        if (next > at && next > available) {           // the row ends before its first page that is missing
            atomicOr(p.err, KDA_DEVERR_EXHAUSTED);
            len = min(len, (shared + max(0, available - at)) * p.page_size);
        }
        p.lens_out[i] = len;
        int src = -1, dst = -1;
        if (copy) {
            src = p.table[(int64_t)q * p.max_pages + full];
            if (at < available) {
                int c = 0, r = at;
                for (; c < NC - 1 && r >= s.totals[c]; ++c) r -= s.totals[c];
                dst = s.listed[min(c * seg, p.num_pages) + r];
            }
            if (src < 0 || src >= p.num_pages || dst < 0) {
                if (dst >= 0) atomicOr(p.err, KDA_DEVERR_PAGES);
                src = dst = -1;
            }
            s.src[copy_at[i]] = src;
            s.dst[copy_at[i]] = dst;
        }
        if (p.copy_src) {
            p.copy_src[i] = src;
            p.copy_dst[i] = dst;
        }
    }
    if (WHOLE) {
        cluster_sync();
        fork_finish(p, s, set);
    }
}

// What is more than the cluster should move by itself.
__global__ void __launch_bounds__(CT, COPY_CTAS) kda_cache_fork_finish_kernel(ForkParams p, ForkScratch s,
                                                                   const __grid_constant__ PoolSet set) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    fork_finish(p, s, set);
}

struct CompactScratch {
    int32_t* movers;             // [num_pages] live pages at n_live and above, the last first
    int32_t* holes;              // [num_pages] free pages below n_live
    int32_t* src;                // [num_pages] the copies
    int32_t* dst;
    int32_t* totals;             // [2][NC] live pages, holes per CTA; then the copies' number
};

CompactScratch compact_scratch(int32_t* w, int32_t num_pages, size_t* ints) {
    CompactScratch s;
    size_t at = 0;
    auto take = [&](size_t n) { int32_t* p = w ? w + at : nullptr; at += pad(n); return p; };
    s.totals = take(2 * NC + 1);
    s.movers = take(num_pages);
    s.holes = take(num_pages);
    s.src = take(num_pages);
    s.dst = take(num_pages);
    if (ints) *ints = at;
    return s;
}

// With n live pages and `below` of them under n, the live page of rank r >= below (counted from 0) goes to
// the hole of rank r - below.  `below` is known only once every CTA has counted, so the movers are listed
// from the last live page backwards (rank n - 1 first) and paired with the holes a step later.
__global__ void __launch_bounds__(PT) kda_cache_compact_kernel(CompactParams p, CompactScratch s) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ unsigned long long sums[PT / 32];
    const int cta = blockIdx.x, tid = threadIdx.x, gt = cta * PT + tid;
    constexpr int GT = NC * PT;
    const int seg = (p.num_pages + NC - 1) / NC, p0 = min(cta * seg, p.num_pages), p1 = min(p0 + seg, p.num_pages);

    constexpr int BATCH = 8;                           // neighbouring pages of a thread
    int mine = 0;
#pragma unroll 8
    for (int i = p0 + tid; i < p1; i += PT) mine += p.ref[i] > 0;
    unsigned long long total;
    block_scan<unsigned long long, PT>((unsigned long long)mine, total, sums);
    if (tid == 0) s.totals[cta] = (int)total;
    cluster_sync();
    int live = 0, n = 0;                               // live pages before this CTA's, and in all
    for (int c = 0; c < NC; ++c) {
        if (c < cta) live += s.totals[c];
        n += s.totals[c];
    }
    int my_holes = 0;
    for (int t = p0; t < p1; t += BATCH * PT) {
        int ref[BATCH], count = 0;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = t + tid * BATCH + k;
            ref[k] = i < p1 ? p.ref[i] : 0;
            count += ref[k] > 0;
        }
        unsigned long long found;
        int rank = live + (int)block_scan<unsigned long long, PT>((unsigned long long)count, found, sums);
        live += (int)found;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = t + tid * BATCH + k;
            if (i >= p1) break;
            const bool is_live = ref[k] > 0;
            if (is_live && i >= n) {
                s.movers[n - 1 - rank] = i;
            } else {
                p.page_map[i] = is_live ? i : -1;
                if (!is_live && i < n) {
                    s.holes[i - rank] = i;
                    ++my_holes;
                } else {
                    p.ref_out[i] = is_live ? ref[k] : 0;
                }
            }
            rank += is_live;
        }
    }
    block_scan<unsigned long long, PT>((unsigned long long)my_holes, total, sums);
    if (tid == 0) s.totals[NC + cta] = (int)total;
    cluster_sync();
    int moves = 0;
    for (int c = 0; c < NC; ++c) moves += s.totals[NC + c];
    if (gt == 0) s.totals[2 * NC] = moves;
    for (int i = gt; i < moves; i += GT) {
        const int src = s.movers[moves - 1 - i], dst = s.holes[i], ref = p.ref[src];
        s.src[i] = src;
        s.dst[i] = dst;
        p.page_map[src] = dst;
        p.ref_out[dst] = ref;
        p.ref_out[src] = 0;
    }
    cluster_sync();
    for (int64_t e0 = gt; e0 < p.entries; e0 += BATCH * GT) {
        int page[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) page[k] = e0 + k * GT < p.entries ? p.table[e0 + k * GT] : -1;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) page[k] = page[k] >= 0 && page[k] < p.num_pages ? p.page_map[page[k]] : -1;
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (e0 + k * GT < p.entries) p.table_out[e0 + k * GT] = page[k];
    }
}

// CTAs that copy n slots (at most): one per piece as far as they go.
int copy_grid(const PoolSet& set, int64_t n, int sms) {
    int64_t most = 1;
    for (int i = 0; i < set.n; ++i) {
        const int64_t units = n * set.pool[i].layers * ((set.pool[i].slot_bytes + PIECE - 1) / PIECE);
        most = units > most ? units : most;
    }
    return (int)(most < MOST_CTAS * (int64_t)sms ? most : MOST_CTAS * (int64_t)sms);
}

// `after`: the kernel works on what the one launched just before on this stream leaves, and waits for its end
// itself, so that its launch is already done by then.
template <typename... Args, typename... Given>
cudaError_t launch_wide(void (*kernel)(Args...), int grid, bool after, cudaStream_t s, const Given&... given) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(CT);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, given...);
}

template <typename... Args, typename... Given>
cudaError_t launch_cluster(void (*kernel)(Args...), size_t smem, cudaStream_t s, const Given&... given) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(NC);
    cfg.blockDim = dim3(PT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = NC;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, given...);
}

}  // namespace

cudaError_t launch_copy_pages(const PoolSet& pools, const int32_t* src, const int32_t* dst, int32_t n, unsigned* err,
                              cudaStream_t s) {
    static DeviceSetup done;
    int sms = 0;
    const cudaError_t e = device_setup(done, nullptr, 0, &sms);
    if (e != cudaSuccess) return e;
    const int32_t* none = nullptr;
    const int grid = copy_grid(pools, n, sms);
    return launch_wide(kda_copy_kernel, grid, false, s, pools, src, dst, n, none, err);
}

cudaError_t launch_state_fork(const PoolSet& pools, const int32_t* state_idx, const int32_t* parent, int32_t B,
                              int32_t* state_idx_out, unsigned* err, cudaStream_t s) {
    static DeviceSetup done;
    int sms = 0;
    const cudaError_t e = device_setup(done, reinterpret_cast<const void*>(kda_state_fork_kernel), KDA_FORK_MAX_ROWS * 8, &sms);
    if (e != cudaSuccess) return e;
    const int grid = copy_grid(pools, B, sms);
    kda_state_fork_kernel<<<grid, CT, (size_t)B * 8, s>>>(pools, state_idx, parent, B, state_idx_out, err);
    return cudaGetLastError();
}

size_t cache_fork_workspace(int32_t rows_out, int32_t num_pages) {
    size_t ints = 0;
    fork_scratch(nullptr, rows_out, num_pages, &ints);
    return ints * 4;
}

cudaError_t launch_cache_fork(const ForkParams& p, const PoolSet& pools, void* workspace, cudaStream_t s) {
    static DeviceSetup done[2];
    int64_t bytes = (int64_t)p.rows_out * p.max_pages * 4;
    for (int i = 0; i < pools.n; ++i) bytes += (int64_t)p.rows_out * pools.pool[i].layers * pools.pool[i].slot_bytes;
    const bool whole = bytes <= WHOLE_BYTES;
    auto* kernel = whole ? kda_cache_fork_kernel<true> : kda_cache_fork_kernel<false>;
    int sms = 0;
    cudaError_t e = device_setup(done[whole], reinterpret_cast<const void*>(kernel), KDA_FORK_MAX_ROWS * 16, &sms, true);
    if (e != cudaSuccess) return e;
    const ForkScratch sc = fork_scratch(static_cast<int32_t*>(workspace), p.rows_out, p.num_pages, nullptr);
    e = launch_cluster(kernel, ((size_t)p.rows_in + p.rows_out) * 8, s, p, sc, pools);
    if (e != cudaSuccess || whole || p.rows_out == 0) return e;
    const int rows = (p.rows_out + CT / 32 - 1) / (CT / 32), copies = copy_grid(pools, p.rows_out, sms);
    const int grid = rows > copies ? (rows < MOST_CTAS * sms ? rows : MOST_CTAS * sms) : copies;
    return launch_wide(kda_cache_fork_finish_kernel, grid, true, s, p, sc, pools);
}

size_t cache_compact_workspace(int32_t num_pages) {
    size_t ints = 0;
    compact_scratch(nullptr, num_pages, &ints);
    return ints * 4;
}

cudaError_t launch_cache_compact(const CompactParams& p, const PoolSet& pools, void* workspace, unsigned* err,
                                 cudaStream_t s) {
    if (p.num_pages == 0) {
        if (p.entries == 0) return cudaSuccess;
        return cudaMemsetAsync(p.table_out, 0xFF, p.entries * sizeof(int32_t), s);       // no page is live: all -1
    }
    static DeviceSetup done;
    int sms = 0;
    cudaError_t e = device_setup(done, reinterpret_cast<const void*>(kda_cache_compact_kernel), 0, &sms, true);
    if (e != cudaSuccess) return e;
    const CompactScratch sc = compact_scratch(static_cast<int32_t*>(workspace), p.num_pages, nullptr);
    e = launch_cluster(kda_cache_compact_kernel, 0, s, p, sc);
    if (e != cudaSuccess || pools.n == 0) return e;
    const int32_t most = p.num_pages / 2 + 1;
    const int grid = copy_grid(pools, most, sms);
    return launch_wide(kda_copy_kernel, grid, true, s, pools, (const int32_t*)sc.src, (const int32_t*)sc.dst, most,
                       (const int32_t*)(sc.totals + 2 * NC), err);
}

}  // namespace kda
