// C ABI of the decoding operators of a hybrid stack: host-side validation and dispatch.  As for the other
// entry points, every argument is checked before the first CUDA call, so a rejected call launches nothing.

#include <cmath>

#include "kda_serve.cuh"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool table_ok(const void* p) { return p && aligned(p, 4); }
size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
size_t esize(kda_dtype dt) { return dt == KDA_DTYPE_BF16 ? 2 : 4; }
bool known(kda_dtype dt) { return dt == KDA_DTYPE_F32 || dt == KDA_DTYPE_BF16; }
// Words of a row: places up to a chunk past its end are 32-bit numbers.
constexpr int32_t MOST_WORDS = INT32_MAX - (1 << 14) + 1;
// Pages of a pool and of a row's table: those that a grid or a warp steps over past the end are 32-bit numbers, too.
constexpr int32_t MOST_PAGES = INT32_MAX - (1 << 18) + 1, MOST_ROW_PAGES = INT32_MAX - 1023;
bool head_ok(int32_t d) { return d == 16 || d == 64 || d == 128; }

kda_status take_pools(const kda_pool* pools, int32_t n, int32_t slots, kda::PoolSet* out) {
    if (n < 0 || (n > 0 && !pools)) return KDA_ERR_INVALID_ARG;
    if (n > KDA_MAX_POOLS) return KDA_ERR_UNSUPPORTED;
    out->n = 0;
    for (int32_t i = 0; i < n; ++i) {
        const kda_pool& p = pools[i];
        if (p.layers < 0 || p.slots < 0 || p.slot_bytes < 0 || p.layer_stride < 0 || p.slot_stride < 0)
            return KDA_ERR_INVALID_ARG;
        if (p.slot_bytes % 16 || p.layer_stride % 16 || p.slot_stride % 16) return KDA_ERR_INVALID_ARG;
        if (p.slots > 1 && p.slot_stride < p.slot_bytes) return KDA_ERR_INVALID_ARG;
        if (slots >= 0 && p.slots != slots) return KDA_ERR_INVALID_ARG;
        if (p.layers == 0 || p.slots == 0 || p.slot_bytes == 0) continue;
        if (!p.data || !aligned(p.data, 16)) return KDA_ERR_INVALID_ARG;
        out->pool[out->n++] = p;
    }
    return KDA_OK;
}

kda_status take_workspace(const void* ws, size_t bytes, size_t need) {
    return need > 0 && (!ws || bytes < need || !aligned(ws, 256)) ? KDA_ERR_WORKSPACE : KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_attention_decode_workspace_size(int32_t B, int32_t H_q, int32_t H_kv, int32_t d, kda_dtype dt) {
    if (B <= 0 || H_q <= 0 || H_kv <= 0 || H_q % H_kv || !head_ok(d) || !known(dt)) return 0;
    return align_up(kda::attn_workspace(B, H_q, H_kv, d, dt), 256);
}

kda_status kda_attention_decode(const void* q, void* k_pages, void* v_pages, const int32_t* block_table,
                                const int32_t* seq_lens, const void* k_new, const void* v_new, int32_t B, int32_t H_q,
                                int32_t H_kv, int32_t d, int32_t num_pages, int32_t page_size, int32_t max_pages,
                                int64_t k_page_stride, int64_t v_page_stride, kda_dtype dt, float scale,
                                int32_t window, int32_t sinks, void* o, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream) {
    if (B < 0 || H_q <= 0 || H_kv <= 0 || d <= 0 || num_pages < 0 || page_size <= 0 || max_pages < 0 || window < 0 ||
        sinks < 0 || !std::isfinite(scale) || !known(dt))
        return KDA_ERR_INVALID_ARG;
    if (H_q % H_kv != 0) return KDA_ERR_INVALID_ARG;
    if ((int64_t)max_pages * page_size > INT32_MAX - 1023) return KDA_ERR_INVALID_ARG;    // a tile past the end counts, too
    if (B > INT32_MAX - 1023 || (int64_t)H_q * d > INT32_MAX) return KDA_ERR_INVALID_ARG;     // as does a step past the rows
    if (!head_ok(d)) return KDA_ERR_UNSUPPORTED;
    if (B == 0) return KDA_OK;
    if (!q || !o || !table_ok(seq_lens) || !aligned(q, 16) || !aligned(o, 16) || (lse && !aligned(lse, 4)))
        return KDA_ERR_INVALID_ARG;
    if ((k_new == nullptr) != (v_new == nullptr) || !aligned(k_new, 16) || !aligned(v_new, 16))
        return KDA_ERR_INVALID_ARG;
    if (max_pages > 0) {
        if (num_pages == 0 || !k_pages || !v_pages || !table_ok(block_table) || !aligned(k_pages, 16) ||
            !aligned(v_pages, 16))
            return KDA_ERR_INVALID_ARG;
        const int64_t page = (int64_t)H_kv * page_size * d, unit = 16 / (int64_t)esize(dt);
        if (k_page_stride % unit || v_page_stride % unit) return KDA_ERR_INVALID_ARG;
        if (num_pages > 1 && (k_page_stride < page || v_page_stride < page)) return KDA_ERR_INVALID_ARG;
    }
    if (take_workspace(workspace, workspace_bytes, kda_attention_decode_workspace_size(B, H_q, H_kv, d, dt)) != KDA_OK)
        return KDA_ERR_WORKSPACE;

    unsigned* err = nullptr;
    if (kda::device_error_word(&err) != KDA_OK) return KDA_ERR_CUDA;
    kda::AttnParams p{};
    p.q = q; p.k_pages = k_pages; p.v_pages = v_pages; p.table = block_table; p.lens = seq_lens;
    p.k_new = k_new; p.v_new = v_new; p.o = o; p.lse = lse;
    p.workspace = static_cast<unsigned char*>(workspace); p.err = err;
    p.k_stride = k_page_stride; p.v_stride = v_page_stride;
    p.B = B; p.Hq = H_q; p.Hkv = H_kv; p.d = d;
    p.num_pages = num_pages; p.page_size = page_size; p.max_pages = max_pages;
    p.window = window; p.sinks = sinks; p.scale = scale;
    return kda::launch_attention_decode(p, dt, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_beam_select_workspace_size(int32_t N, int32_t K, int32_t V, kda_dtype dt) {
    if (N <= 0 || K <= 0 || K > KDA_BEAM_MAX_K || V <= 0 || V > MOST_WORDS || !known(dt)) return 0;
    return align_up(kda::beam_workspace(N, K, V, dt), 256);
}

kda_status kda_beam_select(const void* logits, int64_t row_stride, const float* beam_scores, const uint8_t* finished,
                           int32_t eos_token, int32_t N, int32_t K, int32_t V, kda_dtype dt, float* scores,
                           int32_t* parent, int32_t* token, uint8_t* finished_out, void* workspace,
                           size_t workspace_bytes, void* stream) {
    if (N < 0 || K <= 0 || V <= 0 || !known(dt) || row_stride < V || eos_token < -1 || eos_token >= V)
        return KDA_ERR_INVALID_ARG;
    if (finished && eos_token < 0) return KDA_ERR_INVALID_ARG;
    if (K > KDA_BEAM_MAX_K) return KDA_ERR_UNSUPPORTED;
    // a candidate's place b * V + v and a row's number n * K + b are 32-bit
    if (V > MOST_WORDS || (int64_t)K * V > INT32_MAX || (int64_t)N * K > INT32_MAX) return KDA_ERR_TOO_LARGE;
    if (N == 0) return KDA_OK;
    if (!logits || !aligned(logits, esize(dt)) || !beam_scores || !aligned(beam_scores, 4) || !scores ||
        !aligned(scores, 4) || !table_ok(parent) || !table_ok(token))
        return KDA_ERR_INVALID_ARG;
    if (take_workspace(workspace, workspace_bytes, kda_beam_select_workspace_size(N, K, V, dt)) != KDA_OK)
        return KDA_ERR_WORKSPACE;
    kda::BeamParams p{};
    p.logits = logits; p.row_stride = row_stride; p.beam_scores = beam_scores; p.finished = finished;
    p.eos = eos_token; p.N = N; p.K = K; p.V = V;
    p.scores = scores; p.parent = parent; p.token = token; p.finished_out = finished_out;
    p.workspace = static_cast<unsigned char*>(workspace);
    return kda::launch_beam_select(p, dt, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_copy_pages(const kda_pool* pools, int32_t num_pools, const int32_t* src, const int32_t* dst, int32_t n,
                          void* stream) {
    kda::PoolSet set{};
    if (n < 0) return KDA_ERR_INVALID_ARG;
    const kda_status st = take_pools(pools, num_pools, -1, &set);
    if (st != KDA_OK) return st;
    if (n == 0 || set.n == 0) return KDA_OK;
    if (!table_ok(dst) || (src && !aligned(src, 4))) return KDA_ERR_INVALID_ARG;
    unsigned* err = nullptr;
    if (kda::device_error_word(&err) != KDA_OK) return KDA_ERR_CUDA;
    return kda::launch_copy_pages(set, src, dst, n, err, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_state_fork(const kda_pool* pools, int32_t num_pools, const int32_t* state_idx, const int32_t* parent,
                          int32_t B, int32_t* state_idx_out, void* stream) {
    kda::PoolSet set{};
    if (B < 0) return KDA_ERR_INVALID_ARG;
    const kda_status st = take_pools(pools, num_pools, -1, &set);
    if (st != KDA_OK) return st;
    if (B > KDA_FORK_MAX_ROWS) return KDA_ERR_TOO_LARGE;
    if (B == 0) return KDA_OK;
    if (!table_ok(state_idx) || !table_ok(parent) || !table_ok(state_idx_out)) return KDA_ERR_INVALID_ARG;
    if (state_idx_out == state_idx || state_idx_out == parent) return KDA_ERR_INVALID_ARG;
    unsigned* err = nullptr;
    if (kda::device_error_word(&err) != KDA_OK) return KDA_ERR_CUDA;
    return kda::launch_state_fork(set, state_idx, parent, B, state_idx_out, err, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_cache_fork_workspace_size(int32_t rows_in, int32_t rows_out, int32_t max_pages, int32_t num_pages) {
    if (rows_in < 0 || rows_out < 0 || max_pages < 0 || num_pages < 0 || (rows_in == 0 && rows_out == 0)) return 0;
    if (rows_in > KDA_FORK_MAX_ROWS || rows_out > KDA_FORK_MAX_ROWS) return 0;
    if (max_pages > MOST_ROW_PAGES || num_pages > MOST_PAGES) return 0;
    return align_up(kda::cache_fork_workspace(rows_out, num_pages), 256);
}

kda_status kda_cache_fork(const int32_t* block_table, const int32_t* seq_lens, int32_t rows_in, const int32_t* parent,
                          const int32_t* grow, int32_t rows_out, int32_t max_pages, int32_t page_size,
                          const int32_t* ref_count, int32_t num_pages, int32_t* block_table_out, int32_t* seq_lens_out,
                          int32_t* ref_count_out, int32_t* copy_src, int32_t* copy_dst, const kda_pool* pools,
                          int32_t num_pools, void* workspace, size_t workspace_bytes, void* stream) {
    if (rows_in < 0 || rows_out < 0 || max_pages < 0 || page_size <= 0 || num_pages < 0) return KDA_ERR_INVALID_ARG;
    if ((int64_t)max_pages * page_size > INT32_MAX || (int64_t)rows_out * max_pages > INT32_MAX ||
        (int64_t)rows_in * max_pages > INT32_MAX || max_pages > MOST_ROW_PAGES || num_pages > MOST_PAGES)
        return KDA_ERR_INVALID_ARG;
    kda::PoolSet set{};
    const kda_status st = take_pools(pools, num_pools, num_pages, &set);
    if (st != KDA_OK) return st;
    if (rows_in > KDA_FORK_MAX_ROWS || rows_out > KDA_FORK_MAX_ROWS) return KDA_ERR_TOO_LARGE;
    if (rows_in == 0 && rows_out == 0) return KDA_OK;
    if (rows_out > 0 && (!table_ok(parent) || !table_ok(seq_lens_out) || (grow && !aligned(grow, 4))))
        return KDA_ERR_INVALID_ARG;
    if (rows_out > 0 && max_pages > 0 && !table_ok(block_table_out)) return KDA_ERR_INVALID_ARG;
    if (rows_in > 0 && (!table_ok(seq_lens) || (max_pages > 0 && !table_ok(block_table)))) return KDA_ERR_INVALID_ARG;
    if (num_pages > 0 && (!table_ok(ref_count) || !table_ok(ref_count_out))) return KDA_ERR_INVALID_ARG;
    if ((copy_src == nullptr) != (copy_dst == nullptr) || !aligned(copy_src, 4) || !aligned(copy_dst, 4))
        return KDA_ERR_INVALID_ARG;
    if ((block_table_out && block_table_out == block_table) || (seq_lens_out && seq_lens_out == seq_lens))
        return KDA_ERR_INVALID_ARG;
    if (take_workspace(workspace, workspace_bytes,
                       align_up(kda::cache_fork_workspace(rows_out, num_pages), 256)) != KDA_OK)
        return KDA_ERR_WORKSPACE;
    unsigned* err = nullptr;
    if (kda::device_error_word(&err) != KDA_OK) return KDA_ERR_CUDA;
    kda::ForkParams p{};
    p.table = block_table; p.lens = seq_lens; p.parent = parent; p.grow = grow; p.ref = ref_count;
    p.table_out = block_table_out; p.lens_out = seq_lens_out; p.ref_out = ref_count_out;
    p.copy_src = copy_src; p.copy_dst = copy_dst; p.err = err;
    p.rows_in = rows_in; p.rows_out = rows_out; p.max_pages = max_pages; p.page_size = page_size; p.num_pages = num_pages;
    return kda::launch_cache_fork(p, set, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK
                                                                                                       : KDA_ERR_CUDA;
}

size_t kda_cache_compact_workspace_size(int32_t num_pages) {
    if (num_pages <= 0 || num_pages > MOST_PAGES) return 0;
    return align_up(kda::cache_compact_workspace(num_pages), 256);
}

kda_status kda_cache_compact(const int32_t* block_table, int32_t rows, int32_t max_pages, const int32_t* ref_count,
                             int32_t num_pages, int32_t* block_table_out, int32_t* ref_count_out, int32_t* page_map,
                             const kda_pool* pools, int32_t num_pools, void* workspace, size_t workspace_bytes,
                             void* stream) {
    if (rows < 0 || max_pages < 0 || num_pages < 0 || num_pages > MOST_PAGES || (int64_t)rows * max_pages > INT32_MAX)
        return KDA_ERR_INVALID_ARG;
    kda::PoolSet set{};
    const kda_status st = take_pools(pools, num_pools, num_pages, &set);
    if (st != KDA_OK) return st;
    const int64_t entries = (int64_t)rows * max_pages;
    if (entries > 0 && (!table_ok(block_table) || !table_ok(block_table_out))) return KDA_ERR_INVALID_ARG;
    if (num_pages > 0 && (!table_ok(ref_count) || !table_ok(ref_count_out) || !table_ok(page_map)))
        return KDA_ERR_INVALID_ARG;
    if (num_pages > 0 && (page_map == ref_count || page_map == ref_count_out)) return KDA_ERR_INVALID_ARG;
    if (num_pages == 0 && entries == 0) return KDA_OK;
    if (take_workspace(workspace, workspace_bytes, kda_cache_compact_workspace_size(num_pages)) != KDA_OK)
        return KDA_ERR_WORKSPACE;
    unsigned* err = nullptr;
    if (kda::device_error_word(&err) != KDA_OK) return KDA_ERR_CUDA;
    kda::CompactParams p{};
    p.table = block_table; p.ref = ref_count; p.table_out = block_table_out; p.ref_out = ref_count_out;
    p.page_map = page_map; p.entries = entries; p.num_pages = num_pages;
    return kda::launch_cache_compact(p, set, workspace, err, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
