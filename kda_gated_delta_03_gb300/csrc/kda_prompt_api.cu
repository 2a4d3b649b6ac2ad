// C ABI of the operators that bring prompts into a hybrid stack and score their tokens: host-side validation and
// dispatch.  As for the other entry points, every argument is checked before the first CUDA call.

#include <cmath>

#include "kda_prompt.cuh"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool table_ok(const void* p) { return p && aligned(p, 4); }
size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
size_t esize(kda_dtype dt) { return dt == KDA_DTYPE_BF16 ? 2 : 4; }
bool known(kda_dtype dt) { return dt == KDA_DTYPE_F32 || dt == KDA_DTYPE_BF16; }
bool head_ok(int32_t d) { return d == 16 || d == 64 || d == 128; }
constexpr int32_t MOST_WORDS = INT32_MAX - (1 << 14) + 1;     // places up to a chunk past a row's end are 32-bit numbers
constexpr int32_t MOST_ROWS = (1 << 28) - 1;                  // a row's clusters of CTAs are numbered in 31 bits
constexpr int64_t MOST_TOKEN = 1 << 30;                       // elements of a token: a CTA's steps past them count, too

// Sizes and addresses that both rotary calls have.
kda_status rotary_args(int32_t T, int32_t Hq, int32_t Hkv, int32_t d, int32_t rot, int64_t qs, int64_t ks, kda_dtype dt,
                       int32_t layout, float scale, const double* inv_freq) {
    if (T < 0 || Hq < 0 || Hkv < 0 || d <= 0 || rot < 0 || rot > d || rot % 2 || !known(dt) || !std::isfinite(scale) ||
        (layout != KDA_ROTARY_HALF && layout != KDA_ROTARY_INTERLEAVED))
        return KDA_ERR_INVALID_ARG;
    if (((int64_t)Hq + 2 * (int64_t)Hkv) * d >= MOST_TOKEN) return KDA_ERR_INVALID_ARG;
    if (qs < (int64_t)Hq * d || ks < (int64_t)Hkv * d) return KDA_ERR_INVALID_ARG;
    if (!head_ok(d)) return KDA_ERR_UNSUPPORTED;
    if (rot > 0 && (!inv_freq || !aligned(inv_freq, 8))) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// The pools of a paged cache and the table that names their pages.
bool pools_ok(const void* k, const void* v, const int32_t* table, int32_t num_pages, int32_t page_size, int32_t max_pages,
              int32_t Hkv, int32_t d, int64_t ks, int64_t vs, kda_dtype dt) {
    if (max_pages == 0) return true;
    if (num_pages == 0 || !k || !v || !table_ok(table) || !aligned(k, 16) || !aligned(v, 16)) return false;
    const int64_t page = (int64_t)Hkv * page_size * d, unit = 16 / (int64_t)esize(dt);
    if (ks % unit || vs % unit) return false;
    return num_pages == 1 || (ks >= page && vs >= page);
}

}  // namespace

extern "C" {

kda_status kda_rotary(const void* q, const void* k, const int32_t* positions, const double* inv_freq, int32_t T,
                      int32_t H_q, int32_t H_kv, int32_t d, int32_t rotary_dim, int64_t q_stride, int64_t k_stride,
                      kda_dtype dt, int32_t layout, float rotary_scale, int32_t inverse, void* q_out,
                      int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
    if (!k) H_kv = 0, k_stride = k_out_stride = 0, k_out = nullptr;
    const kda_status st = rotary_args(T, H_q, H_kv, d, rotary_dim, q_stride, k_stride, dt, layout, rotary_scale, inv_freq);
    if (st != KDA_OK) return st;
    if (q_out_stride < (int64_t)H_q * d || k_out_stride < (int64_t)H_kv * d) return KDA_ERR_INVALID_ARG;
    if (T == 0 || H_q + H_kv == 0) return KDA_OK;
    const size_t e = esize(dt);
    if (!table_ok(positions) || (H_q > 0 && (!q || !q_out)) || (H_kv > 0 && !k_out) || !aligned(q, e) || !aligned(q_out, e) ||
        !aligned(k, e) || !aligned(k_out, e))
        return KDA_ERR_INVALID_ARG;
    if ((q_out == q && q_out_stride != q_stride) || (k && k_out == k && k_out_stride != k_stride)) return KDA_ERR_INVALID_ARG;
    kda::RotaryParams p{};
    p.q = q; p.k = k; p.positions = positions; p.inv_freq = inv_freq; p.q_out = q_out; p.k_out = k_out;
    p.q_stride = q_stride; p.k_stride = k_stride; p.q_out_stride = q_out_stride; p.k_out_stride = k_out_stride;
    p.T = T; p.Hq = H_q; p.Hkv = H_kv; p.d = d; p.rot = rotary_dim;
    p.interleaved = layout == KDA_ROTARY_INTERLEAVED; p.scale = rotary_scale; p.sign = inverse ? -1.f : 1.f;
    return kda::launch_rotary(p, dt, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_cache_append(const void* q, const void* k, const void* v, void* k_pages, void* v_pages,
                            const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_seqlens,
                            const double* inv_freq, int32_t B, int32_t T, int32_t H_q, int32_t H_kv, int32_t d,
                            int32_t rotary_dim, int64_t q_stride, int64_t k_stride, int64_t v_stride, int32_t num_pages,
                            int32_t page_size, int32_t max_pages, int64_t k_page_stride, int64_t v_page_stride,
                            kda_dtype dt, int32_t layout, float rotary_scale, void* q_out, int64_t q_out_stride,
                            void* stream) {
    if (!q) H_q = 0, q_stride = q_out_stride = 0, q_out = nullptr;
    const kda_status st = rotary_args(T, H_q, H_kv, d, rotary_dim, q_stride, k_stride, dt, layout, rotary_scale, inv_freq);
    if (st != KDA_OK) return st;
    if (B < 0 || B > INT32_MAX - 1023 || H_kv == 0 || num_pages < 0 || page_size <= 0 || max_pages < 0 || v_stride < (int64_t)H_kv * d ||
        q_out_stride < (int64_t)H_q * d || (int64_t)max_pages * page_size > INT32_MAX - 1023)
        return KDA_ERR_INVALID_ARG;
    if (T == 0 || B == 0) return KDA_OK;
    const size_t e = esize(dt);
    if (!k || !v || !table_ok(seq_lens) || !table_ok(cu_seqlens) || (H_q > 0 && !q_out) || !aligned(q, e) ||
        !aligned(q_out, e) || !aligned(k, e) || !aligned(v, e) || (q && q_out == q && q_out_stride != q_stride))
        return KDA_ERR_INVALID_ARG;
    // with max_pages = 0 no token has a place, and the (unread) table may be anything
    if (!pools_ok(k_pages, v_pages, block_table, num_pages, page_size, max_pages, H_kv, d, k_page_stride, v_page_stride, dt))
        return KDA_ERR_INVALID_ARG;
    unsigned* err = nullptr;
    if (kda::device_error_word(&err) != KDA_OK) return KDA_ERR_CUDA;
    kda::RotaryParams p{};
    p.q = q; p.k = k; p.v = v; p.inv_freq = inv_freq; p.q_out = q_out; p.k_pages = k_pages; p.v_pages = v_pages;
    p.table = block_table; p.lens = seq_lens; p.cu = cu_seqlens; p.err = err; p.append = 1;
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride; p.q_out_stride = q_out_stride;
    p.k_page_stride = k_page_stride; p.v_page_stride = v_page_stride;
    p.B = B; p.T = T; p.Hq = H_q; p.Hkv = H_kv; p.d = d; p.rot = rotary_dim;
    p.num_pages = num_pages; p.page_size = page_size; p.max_pages = max_pages;
    p.interleaved = layout == KDA_ROTARY_INTERLEAVED; p.scale = rotary_scale; p.sign = 1.f;
    return kda::launch_rotary(p, dt, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_attention_prefill_workspace_size(int32_t B, int32_t T, int32_t H_q, int32_t H_kv, int32_t d, kda_dtype dt) {
    if (B <= 0 || T <= 0 || H_q <= 0 || H_kv <= 0 || H_q % H_kv || !head_ok(d) || !known(dt)) return 0;
    return align_up(kda::chunk_workspace(d, dt), 256);
}

kda_status kda_attention_prefill(const void* q, const void* k_pages, const void* v_pages, const int32_t* block_table,
                                 const int32_t* seq_lens, const int32_t* cu_seqlens, int32_t B, int32_t T, int32_t H_q,
                                 int32_t H_kv, int32_t d, int32_t num_pages, int32_t page_size, int32_t max_pages,
                                 int64_t k_page_stride, int64_t v_page_stride, kda_dtype dt, float scale,
                                 int32_t window, int32_t sinks, void* o, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    if (B < 0 || T < 0 || H_q <= 0 || H_kv <= 0 || d <= 0 || num_pages < 0 || page_size <= 0 || max_pages < 0 || window < 0 ||
        sinks < 0 || !std::isfinite(scale) || !known(dt) || H_q % H_kv)
        return KDA_ERR_INVALID_ARG;
    if ((int64_t)max_pages * page_size > INT32_MAX - 1023) return KDA_ERR_INVALID_ARG;    // a tile past the end counts, too
    if (B > INT32_MAX - 1023 || (int64_t)H_q * d > INT32_MAX || (int64_t)T * H_q > INT32_MAX) return KDA_ERR_INVALID_ARG;
    if (!head_ok(d)) return KDA_ERR_UNSUPPORTED;
    if (B == 0 || T == 0) return KDA_OK;
    if (!q || !o || !table_ok(seq_lens) || !table_ok(cu_seqlens) || !aligned(q, 16) || !aligned(o, 16) || (lse && !aligned(lse, 4)))
        return KDA_ERR_INVALID_ARG;
    if (!pools_ok(k_pages, v_pages, block_table, num_pages, page_size, max_pages, H_kv, d, k_page_stride, v_page_stride, dt))
        return KDA_ERR_INVALID_ARG;
    const size_t need = kda_attention_prefill_workspace_size(B, T, H_q, H_kv, d, dt);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return KDA_ERR_WORKSPACE;
    unsigned* err = nullptr;
    if (kda::device_error_word(&err) != KDA_OK) return KDA_ERR_CUDA;
    kda::ChunkParams p{};
    p.q = q; p.k_pages = k_pages; p.v_pages = v_pages; p.table = block_table; p.lens = seq_lens; p.cu = cu_seqlens;
    p.o = o; p.lse = lse; p.workspace = static_cast<unsigned char*>(workspace); p.err = err;
    p.k_stride = k_page_stride; p.v_stride = v_page_stride;
    p.B = B; p.T = T; p.Hq = H_q; p.Hkv = H_kv; p.d = d;
    p.num_pages = num_pages; p.page_size = page_size; p.max_pages = max_pages;
    p.window = window; p.sinks = sinks; p.scale = scale;
    return kda::launch_attention_prefill(p, dt, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_token_logprobs(const void* logits, int64_t row_stride, const int32_t* tokens, int32_t T, int32_t V,
                              kda_dtype dt, int32_t top, float* logp, float* lse, float* entropy, float* top_logp,
                              int32_t* top_token, void* stream) {
    if (T < 0 || V <= 0 || !known(dt) || row_stride < V || top < 0 || top > V) return KDA_ERR_INVALID_ARG;
    if (top > KDA_LOGPROBS_MAX_TOP) return KDA_ERR_UNSUPPORTED;
    if (V > MOST_WORDS || T > MOST_ROWS) return KDA_ERR_TOO_LARGE;
    if (T == 0) return KDA_OK;
    if (!logits || !aligned(logits, esize(dt)) || !table_ok(tokens) || !table_ok(logp) || (lse && !aligned(lse, 4)) ||
        (entropy && !aligned(entropy, 4)) || (top > 0 && (!table_ok(top_logp) || !table_ok(top_token))))
        return KDA_ERR_INVALID_ARG;
    unsigned* err = nullptr;
    if (kda::device_error_word(&err) != KDA_OK) return KDA_ERR_CUDA;
    kda::LogprobParams p{};
    p.logits = logits; p.tokens = tokens; p.logp = logp; p.lse = lse; p.entropy = entropy;
    p.top_logp = top_logp; p.top_token = top_token; p.err = err;
    p.row_stride = row_stride; p.T = T; p.V = V; p.top = top;
    return kda::launch_token_logprobs(p, dt, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_token_logprobs_backward(const void* logits, int64_t row_stride, const int32_t* tokens, const float* lse,
                                       const float* entropy, const float* grad_logp, const float* grad_entropy, int32_t T,
                                       int32_t V, kda_dtype dt, void* grad, int64_t grad_stride, void* stream) {
    if (T < 0 || V <= 0 || !known(dt) || row_stride < V || grad_stride < V || (entropy == nullptr) != (grad_entropy == nullptr))
        return KDA_ERR_INVALID_ARG;
    if (V > MOST_WORDS || T > MOST_ROWS || T * kda::logprobs_backward_chunks(V, dt) > INT32_MAX) return KDA_ERR_TOO_LARGE;
    if (T == 0) return KDA_OK;
    if (!logits || !aligned(logits, esize(dt)) || !table_ok(tokens) || !table_ok(lse) || !table_ok(grad_logp) ||
        (entropy && (!aligned(entropy, 4) || !aligned(grad_entropy, 4))) || !grad || !aligned(grad, esize(dt)) ||
        (grad == logits && grad_stride != row_stride))
        return KDA_ERR_INVALID_ARG;
    kda::LogprobGradParams p{};
    p.logits = logits; p.tokens = tokens; p.lse = lse; p.entropy = entropy; p.grad_logp = grad_logp;
    p.grad_entropy = grad_entropy; p.grad = grad; p.row_stride = row_stride; p.grad_stride = grad_stride; p.T = T; p.V = V;
    return kda::launch_token_logprobs_backward(p, dt, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
