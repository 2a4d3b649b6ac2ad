// Internal interfaces of the operators that bring prompts into a hybrid stack and score their tokens (rotary positions,
// new tokens into cache pages, attention of chunks over a paged cache, token log probabilities) between their C-ABI
// host code and their kernels.
#pragma once

#include "kda_serve.cuh"

namespace kda {

// Pairs of fp32 numbers in one 64-bit register, and their operations: two in one instruction.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair_of(float a, float b) {
    Pair d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 both(Pair x) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(x));
    return d;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// t / n for 0 <= t < 2^31 and a divisor that the host knows, as a multiplication.
struct Divisor {
    uint32_t magic;
    int32_t shift;
};
inline Divisor divisor(int32_t n) {
    Divisor d{0u, 0};
    while ((2ll << d.shift) < n) ++d.shift;
    if (n > 1) d.magic = (uint32_t)((1ull << (32 + d.shift)) / n + 1);
    return d;
}
__device__ __forceinline__ int over(int t, const Divisor& d) { return d.magic ? (int)(__umulhi((uint32_t)t, d.magic) >> d.shift) : t; }

// Rotary positions, and tokens into cache pages.  Without `append` a token's position is positions[t] and keys go
// to k_out; with it, a packed batch's tokens go to their places in the pages.  Strides in elements.
struct RotaryParams {
    const void* q;               // token t at q + t * q_stride, [Hq, d]; nullptr with Hq = 0
    const void* k;
    const void* v;               // append only
    const int32_t* positions;    // [T]; rotary only
    const double* inv_freq;      // [rot / 2]
    void* q_out;                 // may be q
    void* k_out;                 // rotary only; may be k
    void* k_pages;               // append only
    void* v_pages;
    const int32_t* table;        // [B, max_pages]; append only
    const int32_t* lens;         // [B], new tokens included
    const int32_t* cu;           // [B + 1]
    unsigned* err;
    int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride, k_page_stride, v_page_stride;
    int32_t B, T, Hq, Hkv, d, rot;
    int32_t num_pages, page_size, max_pages;
    int32_t interleaved;
    int32_t append;              // tokens of a packed batch, into pages
    float scale;                 // of the rotated part
    float sign;                  // -1: turned back (the gradient)
};
cudaError_t launch_rotary(const RotaryParams& p, kda_dtype dt, cudaStream_t s);

// Attention of chunks of new tokens, already in their pages.
struct ChunkParams {
    const void* q;               // [T, Hq, d]
    const void* k_pages;         // page p at k_pages + p * k_stride elements, [Hkv, page_size, d]
    const void* v_pages;
    const int32_t* table;        // [B, max_pages]
    const int32_t* lens;         // [B], new tokens included
    const int32_t* cu;           // [B + 1]
    void* o;                     // [T, Hq, d]
    float* lse;                  // [T, Hq], or nullptr
    unsigned char* workspace;
    unsigned* err;
    int64_t k_stride, v_stride;
    int32_t B, T, Hq, Hkv, d;
    int32_t num_pages, page_size, max_pages;
    int32_t window;              // 0: every token up to the query's own
    int32_t sinks;
    float scale;
};
size_t chunk_workspace(int32_t d, kda_dtype dt);
cudaError_t launch_attention_prefill(const ChunkParams& p, kda_dtype dt, cudaStream_t s);
size_t chunk_tc_workspace(int32_t d);                                       // its tensor-core path
cudaError_t launch_attention_prefill_tc(const ChunkParams& p, cudaStream_t s);

struct LogprobParams {
    const void* logits;          // row r at logits + r * row_stride elements
    const int32_t* tokens;       // [T], -1: none
    float* logp;                 // [T]
    float* lse;                  // [T], or nullptr
    float* entropy;              // [T], or nullptr
    float* top_logp;             // [T, top], or nullptr with top = 0
    int32_t* top_token;          // [T, top]
    unsigned* err;
    int64_t row_stride;
    int32_t T, V, top;
};
cudaError_t launch_token_logprobs(const LogprobParams& p, kda_dtype dt, cudaStream_t s);

struct LogprobGradParams {
    const void* logits;
    const int32_t* tokens;
    const float* lse;            // [T]
    const float* entropy;        // [T], or nullptr
    const float* grad_logp;      // [T]
    const float* grad_entropy;   // [T], or nullptr
    void* grad;                  // row r at grad + r * grad_stride elements; may be logits
    int64_t row_stride, grad_stride;
    int32_t T, V;
};
int64_t logprobs_backward_chunks(int32_t V, kda_dtype dt);    // of a row, wherever it begins; all rows' are numbered in 31 bits
cudaError_t launch_token_logprobs_backward(const LogprobGradParams& p, kda_dtype dt, cudaStream_t s);

}  // namespace kda
