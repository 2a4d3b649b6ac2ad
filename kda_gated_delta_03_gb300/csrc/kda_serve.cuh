// Internal interfaces of the decoding operators of a hybrid stack (attention over a paged cache, beam
// selection, forks of states and cache pages) between their C-ABI host code and their kernels.
#pragma once

#include <atomic>

#include "kda_internal.cuh"

namespace kda {

// The current device's error word (defined with the other entry points' host code).
kda_status device_error_word(unsigned** out);

// The current device's SMs, and a kernel's right to `smem` bytes of dynamic shared memory and to clusters of 16
// CTAs there.  All is asked for once per device: these calls are made for every generated token.  `done` is the
// kernel's own.
struct DeviceSetup {
    std::atomic<int> sms[64] = {};               // 0: not asked yet
};
inline cudaError_t device_setup(DeviceSetup& done, const void* kernel, int smem, int* sms, bool cluster16 = false) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < 64;
    int n = known ? done.sms[dev].load(std::memory_order_acquire) : 0;
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess && smem > 48 * 1024)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess && cluster16)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        if (known) done.sms[dev].store(n, std::memory_order_release);
    }
    *sms = n;
    return cudaSuccess;
}

// Everything the paged attention kernels need, already validated on the host.
struct AttnParams {
    const void* q;               // [B, Hq, d]
    void* k_pages;               // page p at k_pages + p * k_stride elements, [Hkv, page_size, d]
    void* v_pages;
    const int32_t* table;        // [B, max_pages]
    const int32_t* lens;         // [B]
    const void* k_new;           // [B, Hkv, d], or nullptr
    const void* v_new;
    void* o;                     // [B, Hq, d]
    float* lse;                  // [B, Hq], or nullptr
    unsigned char* workspace;
    unsigned* err;
    int64_t k_stride;
    int64_t v_stride;
    int32_t B;
    int32_t Hq;
    int32_t Hkv;
    int32_t d;
    int32_t num_pages;
    int32_t page_size;
    int32_t max_pages;
    int32_t window;              // 0: every token below the length
    int32_t sinks;
    float scale;
    // set by the launcher: t / page_size = umulhi(t, page_magic) >> page_shift for t < 2^31 (page_magic 0: t itself)
    uint32_t page_magic;
    int32_t page_shift;
    int32_t whole;               // set by the launcher: CTA i does all of unit i, and nothing is left to join
};
size_t attn_workspace(int32_t B, int32_t Hq, int32_t Hkv, int32_t d, kda_dtype dt);
cudaError_t launch_attention_decode(const AttnParams& p, kda_dtype dt, cudaStream_t s);

struct BeamParams {
    const void* logits;          // row r at logits + r * row_stride elements
    int64_t row_stride;
    const float* beam_scores;    // [N, K]
    const uint8_t* finished;     // [N, K], or nullptr
    int32_t eos;                 // -1: none
    int32_t N;
    int32_t K;
    int32_t V;
    float* scores;               // [N, K]
    int32_t* parent;
    int32_t* token;
    uint8_t* finished_out;       // or nullptr
    unsigned char* workspace;
};
size_t beam_workspace(int32_t N, int32_t K, int32_t V, kda_dtype dt);
cudaError_t launch_beam_select(const BeamParams& p, kda_dtype dt, cudaStream_t s);

// The pools of one call, passed to kernels by value.
struct PoolSet {
    kda_pool pool[KDA_MAX_POOLS];
    int32_t n;
};
cudaError_t launch_copy_pages(const PoolSet& pools, const int32_t* src, const int32_t* dst, int32_t n, unsigned* err,
                              cudaStream_t s);
cudaError_t launch_state_fork(const PoolSet& pools, const int32_t* state_idx, const int32_t* parent, int32_t B,
                              int32_t* state_idx_out, unsigned* err, cudaStream_t s);

struct ForkParams {
    const int32_t* table;        // [rows_in, max_pages]
    const int32_t* lens;         // [rows_in]
    const int32_t* parent;       // [rows_out]
    const int32_t* grow;         // [rows_out], or nullptr
    const int32_t* ref;          // [num_pages]
    int32_t* table_out;          // [rows_out, max_pages]
    int32_t* lens_out;           // [rows_out]
    int32_t* ref_out;            // [num_pages], may be ref
    int32_t* copy_src;           // [rows_out], or nullptr
    int32_t* copy_dst;
    unsigned* err;
    int32_t rows_in;
    int32_t rows_out;
    int32_t max_pages;
    int32_t page_size;
    int32_t num_pages;
};
size_t cache_fork_workspace(int32_t rows_out, int32_t num_pages);
cudaError_t launch_cache_fork(const ForkParams& p, const PoolSet& pools, void* workspace, cudaStream_t s);

struct CompactParams {
    const int32_t* table;        // [rows * max_pages]
    const int32_t* ref;
    int32_t* table_out;          // may be table
    int32_t* ref_out;            // may be ref
    int32_t* page_map;
    int64_t entries;             // rows * max_pages
    int32_t num_pages;
};
size_t cache_compact_workspace(int32_t num_pages);
cudaError_t launch_cache_compact(const CompactParams& p, const PoolSet& pools, void* workspace, unsigned* err,
                                 cudaStream_t s);

}  // namespace kda
