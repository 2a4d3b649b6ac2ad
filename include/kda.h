/*
 * kda.h -- C ABI of libkda, a single-GPU (sm_103a) implementation of the Kimi
 * Delta Attention (KDA) operator.
 *
 * The operator ("Kimi K3, explained", section "The math", and section "How
 * Kimi Delta Attention works, step by step"): per head a fixed state S is
 * decayed channel by channel, the delta rule erases what S returns for the key
 * and writes the new value, and the query reads the result.  The page writes S
 * as d_v x d_k with o_t = S_t q_t; this library stores the transpose,
 * S[d_k][d_v] (d_v contiguous), so that
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *     o_t = scale * S_t^T q_t
 *
 * which is the same operator.  alpha_t in (0,1]^{d_k} is the per-channel decay
 * (one value per key channel, which is what KDA adds over Gated DeltaNet),
 * beta_t in [0,1] the write strength.  q and k are expected L2-normalised by the
 * caller; the library does not renormalise.
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers to contiguous row-major arrays,
 *    owned by the caller.  The library never allocates, frees or retains them,
 *    and keeps no state between calls except one 32-bit error word per device
 *    (a static device variable, see kda_get_device_error).
 *  - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL = the
 *    legacy default stream) on the current device.  Arguments are validated on
 *    the host before anything is launched; a validation failure launches
 *    nothing and returns the status.  Conditions only visible on the device
 *    (inconsistent cu_seqlens contents, out-of-range state slots) make the
 *    kernels skip the affected work and set bits of the device error word.
 *  - Alignment: q, k, v, o, alpha, states 16 bytes; beta, cu_seqlens,
 *    state_idx 4 bytes; workspace 256 bytes.
 *  - dtype (kda_dtype) applies to q, k, v and o.  beta, alpha and the states
 *    are always float32.
 *  - Supported sizes: d_k == d_v in {16, 64, 128}.  Other sizes return
 *    KDA_ERR_UNSUPPORTED.
 *  - Numerics: log2(alpha) is clamped below at -15 per token (alpha >= 2^-15
 *    ~= 3.1e-5 per token and channel); smaller alphas, including alpha = 0,
 *    decay as if alpha were 2^-15.  Intermediates are float32 (bf16 tensor-core
 *    operands only for the raw bf16 q, k, v).
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define KDA_API __attribute__((visibility("default")))
#else
#define KDA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,  /* null/misaligned pointer, negative size, bad scale        */
    KDA_ERR_UNSUPPORTED = 2,  /* head size or dtype this build has no kernel for           */
    KDA_ERR_WORKSPACE = 3,    /* workspace missing or smaller than the required size       */
    KDA_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed                      */
    KDA_ERR_DEVICE = 5,       /* kda_get_device_error found device-detected errors         */
    KDA_ERR_TOO_LARGE = 6     /* problem exceeds the fixed scratch of kda_prefill_noalloc, or a
                                 limit on rows or words stated with the function            */
} kda_status;

typedef enum { KDA_DTYPE_F32 = 0, KDA_DTYPE_BF16 = 1 } kda_dtype;

/*
 * Layout of alpha (the forget gate).  "Kimi K3, explained", section "The math":
 * with every alpha equal to 1 the update is DeltaNet's delta rule, with one
 * alpha per head it is Gated DeltaNet, and KDA gives every key channel its own.
 */
typedef enum {
    KDA_ALPHA_PER_CHANNEL = 0,  /* KDA: alpha [tokens, H, d_k] float32, 16-byte aligned       */
    KDA_ALPHA_PER_HEAD = 1,     /* Gated DeltaNet: alpha [tokens, H] float32, 4-byte aligned */
    KDA_ALPHA_NONE = 2          /* DeltaNet: no decay; alpha is not read and may be NULL     */
} kda_alpha_mode;

/* Bits of the device error word. */
#define KDA_DEVERR_CU_SEQLENS 0x1u  /* cu_seqlens not monotone / cu[0] != 0 / cu[N] != total  */
#define KDA_DEVERR_STATE_IDX 0x2u   /* decode state_idx entry outside [0, num_slots)          */
#define KDA_DEVERR_TIMEOUT 0x4u     /* a bounded wait inside a kernel gave up (work abandoned) */
#define KDA_DEVERR_SNAPSHOTS 0x8u   /* snapshot_offsets disagree with the sequence lengths       */
#define KDA_DEVERR_RANGE 0x10u      /* one-sequence bf16 d=128 prefill: a key-side chunk product
                                       (Q', M, T' below) beyond fp16's range (|x| > 65504), which
                                       needs keys far from unit norm; results invalid */
#define KDA_DEVERR_PAGES 0x20u      /* a page number outside the pool, or a length the table cannot hold */
#define KDA_DEVERR_EXHAUSTED 0x40u  /* kda_cache_fork: fewer free pages than the new rows need  */
#define KDA_DEVERR_PARENT 0x80u     /* a parent outside [-1, rows)                              */
#define KDA_DEVERR_TOKEN 0x100u     /* a token outside [-1, V)                                  */

/*
 * Bytes of device workspace kda_prefill needs for this problem (0 is a valid
 * answer).  Pure host function; never fails (returns 0 for invalid sizes).
 *  - bf16 with d_k = d_v = 128 (the two-phase path): the per-chunk records
 *    (99,072 bytes per chunk and head; up to 1 GiB of them for one sequence,
 *    up to 16 GiB for several, so that all chunks of a batch of sequences fit
 *    one window), preceded, for several sequences, by their chunk offsets and
 *    their longest-first order (4 (N + 1) and 4 N bytes, each rounded up to
 *    256).  kda_prefill also accepts less, down to one chunk's records after
 *    those offsets; it then walks the chunks in more windows, with identical
 *    results.
 *  - Other several-sequence calls: the longest-first schedule, 4 bytes per
 *    sequence.
 */
KDA_API size_t kda_prefill_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t d_k,
                                  int32_t d_v, kda_dtype dt);

/*
 * Number of kernel launches a kda_prefill call with these arguments makes on the
 * current device (diagnostics: launch budgets, profiler capture ranges), or -1
 * for arguments kda_prefill would reject on the host.  The two-phase path makes
 * two launches per window of chunks (plus two for the chunk offsets and the
 * order of several sequences), and its window count depends on
 * workspace_bytes and on the device's SM count.  Calls cudaGetDevice and
 * cudaDeviceGetAttribute; enqueues nothing.
 */
KDA_API int64_t kda_prefill_launch_count(int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t d_k,
                                         int32_t d_v, kda_dtype dt, size_t workspace_bytes);

/*
 * Chunkwise-parallel prefill over packed variable-length sequences, with state
 * in and state out ("Kimi K3, explained", section "Training in chunks": the
 * sequence is split into chunks, the per-token decay-and-erase products inside
 * a chunk are rewritten in WY form so most of the work becomes matrix
 * products, and only the state is carried from chunk to chunk).  Results equal
 * the token-by-token recurrence above up to rounding.  Append-prefill (the
 * agentic workload of the hex-index review, where new context continues a long
 * history) is this call with state_in set to an earlier call's state_out.
 *
 *   q, k        [total_tokens, H, d_k]  dtype dt
 *   v           [total_tokens, H, d_v]  dtype dt
 *   beta        [total_tokens, H]       float32, write strength in [0,1]
 *   alpha       [total_tokens, H, d_k]  float32, per-channel decay in (0,1]
 *   cu_seqlens  [num_seqs + 1]          int32 device array, cu[0] = 0,
 *               non-decreasing, cu[num_seqs] = total_tokens; sequence n owns
 *               tokens [cu[n], cu[n+1]).  Zero-length sequences are allowed:
 *               their state_out is their state_in (or zero).
 *   state_in    [num_seqs, H, d_k, d_v] float32, or NULL for zero states
 *   state_out   [num_seqs, H, d_k, d_v] float32 (may equal state_in, in place)
 *   o           [total_tokens, H, d_v]  dtype dt, o_t = scale * S_t^T q_t
 *   workspace   device scratch of at least kda_prefill_workspace_size(...)
 *               bytes (may be NULL when that size is 0); contents need not be
 *               initialised and are clobbered.
 * Returns KDA_OK once the work is enqueued.  Bad cu_seqlens contents are
 * reported through the device error word (KDA_DEVERR_CU_SEQLENS); the
 * sequences they affect are skipped.
 */
KDA_API kda_status kda_prefill(const void* q, const void* k, const void* v, const float* beta,
                       const float* alpha, const int32_t* cu_seqlens, int32_t num_seqs,
                       int64_t total_tokens, int32_t H, int32_t d_k, int32_t d_v, kda_dtype dt,
                       float scale, const float* state_in, float* state_out, void* o,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * Options of kda_prefill_ex.  Zero-initialise and set what is used.
 *
 * alpha_mode selects the layout of `alpha` (kda_alpha_mode): per key channel
 * (KDA, the default), one value per token and head (Gated DeltaNet: 4 bytes per
 * token-head instead of 4 * d_k), or none (DeltaNet).
 *
 * State snapshots ("Kimi K3 changed the memory math for agentic AI forever",
 * section "But KDA State Is Not Additive": the recurrent state depends on the
 * whole prefix, so restartable checkpoints and prefix reuse keep copies of it
 * at fixed token intervals): with snapshot_every > 0, the state of sequence n after its
 * first (m + 1) * snapshot_every tokens is written to
 * snapshots[snapshot_offsets[n] + m] for m = 0 .. floor(len_n /
 * snapshot_every) - 1 (a snapshot at len_n equals that sequence's
 * state_out).
 *
 * single_kernel (nonzero): bf16 sequences with d_k = d_v = 128 run the
 * single-kernel tensor-core path (TF32 / bf16 operands, one CTA per sequence,
 * head and value slice; the workspace then needs only the longest-first order
 * of several sequences) instead of the two-phase path, whose per-chunk records
 * and state operand are fp16.  The
 * two-phase path keeps values and states of any magnitude inside fp16's range
 * with exact power-of-two scales (per chunk for v, per chunk and slice for the
 * state); only key-side products far outside O(1), which need keys far from
 * unit norm, set KDA_DEVERR_RANGE, and this option is then the way out.  Results
 * agree to the same tolerance; the two-phase path is faster.
 *   snapshot_every    tokens between snapshots: 0, or a positive multiple of 64
 *   snapshots         [snapshot_offsets[num_seqs], H, d_k, d_v] float32 device
 *                     buffer, 16-byte aligned
 *   snapshot_offsets  [num_seqs + 1] int32 device array, non-decreasing, with
 *                     snapshot_offsets[n + 1] - snapshot_offsets[n] =
 *                     floor(len_n / snapshot_every); a sequence whose count
 *                     disagrees gets no snapshots and sets
 *                     KDA_DEVERR_SNAPSHOTS.
 */
typedef struct kda_prefill_options {
    int32_t snapshot_every;
    float* snapshots;
    const int32_t* snapshot_offsets;
    int32_t alpha_mode;             /* kda_alpha_mode; 0 = KDA_ALPHA_PER_CHANNEL */
    int32_t single_kernel;          /* nonzero: see below */
} kda_prefill_options;

/*
 * kda_prefill with options (NULL options = kda_prefill).  Snapshots add only
 * their own writes (64 KiB per snapshot and head at d = 128); outputs and
 * state_out are those of kda_prefill.
 */
KDA_API kda_status kda_prefill_ex(const void* q, const void* k, const void* v, const float* beta,
                          const float* alpha, const int32_t* cu_seqlens, int32_t num_seqs,
                          int64_t total_tokens, int32_t H, int32_t d_k, int32_t d_v, kda_dtype dt,
                          float scale, const float* state_in, float* state_out, void* o,
                          void* workspace, size_t workspace_bytes, void* stream,
                          const kda_prefill_options* options);

/*
 * Backward pass of kda_prefill (per-channel alpha): given the gradients grad_o
 * of the outputs and grad_state_out of the final states (NULL = zero),
 * computes the gradients of q, k, v, beta, alpha and state_in for the loss
 * sum(o * grad_o) + sum(state_out * grad_state_out).  It is the reverse mode of
 * the token recurrence ("Kimi K3, explained", section "The math"), in three
 * passes: a forward recompute that stores the state at every 64-token
 * boundary; a reverse chain that carries only the state gradient and stores it
 * at the same boundaries (for one bf16 d=128 sequence whose recompute fits one
 * window of records, chunk by chunk from those records: dS_start =
 * Diag(Gamma_C) dS_end - M^T dS_end + Q'^T dO; otherwise token by token); and a
 * chunk-parallel pass that, per (sequence, 64-token chunk, head), takes every
 * gradient of the chunk from its start state and its end-state gradient: at
 * d = 128 in matrix form, the chunk's products of "Training in chunks" run in
 * reverse (on TF32 tensor cores for bf16 inputs, in fp32 for fp32 inputs), at
 * d = 16 and 64 by replaying the chunk and walking it back token by token.
 * Arguments are kda_prefill's, plus:
 *   grad_o          [total_tokens, H, d_v] dtype dt
 *   grad_state_out  [num_seqs, H, d_k, d_v] float32, or NULL
 *   grad_q, grad_k  [total_tokens, H, d_k] dtype dt;  grad_v [total_tokens, H, d_v]
 *   grad_beta       [total_tokens, H] float32;  grad_alpha [total_tokens, H, d_k]
 *   grad_state_in   [num_seqs, H, d_k, d_v] float32, or NULL (not computed)
 *   workspace       at least kda_prefill_backward_workspace_size(...) bytes
 * The decay clamp of the forward (log2 alpha >= -15 per token) is not
 * differentiated: the d = 16 and 64 walk uses alpha as given, the d = 128
 * chunk form the clamped decays inside a chunk (as the forward does), and
 * both give the gradient of alpha itself.
 */
KDA_API size_t kda_prefill_backward_workspace_size(int32_t num_seqs, int64_t total_tokens, int32_t H,
                                           int32_t d_k, int32_t d_v, kda_dtype dt);
KDA_API kda_status kda_prefill_backward(const void* q, const void* k, const void* v, const float* beta,
                                const float* alpha, const int32_t* cu_seqlens, int32_t num_seqs,
                                int64_t total_tokens, int32_t H, int32_t d_k, int32_t d_v, kda_dtype dt,
                                float scale, const float* state_in, const void* grad_o,
                                const float* grad_state_out, void* grad_q, void* grad_k, void* grad_v,
                                float* grad_beta, float* grad_alpha, float* grad_state_in, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * One fused decode step for B sequences, each with H resident states
 * ("Kimi K3, explained", section "How Kimi Delta Attention works, step by
 * step", and the question on constant-cost decode: one fixed-size state update
 * and read per generated token, independent of context length).  Each state is
 * read once, decayed, delta-corrected, written back in place, and queried.
 *
 *   q, k        [B, H, d_k]  dtype dt;  v [B, H, d_v] dtype dt
 *   beta        [B, H] float32;  alpha [B, H, d_k] float32
 *   state       [num_slots, H, d_k, d_v] float32 pool, updated in place
 *   state_idx   [B] int32 device array: row b uses slot state_idx[b]; NULL
 *               means slot b (then num_slots >= B).  Slots must be distinct
 *               within one call.  Out-of-range entries skip the row and set
 *               KDA_DEVERR_STATE_IDX.
 *   o           [B, H, d_v] dtype dt
 */
KDA_API kda_status kda_decode_step(const void* q, const void* k, const void* v, const float* beta,
                           const float* alpha, float* state, const int32_t* state_idx,
                           int32_t num_slots, void* o, int32_t B, int32_t H, int32_t d_k,
                           int32_t d_v, kda_dtype dt, float scale, void* stream);

/*
 * kda_decode_step on a state pool stored in bf16 ([num_slots, H, d_k, d_v]
 * bf16, updated in place): each state is read as bf16, updated in float32 and
 * written back rounded to nearest-even bf16.  The pages size the recurrent
 * state at 2 bytes per element ("Kimi K3 changed the memory math for agentic
 * AI forever", section "Linear Attention's Promise"), which halves the decode
 * step's state traffic.  Every other argument, result and error is kda_decode_step's.  The
 * state carries bf16 rounding from step to step, so results agree with the
 * float32-state step only to bf16 precision.
 */
KDA_API kda_status kda_decode_step_bf16_state(const void* q, const void* k, const void* v, const float* beta,
                                      const float* alpha, void* state, const int32_t* state_idx,
                                      int32_t num_slots, void* o, int32_t B, int32_t H, int32_t d_k,
                                      int32_t d_v, kda_dtype dt, float scale, void* stream);

/*
 * Options of kda_decode_step_ex.  Zero-initialise and set what is used.
 *   alpha_mode   kda_alpha_mode: layout of alpha ([B, H, d_k], [B, H], or not read)
 *   state_dtype  KDA_DTYPE_F32 (default) or KDA_DTYPE_BF16 (the pool is bf16, as
 *                kda_decode_step_bf16_state)
 */
typedef struct kda_decode_options {
    int32_t alpha_mode;
    int32_t state_dtype;
} kda_decode_options;

/* kda_decode_step with options (NULL options = kda_decode_step); `state` is float32 or bf16. */
KDA_API kda_status kda_decode_step_ex(const void* q, const void* k, const void* v, const float* beta,
                              const float* alpha, void* state, const int32_t* state_idx, int32_t num_slots,
                              void* o, int32_t B, int32_t H, int32_t d_k, int32_t d_v, kda_dtype dt,
                              float scale, void* stream, const kda_decode_options* options);

/*
 * kda_prefill without a workspace argument, for callers that cannot allocate
 * device memory.  (The pages have no counterpart; this is an interface
 * convenience.)  Typical callers: a serving process whose memory manager has
 * reserved the GPU's memory up front and hands out no scratch buffers, or a
 * host program that reaches this library only through the C ABI and has no
 * device allocator of its own.  Arguments, results and errors are those of
 * kda_prefill, except:
 *  - bf16 d = 128 runs the single-kernel chunkwise path (kda_prefill's
 *    two-phase path needs its workspace for per-chunk records), as
 *    kda_prefill_ex with single_kernel set; results agree with kda_prefill
 *    within rounding.
 *  - The scratch kda_prefill takes as `workspace` for several sequences (their
 *    longest-first order) lives in a fixed static device array of
 *    KDA_NOALLOC_MAX_SEQS int32 entries (64 KiB), which every GPU that loads
 *    libkda holds until the process exits.  num_seqs > KDA_NOALLOC_MAX_SEQS
 *    returns KDA_ERR_TOO_LARGE before anything is launched.
 *  - The function allocates and frees nothing.  The first call on a device
 *    looks up the array's device address (cudaGetSymbolAddress, with that
 *    device current) and caches it; make that first call on each device before
 *    any stream capture.
 *  - Every call shares the one array, which keeps the last call's contents;
 *    each call rewrites every entry it reads, so nothing needs clearing.  Calls
 *    whose work overlaps on the GPU (for example on two unordered streams)
 *    race on the array and must be serialised by the caller.
 */
#define KDA_NOALLOC_MAX_SEQS 16384
KDA_API kda_status kda_prefill_noalloc(const void* q, const void* k, const void* v, const float* beta,
                                       const float* alpha, const int32_t* cu_seqlens, int32_t num_seqs,
                                       int64_t total_tokens, int32_t H, int32_t d_k, int32_t d_v,
                                       kda_dtype dt, float scale, const float* state_in,
                                       float* state_out, void* o, void* stream);

/*
 * kda_prefill with q, k, v, beta, alpha, cu_seqlens, state_in, state_out and o
 * in HOST memory (same shapes and dtypes as kda_prefill; alpha per key
 * channel).  The inputs cross to the device segment by segment on an internal
 * copy stream while earlier segments compute on `stream`, and each segment's o
 * (and its sequences' final states) cross back on a second internal stream as
 * soon as they are ready, so the transfers and the compute overlap.  One
 * sequence is cut at multiples of 64 tokens with its state carried between
 * segments (the same chunks as one kda_prefill call, so the same results);
 * several sequences are grouped at sequence boundaries.
 *
 *   cu_seqlens       host [num_seqs + 1]: cu[0] = 0, non-decreasing,
 *                    cu[num_seqs] = total_tokens (checked here, on the host)
 *   state_in         host [num_seqs, H, d_k, d_v] float32, or NULL (zeros)
 *   state_out, o     host outputs, written when `stream` completes
 *   device_buffer    device memory of at least
 *                    kda_prefill_host_buffer_size(...) bytes, 256-byte aligned,
 *                    caller-owned: device copies of inputs and outputs and
 *                    the prefill's workspace.  Reuse it only on `stream`.
 *
 * Asynchronous on `stream`: every host buffer must stay valid and unchanged
 * until `stream` completes.  Pinned (page-locked) host memory is needed for
 * the copies to overlap; pageable memory works but serialises them.  Returns
 * KDA_ERR_INVALID_ARG / KDA_ERR_UNSUPPORTED / KDA_ERR_WORKSPACE before any
 * copy or launch, KDA_ERR_CUDA if a CUDA call fails.  As for kda_prefill, the
 * "Kimi K3, explained" section "The math" defines what is computed.
 */
KDA_API size_t kda_prefill_host_buffer_size(int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t d_k,
                                            int32_t d_v, kda_dtype dt);
KDA_API kda_status kda_prefill_host(const void* q, const void* k, const void* v, const float* beta,
                                    const float* alpha, const int32_t* cu_seqlens, int32_t num_seqs,
                                    int64_t total_tokens, int32_t H, int32_t d_k, int32_t d_v, kda_dtype dt,
                                    float scale, const float* state_in, float* state_out, void* o,
                                    void* device_buffer, size_t device_buffer_bytes, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Decoding a hybrid stack.  The pages interleave KDA layers with full-attention layers ("Kimi K3 changed
 * the memory math for agentic AI forever": recurrent states for the former, a paged key-value cache for
 * the latter).  The functions below are what such a decode loop needs next to kda_decode_step: attention
 * of the new token over the paged cache, a beam search's selection, and the bookkeeping that gives every
 * chosen beam its states and its pages.  All of it stays on the device, so that a whole step can be
 * captured in a CUDA graph.
 *
 * A page pool holds num_pages pages of page_size tokens; a page's keys (or values) are [H_kv][page_size][d],
 * contiguous.  Row b of a block table, block_table[b][0 .. max_pages), names the pages that hold tokens
 * 0 .. page_size - 1, page_size .. 2 page_size - 1, ... of sequence b; entries past its last page are -1.
 * ------------------------------------------------------------------------------------------------ */

/*
 * Attention of one new token per sequence over a paged key-value cache:
 *
 *     s_t = scale * q . k_t,   o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m)
 *
 * over the visible tokens t of its row: t < seq_lens[b], and with window > 0 also t >= seq_lens[b] -
 * window or t < sinks (a sliding window behind a few first tokens that stay visible).  Query head h reads
 * key-value head h / (H_q / H_kv).  A row with no visible token gives o = 0 and lse = -inf.  What lies in
 * the pools past a row's end is never used, whatever it holds; a visible value that is not finite makes its
 * column of o not finite (in bf16 a NaN, also where the sum would be an infinity).
 *
 *   q            [B, H_q, d]   dtype dt
 *   k_pages      num_pages pages of [H_kv, page_size, d], dtype dt, page p at k_pages + p * k_page_stride
 *   v_pages      likewise, at v_pages + p * v_page_stride (strides in elements)
 *   block_table  [B, max_pages] int32;  seq_lens [B] int32, the new token included
 *   k_new, v_new [B, H_kv, d] dtype dt, or both NULL: the new token's key and value, which the call
 *                stores at position seq_lens[b] - 1 and attends to.  That position's page must belong
 *                to row b alone.  NULL: the cache holds them already.
 *   o            [B, H_q, d] dtype dt;  lse [B, H_q] float32 or NULL: m + log sum exp(s_t - m)
 *   workspace    kda_attention_decode_workspace_size(...) bytes: partial results of rows whose length is
 *                split over several CTAs, joined in a fixed order (two calls give the same bits)
 * Sizes: d in {16, 64, 128}; H_q a multiple of H_kv; any page_size >= 1; max_pages * page_size and B at most
 * 2^31 - 1024, H_q * d below 2^31.  Alignment: q, k_new, v_new, o and the pools 16 bytes, page strides multiples of 16 bytes.
 * A length outside [0, max_pages * page_size] counts as 0, and a page outside [0, num_pages) as page 0 where it
 * is read; a new token whose page is outside is attended to, but not stored.  All set KDA_DEVERR_PAGES.
 */
KDA_API size_t kda_attention_decode_workspace_size(int32_t B, int32_t H_q, int32_t H_kv, int32_t d, kda_dtype dt);
KDA_API kda_status kda_attention_decode(const void* q, void* k_pages, void* v_pages, const int32_t* block_table,
                                        const int32_t* seq_lens, const void* k_new, const void* v_new, int32_t B,
                                        int32_t H_q, int32_t H_kv, int32_t d, int32_t num_pages, int32_t page_size,
                                        int32_t max_pages, int64_t k_page_stride, int64_t v_page_stride, kda_dtype dt,
                                        float scale, int32_t window, int32_t sinks, void* o, float* lse,
                                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * A beam search's selection: for each of N groups, the K best of its K x V continuations
 *
 *     s(b, v) = beam_scores[b] + (x_bv - lse_b),   lse_b = m + log sum_v exp(x_bv - m),  m = max_v x_bv
 *
 * in float32, by score, the lowest b * V + v first among equal scores.  A score that is not a number
 * (a logit row with a NaN or +inf, or with nothing above -inf) counts as -inf.  A finished beam offers one
 * continuation, eos_token at its unchanged score; its other words count as -inf.
 *
 *   logits       [N * K, V] dtype dt, row r at logits + r * row_stride (elements, >= V)
 *   beam_scores  [N, K] float32;  finished [N, K] bytes, nonzero = finished, or NULL
 *   eos_token    in [0, V), or -1: none (then finished must be NULL)
 *   scores       [N, K] float32, best first (may be beam_scores, in place)
 *   parent       [N, K] int32: the row n * K + b that the new beam continues
 *   token        [N, K] int32;  finished_out [N, K] bytes (token == eos_token or parent finished), or NULL
 *                (may be finished, in place)
 *   workspace    kda_beam_select_workspace_size(...) bytes
 * K <= KDA_BEAM_MAX_K; V at most 2^31 - 2^14, K * V and N * K below 2^31 (KDA_ERR_TOO_LARGE above).
 */
#define KDA_BEAM_MAX_K 32
KDA_API size_t kda_beam_select_workspace_size(int32_t N, int32_t K, int32_t V, kda_dtype dt);
KDA_API kda_status kda_beam_select(const void* logits, int64_t row_stride, const float* beam_scores,
                                   const uint8_t* finished, int32_t eos_token, int32_t N, int32_t K, int32_t V,
                                   kda_dtype dt, float* scores, int32_t* parent, int32_t* token,
                                   uint8_t* finished_out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * A pool of equal slots (resident KDA states, or pages of a cache) on one or several layers: slot s of
 * layer l is the slot_bytes bytes at data + l * layer_stride + s * slot_stride.  Strides and slot_bytes
 * in bytes, multiples of 16; data 16-byte aligned.  A call takes at most KDA_MAX_POOLS pools.
 */
typedef struct kda_pool {
    void* data;
    int64_t layer_stride;
    int64_t slot_stride;
    int64_t slot_bytes;
    int32_t layers;
    int32_t slots;
} kda_pool;
#define KDA_MAX_POOLS 8

/*
 * Copies slots within pools: for i < n, slot src[i] to slot dst[i], on every layer of every pool.
 * src NULL means src[i] = i.  Entries with src or dst negative, or equal, are skipped; one outside a
 * pool is skipped and sets KDA_DEVERR_PAGES.  No dst may occur twice or be another entry's src.
 */
KDA_API kda_status kda_copy_pages(const kda_pool* pools, int32_t num_pools, const int32_t* src, const int32_t* dst,
                                  int32_t n, void* stream);

/*
 * Gives the B rows of a decode batch the KDA states of the rows that they continue: new row i continues
 * row parent[i] (-1: none, a row that starts anew).  The lowest row with a given parent takes over its
 * parent's slot in place; the r-th of the other continuing rows gets the r-th slot (by row) of the rows
 * that nobody continues, and the state is copied there; rows without a parent get the slots that are then
 * left, contents unchanged.  So state_idx_out is a permutation of state_idx, a copy's target is never
 * read, and only states that have to move are moved.
 *   state_idx [B] int32 (distinct slots);  parent [B] int32;  state_idx_out [B] int32, another array
 * B <= KDA_FORK_MAX_ROWS (KDA_ERR_TOO_LARGE above).  A parent outside [-1, B) counts as -1 and sets
 * KDA_DEVERR_PARENT; a copy from or to a slot outside a pool is skipped and sets KDA_DEVERR_STATE_IDX.
 */
#define KDA_FORK_MAX_ROWS 8192
KDA_API kda_status kda_state_fork(const kda_pool* pools, int32_t num_pools, const int32_t* state_idx,
                                  const int32_t* parent, int32_t B, int32_t* state_idx_out, void* stream);

/*
 * Replaces the rows of a block table: new row i continues old row parent[i] (-1: an empty row) and gets
 * room for grow[i] more tokens.  This forks, reorders, frees, starts and extends rows in one call:
 *  - Whole pages are shared: the new row names its parent's pages, and ref_count says how many rows name a
 *    page.  Every old row gives up its pages; a page that nobody names any more is free (count 0).
 *  - A partly filled last page stays with the lowest row that continues its parent; every other one gets a
 *    page of its own, into which the page is copied on every layer of the pools.
 *  - Pages of its own come from the free ones, the lowest first, handed out by new row and then by
 *    position.
 * seq_lens_out[i] = seq_lens[parent[i]] + grow[i].  When the free pages run out, the entries without a page
 * are -1, the row ends before the first of them, and KDA_DEVERR_EXHAUSTED is set (such a row has no place for
 * the tokens that it lacks: a new one is not to be stored at its last place); a length outside
 * [0, max_pages * page_size], a negative grow or one that the table cannot hold, or a page outside the pool
 * is clamped (to an empty row, no growth, the table's end; no page) and sets KDA_DEVERR_PAGES.
 *   block_table     [rows_in, max_pages];  seq_lens [rows_in];  parent, grow [rows_out], grow may be NULL (0)
 *   ref_count       [num_pages];  ref_count_out [num_pages], may be ref_count (in place)
 *   block_table_out [rows_out, max_pages] and seq_lens_out [rows_out]: other arrays than the input's
 *   copy_src, copy_dst [rows_out] or NULL: the page copied for row i and where to, -1 for none (for pools
 *                   that this call does not get: kda_copy_pages takes them)
 *   pools           pools of num_pages slots; num_pools may be 0
 * All tables int32 on the device.  rows_in and rows_out at most KDA_FORK_MAX_ROWS (KDA_ERR_TOO_LARGE above);
 * max_pages * page_size and a table's entries below 2^31, max_pages at most 2^31 - 1024, num_pages at most
 * 2^31 - 2^18.
 */
KDA_API size_t kda_cache_fork_workspace_size(int32_t rows_in, int32_t rows_out, int32_t max_pages, int32_t num_pages);
KDA_API kda_status kda_cache_fork(const int32_t* block_table, const int32_t* seq_lens, int32_t rows_in,
                                  const int32_t* parent, const int32_t* grow, int32_t rows_out, int32_t max_pages,
                                  int32_t page_size, const int32_t* ref_count, int32_t num_pages,
                                  int32_t* block_table_out, int32_t* seq_lens_out, int32_t* ref_count_out,
                                  int32_t* copy_src, int32_t* copy_dst, const kda_pool* pools, int32_t num_pools,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * Moves the live pages (ref_count > 0) of a cache together at the low end of its pools: with n live pages,
 * the live ones at n and above go, in ascending order, to the free ones below n.  page_map [num_pages]
 * receives each page's new number, -1 for a free page; block_table_out [rows, max_pages] is block_table
 * with every entry replaced by its new number (entries outside [0, num_pages) become -1), ref_count_out the
 * counts at the new numbers.  block_table_out may be block_table, ref_count_out may be ref_count.  Other
 * tables and pools of the same pages follow with page_map (kda_copy_pages with src NULL and dst page_map).
 * num_pages at most 2^31 - 2^18, rows * max_pages below 2^31.
 */
KDA_API size_t kda_cache_compact_workspace_size(int32_t num_pages);
KDA_API kda_status kda_cache_compact(const int32_t* block_table, int32_t rows, int32_t max_pages,
                                     const int32_t* ref_count, int32_t num_pages, int32_t* block_table_out,
                                     int32_t* ref_count_out, int32_t* page_map, const kda_pool* pools,
                                     int32_t num_pools, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------------------
 * A prompt's way through a hybrid stack's full-attention layers, and the scores of its tokens.  New tokens of
 * several sequences lie packed one after the other, as kda_prefill takes them: sequence b has tokens
 * cu_seqlens[b] .. cu_seqlens[b + 1] - 1, at positions seq_lens[b] - n_b .. seq_lens[b] - 1 of its cache (n_b of
 * them, seq_lens[b] with the new ones, as kda_cache_fork returns it for grow = n_b).  A chunk may be a whole
 * prompt, a part of one behind what the cache holds already, or one token.  cu_seqlens[0] = 0; cu_seqlens[B] may be
 * less than T, and outputs of the tokens behind it are left as they were.  A sequence whose borders are not
 * 0 <= cu_seqlens[b] <= cu_seqlens[b + 1] <= T counts as empty and sets KDA_DEVERR_CU_SEQLENS (where borders fall, or the
 * first is not 0, a token that lies between those of two sequences goes to either, and tokens of others may be left out).
 * ------------------------------------------------------------------------------------------------ */

#define KDA_ROTARY_HALF 0         /* pairs (x_i, x_{i + rotary_dim / 2}) */
#define KDA_ROTARY_INTERLEAVED 1  /* pairs (x_2i, x_{2i + 1})            */

/*
 * Rotary positions: in the first rotary_dim places of every head of q and k, pair i of token t becomes
 *
 *     rotary_scale * (a cos - b sin, b cos + a sin),   angle = positions[t] * inv_freq[i]
 *
 * and the rest of the head is copied.  inverse != 0 turns by minus the angle, with the same scale: the gradient
 * of the outputs becomes that of the inputs.  Angles are exact to 2^-25 of a radian for every 32-bit position.
 *
 *   q, q_out   [T, H_q, d] dtype dt, token t at q + t * q_stride (elements); likewise k, k_out with H_kv heads.
 *              k NULL: only q.  q_out may be q and k_out may be k, with the same strides; no other overlap.
 *   positions  [T] int32;  inv_freq [rotary_dim / 2] float64, finite, radians a position (how long contexts
 *              stretch them is the caller's choice), NULL with rotary_dim = 0
 * Sizes: d in {16, 64, 128}; rotary_dim even, 0 .. d; H_q * d and H_kv * d at most a token's stride, all of a
 * token's elements below 2^30.  Alignment: an element; 16 bytes, with strides to match, is the fast way.
 */
KDA_API kda_status kda_rotary(const void* q, const void* k, const int32_t* positions, const double* inv_freq,
                              int32_t T, int32_t H_q, int32_t H_kv, int32_t d, int32_t rotary_dim, int64_t q_stride,
                              int64_t k_stride, kda_dtype dt, int32_t layout, float rotary_scale, int32_t inverse,
                              void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream);

/*
 * Stores a packed batch's new keys and values into their pages, keys rotated by their positions in the cache on
 * the way (rotary_dim = 0: as they are).  Queries, if given, are rotated likewise into q_out.
 *   q        NULL, or [T, H_q, d] at q + t * q_stride, and q_out [T, H_q, d] (may be q, with the same stride)
 *   k, v     [T, H_kv, d] dtype dt at k + t * k_stride, v + t * v_stride
 *   k_pages, v_pages, block_table [B, max_pages], seq_lens [B]  as for kda_attention_decode
 *   cu_seqlens [B + 1] int32;  inv_freq, layout, rotary_scale  as for kda_rotary
 * No two new tokens may have the same place, and k, v may not overlap the pools.  A token without a place (a length
 * outside [0, max_pages * page_size], a position below 0 where the length is less than n_b, a page outside [0, num_pages))
 * is not stored and sets KDA_DEVERR_PAGES; the row's other tokens are stored, and its queries rotated all the same.
 * Limits as for kda_rotary and kda_attention_decode.
 */
KDA_API kda_status kda_cache_append(const void* q, const void* k, const void* v, void* k_pages, void* v_pages,
                                    const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_seqlens,
                                    const double* inv_freq, int32_t B, int32_t T, int32_t H_q, int32_t H_kv, int32_t d,
                                    int32_t rotary_dim, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                    int32_t num_pages, int32_t page_size, int32_t max_pages, int64_t k_page_stride,
                                    int64_t v_page_stride, kda_dtype dt, int32_t layout, float rotary_scale,
                                    void* q_out, int64_t q_out_stride, void* stream);

/*
 * Attention of a packed batch's new tokens over a paged cache that holds their keys and values already
 * (kda_cache_append): as kda_attention_decode with the token's own position in the place of the last one.  The token
 * at position i sees the tokens j <= i, and with window > 0 of those only j > i - window and j < sinks.  A token that
 * sees nothing gives o = 0 and lse = -inf.  What a token does not see is not used for it, whatever it holds.
 *   q          [T, H_q, d] dtype dt;  o likewise;  lse [T, H_q] float32 or NULL
 *   cu_seqlens [B + 1] int32;  the other arguments as for kda_attention_decode
 *   workspace  kda_attention_prefill_workspace_size(...) bytes: partial results of units whose keys are split over
 *              several CTAs, joined in a fixed order (two calls give the same bits)
 * bf16: scores, sums and outputs are float32 until the end; at d = 64 and 128 weights are rounded to bf16 for the second
 * product, whose outputs are divided by the sum of the rounded ones.  Limits as for kda_attention_decode, and T * H_q
 * below 2^31.
 * A length outside [0, max_pages * page_size] counts as 0, new tokens before position 0 see nothing, and a page outside
 * [0, num_pages) reads as zeros; all set KDA_DEVERR_PAGES.  A page that no token sees (behind every window) may be
 * any number.
 */
KDA_API size_t kda_attention_prefill_workspace_size(int32_t B, int32_t T, int32_t H_q, int32_t H_kv, int32_t d,
                                                    kda_dtype dt);
KDA_API kda_status kda_attention_prefill(const void* q, const void* k_pages, const void* v_pages,
                                         const int32_t* block_table, const int32_t* seq_lens, const int32_t* cu_seqlens,
                                         int32_t B, int32_t T, int32_t H_q, int32_t H_kv, int32_t d, int32_t num_pages,
                                         int32_t page_size, int32_t max_pages, int64_t k_page_stride,
                                         int64_t v_page_stride, kda_dtype dt, float scale, int32_t window,
                                         int32_t sinks, void* o, float* lse, void* workspace, size_t workspace_bytes,
                                         void* stream);

/*
 * Log probabilities of given tokens under rows of logits, in float32:
 *
 *     lse_t = m + log sum_v exp(x_tv - m),   logp_t = x_ty - lse_t,   entropy_t = -sum_v p_tv log p_tv
 *
 * and the `top` likeliest words of each row, the lowest word first among equal logits (a NaN counts as -inf there).
 * A small -logp or entropy keeps its relative precision.  A row with nothing above -inf gives lse and every log
 * probability -inf and entropy 0; a row with a NaN or +inf gives NaNs.
 *   logits    [T, V] dtype dt, row t at logits + t * row_stride (elements, >= V)
 *   tokens    [T] int32, -1: none (logp_t = 0); one outside [-1, V) counts as -1 and sets KDA_DEVERR_TOKEN
 *   logp [T];  lse [T] or NULL;  entropy [T] or NULL
 *   top_logp, top_token [T, top] float32 and int32, best first; NULL with top = 0
 * top <= KDA_LOGPROBS_MAX_TOP and <= V; V at most 2^31 - 2^14, T at most 2^28 - 1 (KDA_ERR_TOO_LARGE above).
 */
#define KDA_LOGPROBS_MAX_TOP 32
KDA_API kda_status kda_token_logprobs(const void* logits, int64_t row_stride, const int32_t* tokens, int32_t T,
                                      int32_t V, kda_dtype dt, int32_t top, float* logp, float* lse, float* entropy,
                                      float* top_logp, int32_t* top_token, void* stream);

/*
 * Their gradient: grad_tv = grad_logp_t (1[v = y_t] - p_tv) - grad_entropy_t p_tv (log p_tv + entropy_t), with p from
 * the lse that kda_token_logprobs gave, or from the row itself where float32 leaves such an lse too few bits (beyond 1,024
 * from zero: rows masked by a type's lowest value, too).  A token outside [0, V) has no grad_logp; a row whose lse is -inf
 * no gradient.
 *   grad  [T, V] dtype dt, row t at grad + t * grad_stride; may be logits, with the same stride
 *   entropy and grad_entropy [T] float32, or both NULL
 * Limits as for kda_token_logprobs, and all rows' chunks of 4,096 bf16 or 2,048 float32 words (the first one up to 7 or 3
 * words shorter) below 2^31 (KDA_ERR_TOO_LARGE above).
 */
KDA_API kda_status kda_token_logprobs_backward(const void* logits, int64_t row_stride, const int32_t* tokens,
                                               const float* lse, const float* entropy, const float* grad_logp,
                                               const float* grad_entropy, int32_t T, int32_t V, kda_dtype dt,
                                               void* grad, int64_t grad_stride, void* stream);

/*
 * Synchronises `stream`, then reads and clears the current device's error
 * word.  *bits (may be NULL) receives the KDA_DEVERR_* bits that were set.
 * Returns KDA_OK if none were set, KDA_ERR_DEVICE if some were, KDA_ERR_CUDA if
 * a CUDA call failed.
 */
KDA_API kda_status kda_get_device_error(void* stream, uint32_t* bits);

/* Static, human-readable name of a status code. */
KDA_API const char* kda_status_string(kda_status s);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
