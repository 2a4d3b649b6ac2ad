// Rotary positions of queries and keys, and a batch's new tokens into the pages of a key-value cache.
//
//   (a, b) -> scale * (a cos - b sin, b cos + a sin),   angle = position * inv_freq[i]
//
// for the pairs (x_i, x_{i + n}) ("half") or (x_2i, x_{2i + 1}) ("interleaved"), i < n = rot / 2; the rest of the head is
// copied.  Turned by minus the angle it is its own gradient.
//
// Angles: position * inv_freq reaches 1e6 radians and more, where fp32 holds no fraction of a turn.  A frequency is
// made a 64-bit fraction of a turn, once by each thread (fp64, the product's and the constant's lower parts included); its
// product with the position modulo 2^64 is an integer multiplication, which drops whole turns exactly.  Quarter turns come
// off the upper 32 bits of the rest before they become a float, so that the 24 bits are those of an eighth of a turn, and
// sincospi takes that.  So any 32-bit position is as exact as the first one, and no 64-bit sine is needed (one costs more
// than a head's whole traffic).
//
// What bounds it is DRAM: every element is read and written once.  A CTA takes TB tokens: their n angles each are
// worked out once in shared memory and used for all heads of q and k, while the first vectors are on their way.
#include "kda_prompt.cuh"

namespace kda {
namespace {

constexpr int NT = 128;
constexpr int MAX_N = 64;                     // pairs of a head
constexpr int MAX_TB = 2;                     // tokens of a CTA

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
    T x[VEC];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& y, float x) { y = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

// The rotation, with the same roundings wherever it stands: every variant gives the same bits.
__device__ __forceinline__ float across(float a, float b, float2 cs) { return __fmaf_rn(a, cs.x, -__fmul_rn(b, cs.y)); }
__device__ __forceinline__ float along(float a, float b, float2 cs) { return __fmaf_rn(b, cs.x, __fmul_rn(a, cs.y)); }

// inv_freq (radians a position) as a fraction of a turn in 64 bits: f / (2 pi) in two parts, whole turns off the first one.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
    const double c = 0.15915494309189535, c_low = -9.839338337591243e-18;  // 1 / (2 pi)
    const double hi = __dmul_rn(f, c), lo = __fma_rn(f, c_low, __fma_rn(f, c, -hi));
    return (uint64_t)__double2ll_rn((hi - rint(hi)) * 0x1p64) + (uint64_t)__double2ll_rn(lo * 0x1p64);
}

// cos, sin of a 64-bit fraction of a turn.
__device__ __forceinline__ float2 cos_sin(uint64_t phase) {
    const uint32_t x = (uint32_t)(phase >> 32), quarters = (x + (1u << 29)) >> 30;
    float s, c;
    sincospif((float)(int32_t)(x - (quarters << 30)) * 0x1p-31f, &s, &c);
    const float2 y = quarters & 1u ? make_float2(-s, c) : make_float2(c, s);
    return quarters & 2u ? make_float2(-y.x, -y.y) : y;
}

// The sequence of a packed batch that token t belongs to: the first b with cu[b + 1] > t, or B.  A warp looks at 32
// borders at once, so 1,024 sequences take two loads' latency.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int t, int lane) {
    int lo = 0, n = B;                        // the answer is in [lo, lo + n]
    while (n > 0) {
        const int step = (n + 31) / 32, i = lo + min((lane + 1) * step, n) - 1;
        const unsigned past = __ballot_sync(0xFFFFFFFFu, __ldg(cu + i + 1) > t);
        if (past == 0) return lo + n;
        const int first = __ffs(past) - 1;
        const int end = lo + min((first + 1) * step, n) - 1;
        lo += first * step;
        n = end - lo;                         // cu[end + 1] > t: the answer is at most `end`
    }
    return lo;
}

// A token's work: for each head of q and k `turned` items that rotate, then copied vectors; then v's vectors, `whole` a head.
// In the half layout an item is VEC pairs in two vectors, in the interleaved one a vector (or, one element at a time, a pair).
struct Items {
    int32_t turned, items, whole, total;
    Divisor by_items, by_whole, by_total;
};

// VEC elements at a time: 16 bytes where everything is aligned to them, one element else.
template <typename T, int VEC>
__global__ void __launch_bounds__(NT) kda_rotary_kernel(RotaryParams p, Items g, int TB) {
    using V = Vec<T, VEC>;
    __shared__ float2 turn[MAX_TB][MAX_N];                     // cos, sin
    __shared__ int pos_s[MAX_TB];
    __shared__ int page_s[MAX_TB], slot_s[MAX_TB];             // page -1: not stored
    __shared__ int real_s[MAX_TB];                             // a token of some sequence
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = blockIdx.x * TB, n = p.rot >> 1;
    const int tokens = min(TB, p.T - t0);
    if (p.append) {
        if (blockIdx.x == 0)                                   // what is wrong with cu_seqlens as a whole
            for (int b = tid; b <= p.B; b += NT) {
                const int x = __ldg(p.cu + b);
                if (b == 0 ? x != 0 : (x < __ldg(p.cu + b - 1) || x > p.T)) atomicOr(p.err, KDA_DEVERR_CU_SEQLENS);
            }
        if (warp < tokens) {
            const int t = t0 + warp, b = sequence_of(p.cu, p.B, t, lane);
            if (lane == 0) {
                int page = -1, slot = 0, pos = 0, real = 0;
                const int start = b < p.B ? __ldg(p.cu + b) : 0, end = b < p.B ? __ldg(p.cu + b + 1) : 0;
                // a sequence whose borders are not in order counts as empty: its tokens are left alone
                if (start >= 0 && start <= t && t < end && end <= p.T && (b > 0 || start == 0)) {
                    const int len = __ldg(p.lens + b);
                    real = 1;
                    pos = (int)((int64_t)len - ((int64_t)end - t));
                    if (len >= 0 && (int64_t)len <= (int64_t)p.max_pages * p.page_size && pos >= 0) {
                        const int at = pos / p.page_size;
                        slot = pos - at * p.page_size;
                        page = __ldg(p.table + (int64_t)b * p.max_pages + at);
                        if (page < 0 || page >= p.num_pages) page = -1;
                    }
                    if (page < 0) atomicOr(p.err, KDA_DEVERR_PAGES);
                }
                pos_s[warp] = pos, page_s[warp] = page, slot_s[warp] = slot, real_s[warp] = real;
            }
        }
    } else if (tid < tokens) {
        pos_s[tid] = __ldg(p.positions + t0 + tid);
        real_s[tid] = 1;
    }
    __syncthreads();
    if (n > 0) {
        const int group = NT / MAX_N;                          // NT threads: MAX_N pairs of `group` tokens at a time
        const int i = tid % MAX_N;
        if (i < n) {
            const uint64_t f = turn_fraction(__ldg(p.inv_freq + i));
            for (int j = tid / MAX_N; j < tokens; j += group) {
                const float2 cs = cos_sin((uint64_t)(int64_t)pos_s[j] * f);
                turn[j][i] = make_float2(cs.x * p.scale, cs.y * p.scale * p.sign);
            }
        }
        __syncthreads();
    }

    const int heads = (p.Hq + p.Hkv) * g.items, all = tokens * g.total;
    {
        for (int w0 = tid; w0 < all; w0 += NT) {
            const int j = over(w0, g.by_total), w = w0 - j * g.total;
            if (!real_s[j]) continue;
            const int64_t t = t0 + j, page = p.append ? page_s[j] : 0;
            const T* src;
            T* dst;
            int item;
            if (w < heads) {
                const int h = over(w, g.by_items);
                item = w - h * g.items;
                if (h < p.Hq) {
                    src = static_cast<const T*>(p.q) + t * p.q_stride + h * p.d;
                    dst = static_cast<T*>(p.q_out) + t * p.q_out_stride + h * p.d;
                } else {
                    src = static_cast<const T*>(p.k) + t * p.k_stride + (h - p.Hq) * p.d;
                    if (p.append) {
                        if (page < 0) continue;
                        dst = static_cast<T*>(p.k_pages) + page * p.k_page_stride +
                              ((int64_t)(h - p.Hq) * p.page_size + slot_s[j]) * p.d;
                    } else {
                        dst = static_cast<T*>(p.k_out) + t * p.k_out_stride + (h - p.Hq) * p.d;
                    }
                }
            } else {
                if (page < 0) continue;
                const int x = w - heads, h = over(x, g.by_whole), c = (x - h * g.whole) * VEC;
                *reinterpret_cast<V*>(static_cast<T*>(p.v_pages) + page * p.v_page_stride +
                                      ((int64_t)h * p.page_size + slot_s[j]) * p.d + c) =
                    *reinterpret_cast<const V*>(static_cast<const T*>(p.v) + t * p.v_stride + h * p.d + c);
                continue;
            }
            if (item >= g.turned) {
                const int c = 2 * n + (item - g.turned) * VEC;
                *reinterpret_cast<V*>(dst + c) = *reinterpret_cast<const V*>(src + c);
            } else if (!p.interleaved) {
                const int c = item * VEC;
                const V a = *reinterpret_cast<const V*>(src + c), b = *reinterpret_cast<const V*>(src + n + c);
                V x, y;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float2 cs = turn[j][c + i];
                    const float u = to_f(a.x[i]), v = to_f(b.x[i]);
                    from_f(x.x[i], across(u, v, cs));
                    from_f(y.x[i], along(u, v, cs));
                }
                *reinterpret_cast<V*>(dst + c) = x;
                *reinterpret_cast<V*>(dst + n + c) = y;
            } else if constexpr (VEC > 1) {
                const V a = *reinterpret_cast<const V*>(src + item * VEC);
                V x;
#pragma unroll
                for (int i = 0; i < VEC; i += 2) {
                    const float2 cs = turn[j][item * (VEC / 2) + i / 2];
                    const float u = to_f(a.x[i]), v = to_f(a.x[i + 1]);
                    from_f(x.x[i], across(u, v, cs));
                    from_f(x.x[i + 1], along(u, v, cs));
                }
                *reinterpret_cast<V*>(dst + item * VEC) = x;
            } else {
                const float2 cs = turn[j][item];
                const float u = to_f(src[2 * item]), v = to_f(src[2 * item + 1]);
                from_f(dst[2 * item], across(u, v, cs));
                from_f(dst[2 * item + 1], along(u, v, cs));
            }
        }
    }
}

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

template <typename T>
cudaError_t launch(const RotaryParams& p, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    const int n = p.rot / 2;
    const int64_t odd = p.q_stride | p.k_stride | p.v_stride | p.q_out_stride | p.k_out_stride;
    const bool wide = odd % W == 0 && on16(p.q) && on16(p.k) && on16(p.v) && on16(p.q_out) && on16(p.k_out) &&
                      (p.interleaved ? 2 * n : n) % W == 0 && (p.d - 2 * n) % W == 0;
    const int vec = wide ? W : 1, per = p.interleaved ? (wide ? W / 2 : 1) : vec;      // pairs of an item
    Items g;
    g.turned = n / per;
    g.items = g.turned + (p.d - 2 * n) / vec;
    g.whole = p.append ? p.d / vec : 0;
    g.total = (p.Hq + p.Hkv) * g.items + p.Hkv * g.whole;
    g.by_items = divisor(g.items);
    g.by_whole = divisor(g.whole > 0 ? g.whole : 1);
    g.by_total = divisor(g.total);
    // Two tokens a CTA share the frequencies' conversion (16,384 tokens of 40 heads 56 us, with one 57, with four 59); one
    // while the CTAs would not fill the GPU otherwise.
    static DeviceSetup done;
    int sms = 0;
    const cudaError_t e = device_setup(done, nullptr, 0, &sms);
    if (e != cudaSuccess) return e;
    const int TB = p.T > 8 * sms ? MAX_TB : 1;
    const int grid = (int)(((int64_t)p.T + TB - 1) / TB);
    if (wide)
        kda_rotary_kernel<T, W><<<grid, NT, 0, s>>>(p, g, TB);
    else
        kda_rotary_kernel<T, 1><<<grid, NT, 0, s>>>(p, g, TB);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, kda_dtype dt, cudaStream_t s) {
    return dt == KDA_DTYPE_BF16 ? launch<__nv_bfloat16>(p, s) : launch<float>(p, s);
}

}  // namespace kda
