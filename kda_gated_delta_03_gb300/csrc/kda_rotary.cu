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
// What bounds it is DRAM: every element is read and written once.  A CTA takes TB tokens: their n angles each are worked out
// once in shared memory and used for all heads of q and k.  A thread has two vectors of 16 bytes under way at a time, and 16
// CTAs fit an SM: 26,814 tokens of 48 heads into pages 105 us (6.3 TB/s; with one vector 140), 16,384 tokens of 40 heads
// 56.5 us (5.9 TB/s).  Two to four such items loaded before the first is stored were slower (76 to 110 us for the latter).
#include "kda_prompt.cuh"

namespace kda {
namespace {

constexpr int NT = 128;
constexpr int MAX_N = 64;                     // pairs of a head
constexpr int MAX_TB = 2;                     // tokens of a CTA

// VEC elements as they are loaded and stored, and as floats.
template <typename T, int VEC>
struct Vec;
template <typename T>
struct Vec<T, 1> {
    T x;
    __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = (float)x; }
    __device__ __forceinline__ void set(const float (&f)[1]) { x = (T)f[0]; }
};
template <>
struct Vec<float, 4> {
    float4 x;
    __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w; }
    __device__ __forceinline__ void set(const float (&f)[4]) { x = make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Vec<__nv_bfloat16, 8> {
    uint4 x;
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
        x = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Where pair i's cosine and sine lie.  A thread needs those of VEC pairs from item * VEC on, two at a time: the same two of
// neighbouring items lie side by side, so that a warp's reads of 16 bytes meet in no bank.
template <int VEC>
__device__ __forceinline__ int place(int i) {
    return VEC == 1 ? i : (i % VEC / 2) * (2 * MAX_N / VEC) + i / VEC * 2 + i % 2;
}
template <int VEC>
__device__ __forceinline__ float4 two_places(const float2* turn, int item, int k) {
    return *reinterpret_cast<const float4*>(turn + k * (2 * MAX_N / VEC) + item * 2);
}

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

// A token's work: the items of each head of q and k, then v's, `whole` a head.  An item is two vectors of VEC elements, so that a
// thread has two loads under way: those of VEC pairs in the half layout, neighbours in the interleaved one and where
// heads are copied (the second may lie past the head there).
struct Items {
    int32_t turned, items, whole, total;      // turned: items whose vectors are pairs of each other
    Divisor by_items, by_whole, by_total;
};

// VEC elements at a time: 16 bytes where everything is aligned to them, one element else.
template <typename T, int VEC>
__global__ void __launch_bounds__(NT) kda_rotary_kernel(RotaryParams p, Items g, int TB) {
    using V = Vec<T, VEC>;
    __shared__ __align__(16) float2 turn[MAX_TB][MAX_N];       // cos, sin, pair i at place(i)
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
                turn[j][place<VEC>(i)] = make_float2(cs.x * p.scale, cs.y * p.scale * p.sign);
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
            int item, c, apart;
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
                const bool halves = item < g.turned && !p.interleaved;
                c = halves ? item * VEC : p.interleaved ? 2 * item * VEC : 2 * n + 2 * (item - g.turned) * VEC;
                apart = halves ? n : VEC;
            } else {
                if (page < 0) continue;
                const int x = w - heads, h = over(x, g.by_whole);
                item = INT32_MAX, c = (x - h * g.whole) * 2 * VEC, apart = VEC;
                src = static_cast<const T*>(p.v) + t * p.v_stride + h * p.d;
                dst = static_cast<T*>(p.v_pages) + page * p.v_page_stride + ((int64_t)h * p.page_size + slot_s[j]) * p.d;
            }
            const bool two = c + apart < p.d;
            V a = *reinterpret_cast<const V*>(src + c), b{};
            if (two) b = *reinterpret_cast<const V*>(src + c + apart);
            if (item < g.turned) {
                float x[VEC], y[VEC];
                a.get(x), b.get(y);
                auto turned = [&](int i, float2 cs) {
                    const float u = x[i], v = y[i];
                    x[i] = across(u, v, cs);
                    y[i] = along(u, v, cs);
                };
                if constexpr (VEC == 1) {
                    turned(0, turn[j][item]);
                } else {
#pragma unroll
                    for (int k = 0; k < VEC / 2; ++k) {
                        const float4 cs = two_places<VEC>(turn[j], item, k);
                        turned(2 * k, make_float2(cs.x, cs.y));
                        turned(2 * k + 1, make_float2(cs.z, cs.w));
                    }
                }
                a.set(x), b.set(y);
            } else if constexpr (VEC > 1) {
                if (c < 2 * n && item != INT32_MAX) {          // pairs side by side
                    auto turned = [&](V& vec, int second) {
                        float x[VEC];
                        vec.get(x);
#pragma unroll
                        for (int k = 0; k < VEC / 4; ++k) {
                            const float4 cs = two_places<VEC>(turn[j], item, second * (VEC / 4) + k);
                            const float u = x[4 * k], v = x[4 * k + 1], w = x[4 * k + 2], z = x[4 * k + 3];
                            x[4 * k] = across(u, v, make_float2(cs.x, cs.y));
                            x[4 * k + 1] = along(u, v, make_float2(cs.x, cs.y));
                            x[4 * k + 2] = across(w, z, make_float2(cs.z, cs.w));
                            x[4 * k + 3] = along(w, z, make_float2(cs.z, cs.w));
                        }
                        vec.set(x);
                    };
                    turned(a, 0);
                    if (c + VEC < 2 * n) turned(b, 1);
                }
            }
            *reinterpret_cast<V*>(dst + c) = a;
            if (two) *reinterpret_cast<V*>(dst + c + apart) = b;
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
    const int vec = wide ? W : 1;
    Items g;
    g.turned = p.interleaved && wide ? 0 : n / vec;
    const int rest = (p.interleaved && wide ? p.d : p.d - 2 * n) / vec;    // vectors outside of those items
    g.items = g.turned + (rest + 1) / 2;
    g.whole = p.append ? p.d / vec / 2 : 0;
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
