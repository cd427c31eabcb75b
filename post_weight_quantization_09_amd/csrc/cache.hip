// The paged cache of keys and values: rows quantised as they are written, and read back.
//
// A row of a token and head is kept on the symmetric grid of gptq_quantize_layer: s = absmax / (2^(b-1) - 1/2), codes
// round-half-even(x / s).  The rounding is exact, not that of a rounded quotient: with q = rint(x * (1 / s)) the remainder
// x - q s is representable (q has at most 8 bits, |x - q s| is not above s / 2 by more than a few of x's last places), so
// one fused multiply-add gives it and comparing it with s / 2 moves q to the neighbour where that is nearer, or even.
#include "context.hpp"

namespace gptq {

namespace {

struct CacheArgs {
    const void* k;
    const void* v;
    int64_t k_ts, k_hs, v_ts, v_hs;
    const int32_t* slots;
    uint8_t* pages;
    int64_t n_slots, page_stride, head_stride;
    int T, H, D, Dp, page_size;
};

__device__ __forceinline__ int exact_code(float x, float s, float inv, int lo, int hi) {
    float q = rintf(x * inv);
    const float rem = fmaf(-q, s, x), twice = 2.0f * fabsf(rem);
    const bool odd = ((int)q & 1) != 0;
    if (twice > s || (twice == s && odd)) q += copysignf(1.0f, rem);
    return min(max((int)q, lo), hi);
}

template <int BITS>
__device__ __forceinline__ float grid_scale(uint32_t absmax) {
    constexpr float kTop = (float)(1 << (BITS - 1)) - 0.5f;
    return absmax >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : fmaxf(__uint_as_float(absmax) / kTop, 0x1p-126f);
}

// Offset of dimension d of a page's slot within a head's block: keys' rows, values by eight tokens.
template <int BITS>
__device__ __forceinline__ int key_at(int slot, int d, int Dp) { return (slot * Dp + d) * BITS / 8; }
template <int BITS>
__device__ __forceinline__ int value_at(int slot, int d, int Dp) {
    if constexpr (BITS == 4) return ((slot >> 3) * (Dp / 2) + d / 2) * 8 + (slot & 7);
    return (((slot >> 3) * Dp + d) * 8 + (slot & 7)) * (BITS / 8);
}

template <typename E, int BITS>
__global__ __launch_bounds__(64) void cache_write_kernel(CacheArgs a) {
    const int t = blockIdx.x, h = blockIdx.y;
    const bool values = blockIdx.z != 0;
    const int slot = a.slots[t];
    if ((uint32_t)slot >= (uint64_t)a.n_slots) return;
    const E* x = values ? static_cast<const E*>(a.v) + t * a.v_ts + h * a.v_hs
                        : static_cast<const E*>(a.k) + t * a.k_ts + h * a.k_hs;
    const int at = slot % a.page_size;
    uint8_t* block = a.pages + (int64_t)(slot / a.page_size) * a.page_stride + h * a.head_stride;
    const int part = a.page_size * a.Dp * BITS / 8;
    uint8_t* codes = block + (values ? part : 0);
    float s = 1.0f, inv = 1.0f;
    if constexpr (BITS < 16) {
        uint32_t m = 0;
        for (int d = threadIdx.x; d < a.D; d += 64) m = max(m, __float_as_uint((float)x[d]) & 0x7FFFFFFFu);
        for (int i = 32; i; i >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, i));
        s = grid_scale<BITS>(m);
        inv = 1.0f / s;
        if (threadIdx.x == 0) reinterpret_cast<float*>(block + 2 * part)[(values ? a.page_size : 0) + at] = s;
    }
    constexpr int kLow = -(1 << (BITS < 16 ? BITS - 1 : 0)), kHigh = -kLow - 1;
    for (int d = 2 * threadIdx.x; d < a.Dp; d += 128) {
        const float u = d < a.D ? (float)x[d] : 0.0f, w = d + 1 < a.D ? (float)x[d + 1] : 0.0f;
        if constexpr (BITS == 16) {
            *reinterpret_cast<__bf16*>(codes + (values ? value_at<16>(at, d, a.Dp) : key_at<16>(at, d, a.Dp))) = (__bf16)u;
            *reinterpret_cast<__bf16*>(codes + (values ? value_at<16>(at, d + 1, a.Dp) : key_at<16>(at, d + 1, a.Dp))) = (__bf16)w;
        } else {
            const bool fine = s == s;
            const int c0 = fine ? exact_code(u, s, inv, kLow, kHigh) : 0, c1 = fine ? exact_code(w, s, inv, kLow, kHigh) : 0;
            if constexpr (BITS == 8) {
                codes[values ? value_at<8>(at, d, a.Dp) : key_at<8>(at, d, a.Dp)] = (uint8_t)c0;
                codes[values ? value_at<8>(at, d + 1, a.Dp) : key_at<8>(at, d + 1, a.Dp)] = (uint8_t)c1;
            } else {
                codes[values ? value_at<4>(at, d, a.Dp) : key_at<4>(at, d, a.Dp)] = (uint8_t)((c0 & 15) | (c1 << 4));
            }
        }
    }
}

template <typename E, int BITS>
__global__ __launch_bounds__(64) void cache_read_kernel(CacheArgs a) {
    const int t = blockIdx.x, h = blockIdx.y;
    const bool values = blockIdx.z != 0;
    const int slot = a.slots[t];
    E* y = values ? (E*)a.v + t * a.v_ts + h * a.v_hs : (E*)a.k + t * a.k_ts + h * a.k_hs;
    if ((uint32_t)slot >= (uint64_t)a.n_slots) {
        for (int d = threadIdx.x; d < a.D; d += 64) y[d] = (E)0.0f;
        return;
    }
    const int at = slot % a.page_size;
    const uint8_t* block = a.pages + (int64_t)(slot / a.page_size) * a.page_stride + h * a.head_stride;
    const int part = a.page_size * a.Dp * BITS / 8;
    const uint8_t* codes = block + (values ? part : 0);
    float s = 1.0f;
    if constexpr (BITS < 16) s = reinterpret_cast<const float*>(block + 2 * part)[(values ? a.page_size : 0) + at];
    for (int d = threadIdx.x; d < a.D; d += 64) {
        const uint8_t* c = codes + (values ? value_at<BITS>(at, d, a.Dp) : key_at<BITS>(at, d, a.Dp));
        float x;
        if constexpr (BITS == 16) x = (float)*reinterpret_cast<const __bf16*>(c);
        else if constexpr (BITS == 8) x = s * (float)(int8_t)*c;
        else x = s * (float)((int)((uint32_t)*c << (d & 1 ? 24 : 28)) >> 28);
        y[d] = (E)x;
    }
}

CacheArgs cache_args(HeadRows k, HeadRows v, int64_t T, int H, int D, const int32_t* slots, const Pages& p) {
    return {k.p, v.p, k.ts, k.hs, v.ts, v.hs, slots, p.p, p.n * p.page_size, p.page_stride, p.head_stride,
            (int)T, H, D, stored_head_size(D), p.page_size};
}

}  // namespace

hipError_t cache_write(HeadRows k, HeadRows v, bool f32, int64_t T, int H, int D, const int32_t* slots, Pages pages,
                       hipStream_t stream) {
    const CacheArgs a = cache_args(k, v, T, H, D, slots, pages);
    auto pick = [&](auto e) {
        using E = decltype(e);
        return pages.bits == 16 ? cache_write_kernel<E, 16> : pages.bits == 8 ? cache_write_kernel<E, 8> : cache_write_kernel<E, 4>;
    };
    (f32 ? pick(0.0f) : pick((__bf16)0.0f))<<<dim3((unsigned)T, (unsigned)H, 2), 64, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t cache_read(Pages pages, const int32_t* slots, int64_t T, int H, int D, HeadRows k, HeadRows v, bool f32,
                      hipStream_t stream) {
    const CacheArgs a = cache_args(k, v, T, H, D, slots, pages);
    auto pick = [&](auto e) {
        using E = decltype(e);
        return pages.bits == 16 ? cache_read_kernel<E, 16> : pages.bits == 8 ? cache_read_kernel<E, 8> : cache_read_kernel<E, 4>;
    };
    (f32 ? pick(0.0f) : pick((__bf16)0.0f))<<<dim3((unsigned)T, (unsigned)H, 2), 64, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace gptq
