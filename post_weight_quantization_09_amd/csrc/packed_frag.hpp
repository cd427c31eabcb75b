// Matrix-core fragments straight from the packed words of gptq_pack_codes (layout in include/gptq.h).
//
// A layer's weight is W[k][n] = s (c - z), z = 2^(b-1).  v_mfma_f32_16x16x32_bf16 wants, in lane l, eight consecutive
// k (8 (l / 16) ..) of one channel (l % 16) as its B operand: eight codes are 8 b consecutive bits of that channel's
// stream, so a lane reads its own operand as one word (b = 2, 4) or two (b = 3, 5, 6), and 32 k are exactly b words.
// A lane takes the same words of NT neighbouring channels with one 16- (8-) byte load; product j of the NT products
// then covers channels 4 (l % 16) + j, and the lane ends up with NT consecutive channels of each of its rows.
//
// A code is turned into bf16 by writing its b <= 6 bits at the top of the mantissa of 2^-8: the value u (2^b + c), with
// u = 2^-(b+8), is exact and costs one shift and one and-or per pair of codes.  Codes i and i + 4 of the eight share a
// register (they sit 16 bits apart in a 4-bit word), so the A operand is given in the same order of k.  The excess is taken
// off again in fp32:  sum_k x_k (c_k - z) = sum_k x_k (2^b + c_k) - 1.5 2^b sum_k x_k,  with the row sums of x from a
// product with the constant -1.5 2^b u (exact in bf16) or from the pass that lays x out.  It is done for every 128 k (or
// scale group), so the partial sums stay near the size of their result.  That leaves an error of 1e-6 to 4e-6 of the
// result (against 64 bits), which bf16 output cannot show (its own rounding is 1.7e-3) but fp32 output would: fp32 rows,
// whose three parts make three products per conversion anyway, get u (c - z) itself as operand.  Scales multiply the fp32
// partial sums: no weight is rounded.
// The factor u keeps every sum of 128 products below the largest x, so that rows up to the largest value stay finite
// where their result is; 1/u multiplies the finished sums, exactly.
#pragma once

#include "gptq_common.hpp"

namespace gptq {

// Global loads take any alignment (the amdhsa target's unaligned access mode); the types say what is promised.
typedef u32x4 __attribute__((aligned(4))) u32x4_a4;
typedef u32x4 __attribute__((aligned(2))) u32x4_a2;
typedef u32x2 __attribute__((aligned(4))) u32x2_a4;
typedef f32x4 __attribute__((aligned(4))) f32x4_a4;
typedef f32x2 __attribute__((aligned(4))) f32x2_a4;

constexpr int kStepK = 32;          // k of one MFMA step: `bits` words of every channel
constexpr int kChunkSteps = 4;      // steps of one chunk (128 k, the largest scale group)
constexpr int kChunkK = kStepK * kChunkSteps;

// Words a lane reads of one step of one channel.
template <int BITS>
constexpr int kLaneWords = (BITS == 2 || BITS == 4) ? 1 : 2;

// First word (within the step) and bit shift of lane quarter q's eight codes.
template <int BITS>
__device__ __forceinline__ int lane_word(int q) { return (8 * BITS * q) >> 5; }
template <int BITS>
__device__ __forceinline__ int lane_shift(int q) { return (8 * BITS * q) & 31; }
// The second word, or the first again where eight codes do not reach it.
template <int BITS>
__device__ __forceinline__ int lane_word2(int q) {
    return lane_word<BITS>(q) + (lane_shift<BITS>(q) + 8 * BITS > 32 ? 1 : 0);
}

template <int S>
__device__ __forceinline__ uint32_t shl_signed(uint32_t v) {
    if constexpr (S >= 0) return v << S;
    else return v >> (-S);
}

// The exponent of every code's value u (2^b + c) = 2^-8 (1 + c / 2^b), and 1/u.
constexpr int kCodeExponent = -8;
template <int BITS>
constexpr float kCodeUnits = (float)(1 << (BITS - kCodeExponent));

// 2^-8 in both halves of a vector register: with it there, and the mask in a scalar one, and-or is one instruction (a
// VALU instruction of gfx950 reads one scalar or literal at most).
__device__ __forceinline__ uint32_t code_base() {
    uint32_t base = ((uint32_t)(127 + kCodeExponent) << 7) * 0x10001u;
    asm("" : "+v"(base));
    return base;
}

template <int BITS, int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t lo, uint32_t hi, uint32_t base) {
    constexpr uint32_t m = (((1u << BITS) - 1u) << (7 - BITS)) * 0x10001u;
    if constexpr (BITS <= 4) {                // lo holds codes 0..3 from bit 0 and codes 4..7 from bit 16
        return (shl_signed<7 - BITS - BITS * I>(lo) & m) | base;
    } else {
        const uint32_t a = shl_signed<7 - BITS - BITS * I>(lo), b = shl_signed<23 - BITS - BITS * I>(hi);
        return (((a & 0xFFFFu) | (b & 0xFFFF0000u)) & m) | base;
    }
}

// Eight codes (in words w0, w1 at bit `sh`) -> bf16 values u (2^b + c), register i = codes (i, i + 4).
template <int BITS>
__device__ __forceinline__ bf16x8 codes_to_frag(uint32_t w0, uint32_t w1, int sh, uint32_t base) {
    uint32_t lo, hi = 0;
    if constexpr (BITS == 4) {
        lo = w0;
    } else if constexpr (BITS == 2) {
        lo = __builtin_amdgcn_perm(0u, w0, sh ? 0x0C030C02u : 0x0C010C00u);
    } else {
        const uint64_t v = (((uint64_t)w1 << 32) | w0) >> sh;
        if constexpr (BITS == 3) {
            const uint32_t t = (uint32_t)v;
            lo = (t & 0xFFFu) | ((t & 0xFFF000u) << 4);
        } else {
            lo = (uint32_t)v;
            hi = (uint32_t)(v >> (4 * BITS));
        }
    }
    u32x4 r;
    r[0] = code_pair<BITS, 0>(lo, hi, base);
    r[1] = code_pair<BITS, 1>(lo, hi, base);
    r[2] = code_pair<BITS, 2>(lo, hi, base);
    r[3] = code_pair<BITS, 3>(lo, hi, base);
    return __builtin_bit_cast(bf16x8, r);
}

// The same as bf16 values u (c - z): the excess taken off in fp32 (both steps exact), five more operations per pair.
template <int BITS>
__device__ __forceinline__ bf16x8 codes_to_exact_frag(uint32_t w0, uint32_t w1, int sh, uint32_t base) {
    constexpr float excess = 1.5f / (float)(1 << -kCodeExponent);
    const u32x4 v = __builtin_bit_cast(u32x4, codes_to_frag<BITS>(w0, w1, sh, base));
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        r[i] = __builtin_amdgcn_perm(__float_as_uint(bf16hi_to_f32(v[i]) - excess),
                                     __float_as_uint(bf16lo_to_f32(v[i]) - excess), 0x07060302u);
    return __builtin_bit_cast(bf16x8, r);
}

// -1.5 2^b u in both halves of a register (exact: 2^-8 (1 + 1/2)).
__device__ __forceinline__ bf16x8 minus_excess_frag() {
    constexpr uint32_t v = 0x80008000u | (((uint32_t)(127 + kCodeExponent) << 7) | 0x40u) * 0x10001u;
    return __builtin_bit_cast(bf16x8, u32x4{v, v, v, v});
}

// Eight consecutive bf16 in natural order -> register i = elements (i, i + 4).
__device__ __forceinline__ u32x4 pair_order(u32x4 v) {
    u32x4 r;
    r[0] = __builtin_amdgcn_perm(v[2], v[0], 0x05040100u);
    r[1] = __builtin_amdgcn_perm(v[2], v[0], 0x07060302u);
    r[2] = __builtin_amdgcn_perm(v[3], v[1], 0x05040100u);
    r[3] = __builtin_amdgcn_perm(v[3], v[1], 0x07060302u);
    return r;
}

// Eight fp32 values as three bf16 parts whose sum is exact (24 = 3 x 8 mantissa bits): part p in natural order.  They
// are cut off, not rounded: rounded up, the parts of values near the largest one would be infinite, or their sum on the way.
// A non-finite value goes into the first part as it is; its remainders, NaN by then, are taken as zero.
__device__ __forceinline__ void split3(const float (&x)[8], u32x4 (&part)[3]) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
    for (int p = 0; p < 3; ++p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            part[p][i] = __builtin_amdgcn_perm(__float_as_uint(r[2 * i + 1]), __float_as_uint(r[2 * i]), 0x07060302u);
            const float a = r[2 * i] - bf16lo_to_f32(part[p][i]), b = r[2 * i + 1] - bf16hi_to_f32(part[p][i]);
            r[2 * i] = a == a ? a : 0.f;
            r[2 * i + 1] = b == b ? b : 0.f;
        }
    }
}

// Eight elements k .. k + 7 of a row as they are in memory (bf16: 16 bytes, fp32: 32), zero from K on.
template <int PARTS>
struct RawOctet {
    u32x4 v[PARTS == 1 ? 1 : 2];

    __device__ __forceinline__ void whole(const char* p) {
        if constexpr (PARTS == 1) {
            v[0] = *reinterpret_cast<const u32x4_a2*>(p);
        } else {
            v[0] = reinterpret_cast<const u32x4_a4*>(p)[0];
            v[1] = reinterpret_cast<const u32x4_a4*>(p)[1];
        }
    }
    __device__ __forceinline__ void zero() {
        v[0] = u32x4{0u, 0u, 0u, 0u};
        if constexpr (PARTS != 1) v[1] = u32x4{0u, 0u, 0u, 0u};
    }
    // `left` of the row's `all` elements remain from p on (may be none or negative).  The last octet is loaded whole, from
    // further left, and moved; only rows shorter than an octet go element by element.
    __device__ __forceinline__ void some(const char* p, int left, int all) {
        if (left >= 8) {
            whole(p);
            return;
        }
        if (left <= 0) {
            zero();
            return;
        }
        if (all < 8) {
            zero();
            for (int i = 0; i < left; ++i) {
                if constexpr (PARTS == 1) {
                    const uint32_t e = reinterpret_cast<const uint16_t*>(p)[i];
#pragma unroll
                    for (int d = 0; d < 4; ++d) v[0][d] |= i >> 1 == d ? e << (16 * (i & 1)) : 0u;
                } else {
                    const uint32_t e = reinterpret_cast<const uint32_t*>(p)[i];
#pragma unroll
                    for (int d = 0; d < 8; ++d) v[d >> 2][d & 3] = i == d ? e : v[d >> 2][d & 3];
                }
            }
            return;
        }
        const int by = 8 - left;                     // 1 .. 7 elements down
        whole(p - by * (PARTS == 1 ? 2 : 4));
        constexpr int kWords = PARTS == 1 ? 4 : 8;
        uint32_t u[kWords];
#pragma unroll
        for (int d = 0; d < kWords; ++d) u[d] = v[d >> 2][d & 3];
        if constexpr (PARTS == 1) {
            if (by & 1) {
#pragma unroll
                for (int d = 0; d < 4; ++d) u[d] = (u[d] >> 16) | (d < 3 ? u[d + 1] << 16 : 0u);
            }
        }
        const int words = PARTS == 1 ? by >> 1 : by;
#pragma unroll
        for (int step = 1; step < kWords; step <<= 1) {
            if (words & step) {
#pragma unroll
                for (int d = 0; d < kWords; ++d) u[d] = d + step < kWords ? u[d + step] : 0u;
            }
        }
#pragma unroll
        for (int d = 0; d < kWords; ++d) v[d >> 2][d & 3] = u[d];
    }
    // As bf16 parts in natural order.
    __device__ __forceinline__ void parts(u32x4 (&part)[PARTS]) const {
        if constexpr (PARTS == 1) {
            part[0] = v[0];
        } else {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v[i >> 2][i & 3]);
            split3(x, part);
        }
    }
};

template <int PARTS>
__device__ __forceinline__ void load_octet(const void* row, int k, int K, u32x4 (&part)[PARTS]) {
    RawOctet<PARTS> r;
    r.some(static_cast<const char*>(row) + (int64_t)k * (PARTS == 1 ? 2 : 4), K - k, K);
    r.parts(part);
}

__device__ __forceinline__ f32x4 mfma16(u32x4 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), b, c, 0, 0, 0);
}

// silu(g) u = g u / (1 + e^-g); e^-g overflows to infinity for g below -88 and the quotient is then 0 as it should be.
__device__ __forceinline__ float gated(float g, float u) { return g / (1.f + expf(-g)) * u; }

}  // namespace gptq
