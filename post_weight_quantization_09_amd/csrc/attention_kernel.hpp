// Attention of new tokens over their pages, on the matrix cores.
//
// A wave takes 32 tokens at a time and 16 query heads of one key head, with two products of v_mfma_f32_16x16x32_bf16 whose
// operands come straight from the pages, without LDS and without moving a value between lanes:
//   scores   S^T (tokens x heads) = K Q^T.  Lane l gives, as row l % 16 of the A operand, eight dimensions of one token; which
//            token is row m is free, and tile T of two takes token 8 (m / 4) + 4 T + m % 4.  The result's lane then holds for
//            head l % 16 the tokens 8 (l / 16) .. + 7;
//   output   O^T (dimensions x heads) += V^T P^T.  Those eight tokens are exactly the K octet that the B operand wants in this
//            lane, so the probabilities go in where the scores came out; the A operand wants eight tokens of one dimension,
//            which is how the pages store values.
// Codes become bf16 exactly: 8 bits by v_cvt_f32_i32 of a byte, 4 bits for fp32 rows by v_cvt_off_f32_i4 (code / 16); for bf16
// rows two 4-bit codes become bf16 by a shift and one and-xor that sets sign and exponent, code + 24 in the low half of a
// register and code - 23 in the high half, and the excess 24 sum(low) - 23 sum(high) is taken off the sums in fp32: that of
// the scores before they are begun, that of the output after them, from a product with (24, -23).  The signs alternate so that
// the sums stay near the size of their result (an excess of one sign would reach 24 where the mean of many codes is near 0).
// A token's key scale multiplies its score, its value scale its probability.  Probabilities (times that scale), and q of fp32
// rows, are cut into three bf16 parts each (exact), so that nothing is rounded but sums.  Fewer parts were measured for bf16
// rows.  One: its error, 2^-9 of each of many terms of either sign, is as large in their sum as the output's own rounding
// (against 64 bits 2.5e-3 where that alone is 1.7e-3).  Two, 16 bits: that rounding falls the other way in 0.4% of the outputs, with
// three in 0.06% as between two orders of the sum (4 bits: 0.3%, by the sums of the excess); 131072 tokens in 4 bits 44.4 us with
// two, 44.9 with three, heads of 64 45.0 and 47.3, no other case measured by more than 3%.
//
// Softmax: scores are kept times log2 e.  A lane's maximum is raised (and what was summed rescaled) only where a score passes it
// by 8: probabilities then reach 2^8, which fp32 sums and bf16 factors bear as well as 1, and few steps rescale.
//
// Work is shared out by blocks of 32 tokens: all blocks of all segments (a request and 16 query heads of a key head) lie on
// one line, and wave w takes the w-th piece of it, whatever the lengths: an even share for 64 ragged requests as for one of
// 131072 tokens beside short ones.  Every workgroup scans the lengths for itself, R / 64 of them a lane, one load after the other:
// nothing beside the rest up to some hundred requests, most of the time of very many (below).  A wave that has a whole segment writes its
// output; one that has a part of it writes unnormalised sums, which the join adds in order.  Waves share nothing else: no LDS
// and no barrier in the loop, and little code, which counts where a call is short (the instructions of a launch come from
// memory once per CU).  (Four waves of a workgroup on one segment, joined in LDS, with three times the code before the loop:
// 111 us against 91 for 64 ragged requests, 15 against 12 for a short one.)
//
// Measured on MI355X, heads of 128: 256 requests of 1950 tokens in 16 bits, 1.02 GB, 190 to 195 us and 7 of the join (5.2 TB/s of
// reads; a copy moves 4.9); 64 ragged requests in 8 bits, 415 MB, 83 to 86 and 7 us (4.9 TB/s); 131072 tokens in 4 bits, 64 query
// heads, 145 MB, 37 to 39 and 8 us: there vector instructions take 48% of the cycles (some 380 a block: conversions, softmax,
// addresses), and with three waves a SIMD most of the rest is their waiting for a block's loads, which are
// issued when the block before is done.  A call whose work is nothing takes 7 + 4 us: lengths, page table and pages are three
// latencies in a row, the join a launch.  Many requests, 4 query heads on one or two of 128, 8 bits: 2048 of 95 tokens 43 us, 16384
// of 40 154, 65536 of 20 (heads of 64) 478.  Groups of more than 16 query heads are two segments, each of which reads the keys and
// values: 16 requests of 4000 tokens, 4 key heads, 16 and 20 query heads each: 16 bits 32 and 47 us, 8 bits 26 and 34, 4 bits 25
// and 29.
#pragma once

#include "attention.hpp"

namespace gptq {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRaise = 8.0f;
constexpr int kMostExponent = 120;              // of to_log2's power of two: what it multiplies is below 2^6

__device__ __forceinline__ uint32_t high_halves(float lo, float hi) {
    return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

// One instruction, without the canonicalisations that fmaxf asks for: a NaN is passed over, as by fmaxf.
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(y), "v"(z));
    return r;
}

// the largest of lanes l, l ^ 16, l ^ 32, l ^ 48
__device__ __forceinline__ float max_of_quarters(float x) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
    r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ float sum_of_quarters(float x) {
    auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Eight bytes as bf16 (exact).
__device__ __forceinline__ bf16x8 bytes_to_bf16(uint32_t w0, uint32_t w1) {
    u32x4 r;
    r[0] = high_halves((float)(int8_t)w0, (float)(int8_t)(w0 >> 8));
    r[1] = high_halves((float)(int8_t)(w0 >> 16), (float)(int8_t)(w0 >> 24));
    r[2] = high_halves((float)(int8_t)w1, (float)(int8_t)(w1 >> 8));
    r[3] = high_halves((float)(int8_t)(w1 >> 16), (float)(int8_t)(w1 >> 24));
    return __builtin_bit_cast(bf16x8, r);
}

// code / 16 of the low half of byte I
template <int I>
__device__ __forceinline__ float nibble(uint32_t w) { return __builtin_amdgcn_cvt_off_f32_i4((w >> 8 * I) & 0xFFu); }

__device__ __forceinline__ uint32_t upper_nibbles(uint32_t w) {
    uint32_t h = w >> 4;
    asm("" : "+v"(h));                  // kept apart from the byte shifts, which the conversion then does by itself
    return h;
}

// The low halves of eight bytes as bf16, code / 16 (exact).
__device__ __forceinline__ bf16x8 nibbles_to_bf16(uint32_t w0, uint32_t w1) {
    u32x4 r;
    r[0] = high_halves(nibble<0>(w0), nibble<1>(w0));
    r[1] = high_halves(nibble<2>(w0), nibble<3>(w0));
    r[2] = high_halves(nibble<0>(w1), nibble<1>(w1));
    r[3] = high_halves(nibble<2>(w1), nibble<3>(w1));
    return __builtin_bit_cast(bf16x8, r);
}

// Four bytes' halves in order (low, high of byte 0, ...) as bf16, code / 16 (exact).
__device__ __forceinline__ bf16x8 word_to_bf16(uint32_t w) {
    const uint32_t h = upper_nibbles(w);
    u32x4 r;
    r[0] = high_halves(nibble<0>(w), nibble<0>(h));
    r[1] = high_halves(nibble<1>(w), nibble<1>(h));
    r[2] = high_halves(nibble<2>(w), nibble<2>(h));
    r[3] = high_halves(nibble<3>(w), nibble<3>(h));
    return __builtin_bit_cast(bf16x8, r);
}

// Two 4-bit codes at bits 0 and 16 of w >> SHIFT as bf16 code + 24 and code - 23: in two's complement n ^ 8 is code + 8 and
// n ^ 7 is 7 - code, which are the upper mantissa bits of 16 (1 + (code + 8) / 16) and -16 (1 + (7 - code) / 16).
constexpr uint32_t kExcess = 0xC1B841C0u;      // (24, -23)
template <int SHIFT>
__device__ __forceinline__ uint32_t excess_pair(uint32_t w) {
    uint32_t x;
    if constexpr (SHIFT < 3) x = w << (3 - SHIFT);
    else x = w >> (SHIFT - 3);
    return (x & 0x00780078u) ^ kExcess;
}

// A word's eight codes: register i holds codes i and i + 4.
__device__ __forceinline__ bf16x8 word_to_excess(uint32_t w) {
    return __builtin_bit_cast(bf16x8, u32x4{excess_pair<0>(w), excess_pair<4>(w), excess_pair<8>(w), excess_pair<12>(w)});
}
// The low (0) or high (4) halves of eight bytes: registers (0, 2), (1, 3), (4, 6), (5, 7).
template <int HALF>
__device__ __forceinline__ bf16x8 nibbles_to_excess(uint32_t w0, uint32_t w1) {
    return __builtin_bit_cast(bf16x8, u32x4{excess_pair<HALF>(w0), excess_pair<HALF + 8>(w0), excess_pair<HALF>(w1), excess_pair<HALF + 8>(w1)});
}

// Eight fp32 values as three bf16 operands, each cut off after eight bits (exact).
__device__ __forceinline__ void split8(const float (&x)[8], bf16x8 (&out)[3]) {
    float rest[8];
    for (int i = 0; i < 8; ++i) rest[i] = x[i];
    for (int p = 0; p < 3; ++p) {
        u32x4 r;
        for (int i = 0; i < 4; ++i) r[i] = high_halves(rest[2 * i], rest[2 * i + 1]);
        for (int i = 0; i < 8; ++i) rest[i] -= __uint_as_float(__float_as_uint(rest[i]) & 0xFFFF0000u);
        out[p] = __builtin_bit_cast(bf16x8, r);
    }
}

// Eight elements of any alignment that their type has.
template <typename E>
struct Eight;
template <>
struct Eight<__bf16> {
    typedef u32x4 __attribute__((aligned(2))) any;
    u32x4 v;
    __device__ void load(const __bf16* p) { v = *reinterpret_cast<const any*>(p); }
    __device__ void clear() { v = u32x4{0, 0, 0, 0}; }
    __device__ float most() const {
        float x = 0.0f;
        for (int i = 0; i < 4; ++i) x = fmaxf(x, fmaxf(fabsf(bf16lo_to_f32(v[i])), fabsf(bf16hi_to_f32(v[i]))));
        return x;
    }
    __device__ void scale(int e) {                                  // exact, but for what falls below the smallest values
        for (int i = 0; i < 4; ++i) v[i] = high_halves(ldexpf(bf16lo_to_f32(v[i]), e), ldexpf(bf16hi_to_f32(v[i]), e));
    }
    __device__ void operand(bf16x8 (&q)[1]) const { q[0] = __builtin_bit_cast(bf16x8, v); }
    // The order of word_to_excess; returns the negative of the excess that its sum will have.
    __device__ float codes_order() {
        v = u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                  __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
        float low = 0.0f, high = 0.0f;
        for (int i = 0; i < 4; ++i) low += bf16lo_to_f32(v[i]), high += bf16hi_to_f32(v[i]);
        return 23.0f * high - 24.0f * low;
    }
};
template <>
struct Eight<float> {
    typedef f32x4 __attribute__((aligned(4))) any;
    float v[8];
    __device__ void load(const float* p) {
        for (int i = 0; i < 2; ++i) {
            const f32x4 x = reinterpret_cast<const any*>(p)[i];
            for (int j = 0; j < 4; ++j) v[4 * i + j] = x[j];
        }
    }
    __device__ void clear() {
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
    __device__ float most() const {
        float x = 0.0f;
        for (int i = 0; i < 8; ++i) x = fmaxf(x, fabsf(v[i]));
        return x;
    }
    __device__ void scale(int e) {
        for (int i = 0; i < 8; ++i) v[i] = ldexpf(v[i], e);
    }
    __device__ void operand(bf16x8 (&q)[3]) const { split8(v, q); }
};

// Four values rounded to rows of any alignment that their type has.
__device__ __forceinline__ void store_four(__bf16* p, f32x4 x) {
    typedef u32x2 __attribute__((aligned(2))) any;
    *reinterpret_cast<any*>(p) = u32x2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
}
__device__ __forceinline__ void store_four(float* p, f32x4 x) {
    typedef f32x4 __attribute__((aligned(4))) any;
    *reinterpret_cast<any*>(p) = x;
}

// a / b where the quotient is below 2^20: from a reciprocal, put right by one where that was needed (a, b < 2^31).
__device__ __forceinline__ uint32_t small_quotient(uint32_t a, uint32_t b) {
    const uint32_t q = (uint32_t)((float)a * __builtin_amdgcn_rcpf((float)b));
    const int rest = (int)(a - q * b);
    return rest < 0 ? q - 1 : rest >= (int)b ? q + 1 : q;
}

// Inclusive sums over the lanes of a wave.
__device__ __forceinline__ uint32_t scan_of_wave(uint32_t x, int lane) {
    for (int i = 1; i < 64; i *= 2) {
        const uint32_t y = __shfl_up(x, i);
        if (lane >= i) x += y;
    }
    return x;
}

template <int WORDS>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* to) {
    static_assert(WORDS == 1 || WORDS == 2 || WORDS == 4);
    if constexpr (WORDS == 4) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(p);
        for (int i = 0; i < 4; ++i) to[i] = v[i];
    } else if constexpr (WORDS == 2) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(p);
        to[0] = v[0], to[1] = v[1];
    } else {
        to[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// Visible tokens [first, n) of a request and the blocks that hold them (one at least, so that its output is written).
struct Visible {
    uint32_t first, n;
    __device__ uint32_t block() const { return first / kBlockTokens; }
    __device__ uint32_t blocks() const {
        const uint32_t end = (n + kBlockTokens - 1) / kBlockTokens;
        return end > block() ? end - block() : 1u;
    }
};

__device__ __forceinline__ Visible visible(const AttentionKernelArgs& a, int r) {
    const int32_t given = a.lengths[r];
    Visible v;
    v.n = given < 0 ? 0u : min((uint32_t)given, a.max_tokens);
    v.first = a.window > 0 && (int64_t)v.n > a.window ? v.n - (uint32_t)a.window : 0u;
    return v;
}

template <int NC, int BITS, int PARTS>
struct AttentionTraits {
    static constexpr int kDp = 32 * NC;
    static constexpr int kRow = kDp * BITS / 8;                     // bytes of a key
    static constexpr int kWordsPerChunk = BITS / 4;                 // of a lane's eight dimensions
    // chunks whose dimensions lie side by side in a lane, for loads of 16 bytes
    static constexpr int kSide = BITS == 16 ? 1 : BITS == 8 ? (NC % 2 ? 1 : 2) : NC % 4 == 0 ? 4 : NC % 2 == 0 ? 2 : 1;
    static constexpr int kKeyLoads = NC / kSide;
    static constexpr int kKeyLoadWords = kSide * kWordsPerChunk;
    // neighbouring dimensions whose value octets a lane loads together
    static constexpr int kDims = BITS == 16 ? 1 : BITS == 8 ? 2 : NC % 2 ? 2 : 4;
    static constexpr int kValueLoads = 2 * NC / kDims;
    static constexpr int kValueLoadWords = kDims * BITS / 4;
    static constexpr bool kExcess = BITS == 4 && PARTS == 1;        // codes enter as code + 24 and code - 23
    static constexpr float kUnit = BITS == 4 && !kExcess ? 16.0f : 1.0f;
    static constexpr int kProbabilityParts = 3;                     // bf16 operands of a probability times its value's scale
    // q's lower parts may be zeros: times an infinite key they are NaN where the product is an infinity, which the first part's sum
    // has by itself (a NaN in a key, or a zero in q, makes that one NaN too)
    static constexpr bool kLowApart = BITS == 16 && PARTS > 1;
    static constexpr int kTiles = 2 * NC + (kExcess ? 1 : 0);       // of the output, and the sums of its excess
};

// What a lane holds of 32 tokens.
template <int NC, int BITS, int PARTS>
struct Block {
    using Tr = AttentionTraits<NC, BITS, PARTS>;
    uint32_t k[2][NC * Tr::kWordsPerChunk];
    uint32_t v[2 * NC * Tr::kWordsPerChunk];
    float ks[8], vs[8];
    uint32_t seen;                                                  // of the tokens 8 (l / 16) + j: bit j
    bool whole;                                                     // every token of the 32 is seen
};

// Page and place in it of the two halves of 32 tokens; -1 where there is none.  The same for all lanes of a wave, and read by
// scalar loads (the table is not written while the kernel runs).
struct Halves {
    uint32_t t0;
    int32_t page[2];
    uint32_t slot[2];
};

__device__ __forceinline__ Halves look_up(const AttentionKernelArgs& a, const int32_t* table, const Visible& vis, uint32_t t0) {
    Halves h;
    h.t0 = t0;
    for (int i = 0; i < 2; ++i) {
        const uint32_t t = t0 + 16 * i, j = a.by_page.quotient(t);
        h.page[i] = t < vis.n ? (const int32_t)*(const __attribute__((address_space(4))) int32_t*)(table + j) : -1;
        h.slot[i] = t - j * a.page_size;
    }
    return h;
}

template <int NC, int BITS, int PARTS>
__device__ __forceinline__ void load_block(const AttentionKernelArgs& a, const Visible& vis, const Halves& at,
                                           const uint8_t* head, int lane, Block<NC, BITS, PARTS>& b) {
    using Tr = AttentionTraits<NC, BITS, PARTS>;
    const int m = lane & 15, quarter = lane >> 4;
    const uint32_t t0 = at.t0;
    const bool ok0 = (uint32_t)at.page[0] < a.n_pages, ok1 = (uint32_t)at.page[1] < a.n_pages;
    // a half without a page reads page 0 and is masked
    const uint32_t s0 = ok0 ? at.slot[0] : 0u, s1 = ok1 ? at.slot[1] : 0u;
    const uint8_t* block0 = head + (ok0 ? at.page[0] : 0) * a.page_stride;
    const uint8_t* block1 = head + (ok1 ? at.page[1] : 0) * a.page_stride;
    const uint32_t part = (uint32_t)a.page_size * Tr::kRow;
    b.whole = ok0 && ok1 && t0 >= vis.first && t0 + 32 <= vis.n;
    const bool key_second = m >= 8, value_second = quarter >= 2;
    {
        const uint8_t* p = (key_second ? block1 : block0) + (key_second ? s1 : s0) * Tr::kRow +
                           (8 * ((m >> 2) & 1) + (m & 3)) * Tr::kRow + quarter * Tr::kKeyLoadWords * 4;
        for (int T = 0; T < 2; ++T)
            for (int i = 0; i < Tr::kKeyLoads; ++i)
                load_words<Tr::kKeyLoadWords>(p + 4 * T * Tr::kRow + i * Tr::kKeyLoadWords * 16, &b.k[T][i * Tr::kKeyLoadWords]);
    }
    const uint8_t* block = value_second ? block1 : block0;
    const uint32_t slot = (value_second ? s1 : s0) + 8 * (quarter & 1);
    if constexpr (BITS < 16) {
        const uint8_t* p = block + 2 * part + 4 * slot;
        for (int i = 0; i < 2; ++i) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(p + 16 * i);
            const f32x4 y = *reinterpret_cast<const f32x4*>(p + 16 * i + 4 * a.page_size);
            for (int j = 0; j < 4; ++j) b.ks[4 * i + j] = x[j], b.vs[4 * i + j] = y[j];
        }
    }
    {
        const uint8_t* p = block + part + (slot / 8 * Tr::kDp + m * Tr::kDims) * BITS;
        for (int i = 0; i < Tr::kValueLoads; ++i)
            load_words<Tr::kValueLoadWords>(p + i * 16 * Tr::kDims * BITS, &b.v[i * Tr::kValueLoadWords]);
    }
    if (!b.whole) {
        const uint32_t t = t0 + 8 * quarter;
        uint32_t seen = 0;
        for (uint32_t j = 0; j < 8; ++j) seen |= (uint32_t)(t + j >= vis.first && t + j < vis.n) << j;
        b.seen = (value_second ? ok1 : ok0) ? seen : 0u;
    }
}

// less: what the scores begin with (the negative of their excess); to_log2 2^more: what brings them to powers of two, far: whether
// any lane's `more` is not 0
template <int NC, int BITS, int PARTS>
__device__ __forceinline__ void step(Block<NC, BITS, PARTS>& b, const bf16x8 (&q)[NC][PARTS], float less, float to_log2, bool far, int more,
                                     float& m, float& l, f32x4 (&o)[AttentionTraits<NC, BITS, PARTS>::kTiles]) {
    using Tr = AttentionTraits<NC, BITS, PARTS>;
    f32x4 s[2];
    for (int T = 0; T < 2; ++T) {
        f32x4 acc = {less, less, less, less}, low = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int c = 0; c < NC; ++c) {
            const uint32_t* w = &b.k[T][c * Tr::kWordsPerChunk];
            bf16x8 k;
            if constexpr (BITS == 16) k = __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
            else if constexpr (BITS == 8) k = bytes_to_bf16(w[0], w[1]);
            else if constexpr (Tr::kExcess) k = word_to_excess(w[0]);
            else k = word_to_bf16(w[0]);
            for (int p = PARTS - 1; p >= 0; --p) {
                f32x4& sum = Tr::kLowApart && p > 0 ? low : acc;
                sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[c][p], sum, 0, 0, 0);
            }
        }
        if constexpr (Tr::kLowApart)
            for (int i = 0; i < 4; ++i) acc[i] += low[i] == low[i] ? low[i] : 0.0f;
        s[T] = acc;
    }
    float x[8];
    for (int j = 0; j < 8; ++j) {
        x[j] = s[j / 4][j % 4];
        if constexpr (BITS < 16) x[j] *= b.ks[j];
        x[j] *= to_log2;
    }
    if (far) {
        for (int j = 0; j < 8; ++j) x[j] = ldexpf(x[j], more);
    }
    if (!b.whole) {
        for (int j = 0; j < 8; ++j) x[j] = b.seen >> j & 1 ? x[j] : -INFINITY;
        // what an unseen slot holds may not be a number
        if constexpr (BITS < 16) {
            for (int j = 0; j < 8; ++j) b.vs[j] = b.seen >> j & 1 ? b.vs[j] : 0.0f;
        } else {
            u32x4 mask;
            for (int i = 0; i < 4; ++i)
                mask[i] = (b.seen >> 2 * i & 1 ? 0xFFFFu : 0u) | (b.seen >> (2 * i + 1) & 1 ? 0xFFFF0000u : 0u);
            for (int i = 0; i < 8 * NC; ++i) b.v[i] &= mask[i & 3];
        }
    }
    float top = max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), max3(x[6], x[7], x[7]));
    top = max_of_quarters(top);
    if (__any(top > m + kRaise)) {
        const float now = fmaxf(m, top), base = now == -INFINITY ? 0.0f : now;
        const float keep = __builtin_amdgcn_exp2f(m - base);
        m = now;
        l *= keep;
        for (int i = 0; i < Tr::kTiles; ++i) o[i] *= keep;
    }
    const float base = m == -INFINITY ? 0.0f : m;
    float p8[8];
    for (int j = 0; j < 8; ++j) {
        const float p = __builtin_amdgcn_exp2f(x[j] - base);
        l += p;
        p8[j] = p;
        if constexpr (BITS < 16) p8[j] *= b.vs[j];
    }
    constexpr int kParts = Tr::kProbabilityParts;
    bf16x8 p[kParts];
    if constexpr (Tr::kExcess) {
        const float in_order[8] = {p8[0], p8[2], p8[1], p8[3], p8[4], p8[6], p8[5], p8[7]};
        split8(in_order, p);
        const bf16x8 excess = __builtin_bit_cast(bf16x8, u32x4{kExcess, kExcess, kExcess, kExcess});
        for (int part = kParts - 1; part >= 0; --part)
            o[2 * NC] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(excess, p[part], o[2 * NC], 0, 0, 0);
    } else {
        split8(p8, p);
    }
    for (int i = 0; i < Tr::kValueLoads; ++i) {
        const uint32_t* w = &b.v[i * Tr::kValueLoadWords];
        for (int e = 0; e < Tr::kDims; ++e) {
            bf16x8 v;
            if constexpr (BITS == 16) v = __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
            else if constexpr (BITS == 8) v = bytes_to_bf16(w[2 * e], w[2 * e + 1]);
            else if constexpr (Tr::kExcess) v = e % 2 == 0 ? nibbles_to_excess<0>(w[e], w[e + 1]) : nibbles_to_excess<4>(w[e - 1], w[e]);
            else if (e % 2 == 0) v = nibbles_to_bf16(w[e], w[e + 1]);
            else v = nibbles_to_bf16(upper_nibbles(w[e - 1]), upper_nibbles(w[e]));
            f32x4& acc = o[i * Tr::kDims + e];
            for (int part = kParts - 1; part >= 0; --part) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p[part], acc, 0, 0, 0);
        }
    }
}

// q of a lane's head as B operands.  Values of extreme size are brought near one by a power of two (which to_log2 and `more` take
// back: their product may pass the largest number where the scores do not), so that no sum on the way leaves the range of fp32.
template <typename E, int NC, int BITS, int PARTS>
__device__ __forceinline__ void load_q(const E* x, bool wanted, int D, int quarter, float scale, int exponent,
                                       bf16x8 (&q)[NC][PARTS], float& less, float& to_log2, int& more) {
    using Tr = AttentionTraits<NC, BITS, PARTS>;
    Eight<E> y[NC];
    for (int c = 0; c < NC; ++c) {
        const int d = 32 * Tr::kSide * (c / Tr::kSide) + 8 * Tr::kSide * quarter + 8 * (c % Tr::kSide);
        const bool in = wanted && d < D;                            // a row is read from its start where nothing of it is wanted
        y[c].load(x + (in ? d : 0));
        if (!in) y[c].clear();
    }
    float most = 0.0f;
    for (int c = 0; c < NC; ++c) most = fmaxf(most, y[c].most());
    most = max_of_quarters(most);
    if (__any(most > 0x1p20f || (most < 0x1p-20f && most > 0.0f))) {
        const int e = most == 0.0f || most == INFINITY ? 0 : ilogbf(most);
        for (int c = 0; c < NC; ++c) y[c].scale(-e);
        exponent += e;
    }
    more = max(exponent - kMostExponent, 0);
    // an infinity makes every score infinite or NaN: NaN for all of them, whatever the signs that it meets
    to_log2 = most == INFINITY ? NAN : ldexpf(Tr::kUnit * scale, exponent - more);
    less = 0.0f;
    for (int c = 0; c < NC; ++c) {
        if constexpr (Tr::kExcess) less += y[c].codes_order();
        y[c].operand(q[c]);
    }
    if constexpr (Tr::kExcess) less = sum_of_quarters(less);
}

template <typename E, int NC, int BITS, int PARTS>
__global__ __launch_bounds__(64, attention_waves(NC, BITS, PARTS)) void attention_kernel(AttentionKernelArgs a) {
    using Tr = AttentionTraits<NC, BITS, PARTS>;
    const int lane = threadIdx.x, quarter = lane >> 4, n = lane & 15;

    // the line of all blocks: a scan over the requests' lengths on it, `share` requests a lane
    const int share = (a.R + 63) / 64;
    uint32_t mine = 0;
    for (int i = 0; i < share; ++i)
        if (lane * share + i < a.R) mine += visible(a, lane * share + i).blocks() + kBeginCost;
    const uint32_t line = scan_of_wave(mine, lane), total = (uint32_t)__builtin_amdgcn_readlane((int)line, 63) * a.segments;
    const uint32_t chunk = max(kLeastPiece, a.by_pieces.quotient(total) + 1);
    const uint32_t piece = blockIdx.x;
    const bool by_piece = a.R * a.segments > (int)gridDim.x;        // how records are numbered
    if (by_piece && lane == 0) a.records[piece].parts = 0;          // also where there is no such piece
    if ((uint64_t)piece * chunk >= total) return;
    const uint32_t begin = piece * chunk, end = min(begin + chunk, total);

    // the request that the piece begins in: the lane whose requests hold it, then the one among those
    const uint32_t at = a.by_segments.quotient(begin);
    const int before = __popcll(__ballot(line <= at));
    int r = before * share;
    uint32_t base = before ? (uint32_t)__builtin_amdgcn_readlane((int)line, before - 1) : 0u;   // of request r, in places of one segment
    for (; share > 1; r += 64) {
        const uint32_t inner = scan_of_wave(r + lane < a.R ? visible(a, r + lane).blocks() + kBeginCost : 0u, lane) + base;
        const int under = __popcll(__ballot(inner <= at));
        if (under) base = (uint32_t)__builtin_amdgcn_readlane((int)inner, under - 1);
        if (under < 64) {
            r += under;
            break;
        }
    }

    uint32_t pos = begin, start = base * a.segments;                // of request r on the line
    for (; pos < end; ++r) {
        Visible vis = visible(a, r);
        vis.n = (uint32_t)__builtin_amdgcn_readfirstlane((int)vis.n);
        vis.first = (uint32_t)__builtin_amdgcn_readfirstlane((int)vis.first);
        const uint32_t length = vis.blocks() + kBeginCost;
        int segment = (int)small_quotient(pos - start, length);
        uint32_t from = pos - start - segment * length;
        start += a.segments * length;
        for (; segment < a.segments && pos < end; ++segment, from = 0) {
            // places [from, upto) of the segment's line; the first kBeginCost of it are no blocks
            const uint32_t upto = min(length, from + (end - pos));
            const uint32_t off = max(from, kBeginCost) - kBeginCost;
            const int count = (int)(upto - kBeginCost) - (int)off;
            const bool starts = off == 0, ends = upto == length;
            pos += upto - from;
            if (count <= 0) continue;
            const int h = segment / a.tiles, tile = segment - h * a.tiles;
            const int heads = min(kTileHeads, a.group - tile * kTileHeads), hq = h * a.group + tile * kTileHeads;
            if (starts) {
                // the pieces that hold the rest; a segment in one piece leaves nothing to join
                const uint32_t last = small_quotient(pos - upto + length - 1, chunk);
                if (lane == 0 && (!ends || !by_piece))
                    a.records[by_piece ? (int)piece : r * a.segments + segment] = {r, segment, (int32_t)piece, (int32_t)(ends ? 0 : last - piece + 1)};
            }

            // the first block, then q of the tile's heads as B operands
            const uint8_t* head = a.pages + h * a.head_stride;
            const int32_t* table = a.table + r * a.ld_table;
            uint32_t t = (uint32_t)__builtin_amdgcn_readfirstlane((int)((vis.block() + off) * kBlockTokens));
            int todo = vis.n > vis.first ? count : 0;
            asm("" : "+v"(todo));                                   // as a lane's own the loop leaves the block in its registers
            Block<NC, BITS, PARTS> b;
            if (todo > 0) load_block(a, vis, look_up(a, table, vis, t), head, lane, b);
            Halves next = look_up(a, table, vis, t += kBlockTokens);        // a block's pages are known when its turn comes
            bf16x8 q[NC][PARTS];
            float less, to_log2;
            int more;
            load_q<E, NC, BITS, PARTS>(static_cast<const E*>(a.q) + r * a.q_rs + (hq + min(n, heads - 1)) * a.q_hs, n < heads, a.D,
                                       quarter, a.scale_log2e, a.scale_exponent, q, less, to_log2, more);
            const bool far = __any(more > 0);

            f32x4 o[Tr::kTiles];
            for (int i = 0; i < Tr::kTiles; ++i) o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            float m = -INFINITY, l = 0.0f;
            while (todo > 0) {
                step<NC, BITS, PARTS>(b, q, less, to_log2, far, more, m, l, o);
                if (--todo > 0) {
                    load_block(a, vis, next, head, lane, b);
                    next = look_up(a, table, vis, t = (uint32_t)__builtin_amdgcn_readfirstlane((int)(t + kBlockTokens)));
                }
            }
            l = sum_of_quarters(l);
            if (n >= heads) continue;

            // four neighbouring dimensions at a time: j of value load i
            const bool whole = starts && ends;
            const uint32_t place = (2 * piece + (starts ? 1 : 0)) * a.rows + n;
            const float inverse = Tr::kUnit * (whole ? l == 0.0f ? 0.0f : 1.0f / l : 1.0f);
            E* to = static_cast<E*>(a.out) + r * a.o_rs + (hq + n) * a.o_hs;
            float* part = a.partial_o + (uint64_t)place * Tr::kDp;
            for (int i = 0; i < Tr::kValueLoads; ++i)
                for (int j = 0; j < Tr::kDims; ++j) {
                    const int d = (16 * i + 4 * quarter) * Tr::kDims + 4 * j;
                    f32x4 y;
                    for (int z = 0; z < 4; ++z) y[z] = o[i * Tr::kDims + (4 * j + z) % Tr::kDims][(4 * j + z) / Tr::kDims];
                    if constexpr (Tr::kExcess) y -= o[2 * NC];
                    if (!whole) *reinterpret_cast<f32x4*>(part + d) = y * inverse;
                    else if (d < a.D) store_four(to + d, l == 0.0f ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : y * inverse);
                }
            if (quarter == 0) {
                if (!whole) *reinterpret_cast<f32x2*>(a.partial_ml + 2 * (uint64_t)place) = f32x2{m, l};
                else if (a.lse) a.lse[(int64_t)r * a.Hq + hq + n] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
            }
        }
    }
}

template <int BITS>
hipError_t launch_attention(const AttentionKernelArgs& a, int chunks, bool f32, hipStream_t stream) {
    const auto launch = [&](auto e, auto parts, auto nc) {
        using E = decltype(e);
        constexpr int P = decltype(parts)::value, NC = decltype(nc)::value;
        attention_kernel<E, NC, BITS, P><<<dim3((unsigned)a.pieces), 64, 0, stream>>>(a);
    };
    const auto pick = [&](auto e, auto parts) {
        switch (chunks) {
            case 2: return launch(e, parts, std::integral_constant<int, 2>{});
            case 3: return launch(e, parts, std::integral_constant<int, 3>{});
            case 4: return launch(e, parts, std::integral_constant<int, 4>{});
            case 6: return launch(e, parts, std::integral_constant<int, 6>{});
            default: return launch(e, parts, std::integral_constant<int, 8>{});
        }
    };
    if (f32) pick(0.0f, std::integral_constant<int, 3>{});
    else pick((__bf16)0.0f, std::integral_constant<int, 1>{});
    return hipGetLastError();
}

}  // namespace gptq
