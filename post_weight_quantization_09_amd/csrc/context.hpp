// Rotary positions, the paged cache of keys and values and the attention over it: what their files share (rotary.hip,
// cache.hip, attention.hip; the pages' layout in include/gptq.h).
#pragma once

#include <type_traits>

#include "gptq_common.hpp"

namespace gptq {

// Two values rounded to bf16 (lo | hi << 16), by one instruction.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// T x H rows of D elements; row (t, h) at t * ts + h * hs elements.
struct HeadRows {
    void* p;
    int64_t ts, hs;
};

struct Pages {
    uint8_t* p;
    int64_t n, page_stride, head_stride;   // bytes from one page, one head to the next
    int page_size, bits;
};

// t / d = (umulhi(t, mul) + t) >> shift for t < 2^31
struct Divisor {
    uint32_t mul, shift;
    Divisor(uint32_t d = 1) : shift(0) {
        while (((uint64_t)1 << shift) < d) ++shift;
        mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - d)) / d + 1);
    }
    __device__ uint32_t quotient(uint32_t t) const { return (__umulhi(t, mul) + t) >> shift; }
};

constexpr int64_t kMaxHeadSize = 256;

// Elements that a row of D is stored with: the widths that the attention kernel is compiled for.
inline int stored_head_size(int64_t D) {
    for (int n : {64, 96, 128, 192, 256})
        if (D <= n) return n;
    return 0;
}

// Bytes of one head's part of a page.
inline int64_t cache_block_bytes(int64_t page_size, int64_t D, int bits) {
    return 2 * page_size * (stored_head_size(D) * bits / 8) + (bits < 16 ? 8 * page_size : 0);
}

hipError_t rotary(HeadRows x, bool f32, int64_t T, int H, int D, const int32_t* positions, const double* freqs, int rot,
                  float factor, bool interleaved, HeadRows y, hipStream_t stream);

hipError_t cache_write(HeadRows k, HeadRows v, bool f32, int64_t T, int H, int D, const int32_t* slots, Pages pages,
                       hipStream_t stream);
hipError_t cache_read(Pages pages, const int32_t* slots, int64_t T, int H, int D, HeadRows k, HeadRows v, bool f32,
                      hipStream_t stream);

struct AttentionArgs {
    HeadRows q, out;
    bool f32;
    int R, Hq, H, D;
    Pages pages;
    const int32_t* table;
    int64_t ld_table, max_pages;
    const int32_t* lengths;
    float scale;
    int64_t window;
    float* lse;
};

// Whether the blocks of all requests and heads can be counted in 32 bits.
bool attention_line_ok(int64_t R, int64_t Hq, int64_t H, int64_t max_tokens);
size_t attention_workspace_bytes(int64_t R, int64_t Hq, int64_t H, int64_t D);
hipError_t cache_attention(const AttentionArgs& a, void* workspace, hipStream_t stream);

}  // namespace gptq
