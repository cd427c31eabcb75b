// What the attention's host code (attention.hip) and its kernels (attention_kernel.hpp, one file per width of the cache)
// share.
#pragma once

#include "context.hpp"

namespace gptq {

constexpr int kBlockTokens = 32;        // tokens of a wave's step: the K of the second product
constexpr int kTileHeads = 16;          // query heads of a step: the N of both products

// A segment's length on the line of all work: its blocks, and what beginning with it costs beside them (places before its blocks,
// at which nothing is done), so that waves with many segments get fewer blocks.
constexpr uint32_t kBeginCost = 1;      // 32 ragged requests of up to 1024: 17.8 us with 3, 16.8 with 1; 256 of 1900: 206 with 6, 204 with 1
constexpr uint32_t kLeastPiece = 2;     // places of a wave's piece

// A segment (a request and up to 16 query heads of one key head) whose sums several pieces hold, from `first` on.
struct AttentionRecord {
    int32_t request, segment, first, parts;     // parts 0: nothing to join
};

struct AttentionKernelArgs {
    const void* q;
    void* out;
    int64_t q_rs, q_hs, o_rs, o_hs;
    float* lse;
    const uint8_t* pages;
    int64_t page_stride, head_stride;
    uint32_t n_pages;
    int page_size;
    Divisor by_page, by_segments, by_pieces;
    const int32_t* table;
    int64_t ld_table;
    uint32_t max_tokens;                // of the table's columns
    const int32_t* lengths;
    float scale_log2e;                  // scale log2 e is scale_log2e 2^scale_exponent, scale_log2e of size one
    int scale_exponent;
    int64_t window;
    int R, Hq, H, D, group;             // group = Hq / H query heads share a key head
    int tiles, segments;                // per key head and per request
    int pieces;                         // workgroups of the launch
    float* partial_o;                   // two slots per piece (ends and begins there), rows x Dp
    float* partial_ml;                  // rows x 2
    int rows;                           // of a slot: min(group, 16)
    AttentionRecord* records;
};

// Waves of a SIMD that the registers are laid out for (512 among them; three waves have 168 each), and pieces of a launch: one
// for each of the 256 CUs' waves.  Measured both ways: heads of 256 in 16 bits 59 us with one wave, 78 with two, which spill; heads
// of 128 in 4 bits 48 with three, 57 with two; of 64 in 8 bits 66 with three, 76 with two, 65 with four (and a third more partial
// sums to join); of 128 in 16 bits 203 with two, 208 with three.
constexpr int attention_waves(int chunks, int bits, int parts) {
    if (parts == 1) return bits == 16 && chunks == 8 ? 1 : chunks <= (bits == 16 ? 3 : 4) ? 3 : 2;
    return chunks <= 4 ? 2 : 1;
}
constexpr int attention_pieces(int chunks, int bits, int parts) { return 1024 * attention_waves(chunks, bits, parts); }

// The most pieces of any width of the cache and type of the rows.
constexpr int most_pieces(int chunks) { return attention_pieces(chunks, 4, 1); }
constexpr int kMaxPieces = most_pieces(4);
constexpr int64_t kMaxLine = (int64_t)1 << 31;  // places

// chunks: stored head size / 32.
template <int BITS>
hipError_t launch_attention(const AttentionKernelArgs& a, int chunks, bool f32, hipStream_t stream);

}  // namespace gptq
