// Host interface of the products with packed weights (matmul.hip; kernels in matmul_rows.hpp, matmul_split.hpp, matmul_tile.hpp).
#pragma once

#include "gptq_common.hpp"

namespace gptq {

struct MatmulArgs {
    // activations: row r of the product is row rows[r] (or r) of X; E experts own rows [offsets[e], offsets[e + 1])
    const void* X = nullptr;
    int64_t ldx = 0, x_rows = 0;
    const int32_t* rows = nullptr;
    int64_t M = 0;
    const int32_t* offsets = nullptr;      // nullptr: one expert owns every row
    int E = 1;
    bool f32 = false;                      // X and Y are fp32 (else bf16)
    // packed weights
    const uint32_t* packed = nullptr;
    int64_t ldp = 0, p_stride = 0;
    int64_t K = 0, N = 0;                  // N: channels of the packed weight
    int bits = 4;
    const float* scales = nullptr;
    int64_t s_stride = 0;
    int groupsize = 0;                     // 0: one scale per channel
    bool swiglu = false;                   // Y = silu(first half) * second half, N / 2 columns
    void* Y = nullptr;
    int64_t ldy = 0;
    // low-rank adapters of requests (E == 1)
    const uint16_t* A = nullptr;           // n_adapters x rank x K
    const uint16_t* B = nullptr;           // n_adapters x N x rank
    int64_t lda = 0, a_stride = 0, ldb = 0, b_stride = 0;
    const float* alpha = nullptr;
    int64_t n_adapters = 0;
    int rank = 0;
    const int32_t* requests = nullptr;
    const int32_t* adapter = nullptr;
    int64_t n_requests = 0;
};

size_t matmul_workspace_bytes(bool f32, int64_t M, int64_t K, int64_t N, int64_t experts, int64_t rank);
hipError_t packed_matmul(const MatmulArgs& a, void* workspace, hipStream_t stream);

// What the kernels see.
struct MatmulKernelArgs {
    const void* X;
    int64_t ldx, x_rows;
    const int32_t* rows;
    int64_t M;
    const int32_t* offsets;
    int E;
    const uint32_t* packed;
    int64_t p_stride;
    uint32_t ldp;
    int K, N;
    int nwords;                            // words per channel
    const float* scales;
    int64_t s_stride;
    int lg_group;                          // log2 of the MFMA steps per scale (0, 1, 2; per channel 2)
    int s_row;                             // floats from one group's scales to the next (per channel 0)
    int last_group;
    void* Y;
    int64_t ldy;
    // adapters: H = alpha A x of every row, M x hrank fp32, in h_parts parts to be added (more than one only for the tile
    // kernel's runs), and the adapter of every row (-1: none)
    const float* H;
    int hrank, h_parts;
    const int32_t* row_adapter;
    const float* Z;                        // H B^T, M x N, where the tile kernel is given it ready; else nullptr
    const uint16_t* B;
    int64_t ldb, b_stride;
    int rank;
    // rows laid out for the tile kernel: PARTS x [K / 8][Mp] octets, and per row and group the sum of x times -1.5 2^-8
    const uint16_t* XT;
    const float* sums;
    int64_t Mp;
    const int32_t* tiles;                  // (expert, first row, end) of every row tile, then a negative expert
};

}  // namespace gptq
