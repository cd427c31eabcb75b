// The launches of matmul_b2.hip .. matmul_b6.hip.
#pragma once

#include "matmul.hpp"

namespace gptq {

#define GPTQ_MATMUL_WIDTH(B)                                                                                           \
    hipError_t rows_b##B(const MatmulKernelArgs& k, bool f32, bool swiglu, hipStream_t stream);                        \
    hipError_t split_b##B(const MatmulKernelArgs& k, bool f32, int row_tiles, int ntm, bool swiglu, hipStream_t stream); \
    hipError_t tile_b##B(const MatmulKernelArgs& k, bool f32, int row_tiles, int ntm, bool swiglu, hipStream_t stream);
GPTQ_MATMUL_WIDTH(2)
GPTQ_MATMUL_WIDTH(3)
GPTQ_MATMUL_WIDTH(4)
GPTQ_MATMUL_WIDTH(5)
GPTQ_MATMUL_WIDTH(6)
#undef GPTQ_MATMUL_WIDTH

}  // namespace gptq
