// The launches of matmul_b2.hip .. matmul_b6.hip and adapter.hip.
#pragma once

#include "matmul.hpp"

namespace gptq {

#define GPTQ_MATMUL_WIDTH(B)                                                                                       \
    hipError_t rows_b##B(const MatmulKernelArgs& k, bool f32, int row_tiles, bool swiglu, hipStream_t stream);     \
    hipError_t tile_b##B(const MatmulKernelArgs& k, bool f32, int row_tiles, int ntm, bool swiglu, hipStream_t stream);
GPTQ_MATMUL_WIDTH(2)
GPTQ_MATMUL_WIDTH(3)
GPTQ_MATMUL_WIDTH(4)
GPTQ_MATMUL_WIDTH(5)
GPTQ_MATMUL_WIDTH(6)
#undef GPTQ_MATMUL_WIDTH

// H = alpha (A x) of every row and the rows' adapters (adapter.hip).
hipError_t adapter_shrink(const MatmulArgs& a, float* H, int hrank, int32_t* row_adapter, hipStream_t stream);

}  // namespace gptq
