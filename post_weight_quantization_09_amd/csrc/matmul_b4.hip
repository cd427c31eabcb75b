// The packed products for 4-bit codes (one file per width, so that they compile side by side).
#include "matmul_launch.hpp"
#include "matmul_split.hpp"
#include "matmul_tile.hpp"

namespace gptq {

hipError_t rows_b4(const MatmulKernelArgs& k, bool f32, bool swiglu, hipStream_t stream) {
    return launch_rows<4>(k, f32, swiglu, stream);
}

hipError_t split_b4(const MatmulKernelArgs& k, bool f32, int row_tiles, int ntm, bool swiglu, hipStream_t stream) {
    return launch_split<4>(k, f32, row_tiles, ntm, swiglu, stream);
}

hipError_t tile_b4(const MatmulKernelArgs& k, bool f32, int row_tiles, int ntm, bool swiglu, hipStream_t stream) {
    return launch_tile<4>(k, f32, row_tiles, ntm, swiglu, stream);
}

}  // namespace gptq
