// The attention's kernels for a cache of 8 bits.
#include <type_traits>

#include "attention_kernel.hpp"

namespace gptq {

template hipError_t launch_attention<8>(const AttentionKernelArgs&, int, bool, hipStream_t);

}  // namespace gptq
