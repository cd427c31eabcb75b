// Host interface of routing and joining (see route.hip).
#pragma once

#include "gptq_common.hpp"

namespace gptq {

constexpr int64_t kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopk = 32;

size_t route_workspace_bytes(int64_t T, int64_t E);

hipError_t route(const void* logits, bool f32, int64_t T, int64_t E, int64_t ld, int topk, bool renorm, float* weights,
                 int32_t* experts, int32_t* offsets, int32_t* rows, int32_t* positions, void* workspace,
                 hipStream_t stream);

hipError_t combine(const void* Y, bool f32, int64_t M, int64_t ldy, const int32_t* positions, const float* weights,
                   int64_t T, int topk, int64_t N, void* out, int64_t ldo, hipStream_t stream);

}  // namespace gptq
