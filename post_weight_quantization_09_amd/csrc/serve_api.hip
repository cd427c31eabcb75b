// C ABI of the serving calls: routing, products with packed weights, joining (see include/gptq.h).
#include <algorithm>

#include "matmul.hpp"
#include "route.hpp"
#include "timer.hpp"

using namespace gptq;

namespace {

bool ws_ok(const void* ws, size_t have, size_t need) {
    if (need == 0) return true;
    return ws != nullptr && (reinterpret_cast<uintptr_t>(ws) % kAlign) == 0 && have >= need;
}

bool dtype_ok(gptq_dtype_t d) { return d == GPTQ_DTYPE_F32 || d == GPTQ_DTYPE_BF16; }

constexpr int64_t kMaxTokens = (int64_t)1 << 27;      // of gptq_route: a launch has fewer than 2^32 threads
constexpr int64_t kMaxRows = (int64_t)1 << 30, kMaxK = (int64_t)1 << 22, kMaxN = (int64_t)1 << 22;
constexpr int64_t kMaxExperts = 16384, kMaxRequests = (int64_t)1 << 24, kMaxAdapters = (int64_t)1 << 24;

// The launch over tiles of 64 rows x 256 channels has fewer than 2^32 threads.
bool tiles_ok(int64_t M, int64_t N, int64_t E) {
    return ceil_div(M, E) <= 64 || (ceil_div(M, 64) + E + 3) * ceil_div(N, 256) < (int64_t)1 << 24;
}

// The checks that gptq_expert_matmul and gptq_adapter_matmul share.
bool layer_ok(const void* X, gptq_dtype_t dtype, int64_t x_rows, int64_t ldx, int64_t M, const uint32_t* packed,
              int64_t ldp, int64_t K, int64_t N, int bits, const float* scales, int64_t groupsize, int64_t width,
              const void* Y, int64_t ldy, int64_t E) {
    if (!dtype_ok(dtype) || !packed || !scales || M < 0 || M > kMaxRows || K < 1 || K > kMaxK) return false;
    if (N < 4 || N > kMaxN || bits < 2 || bits > 6 || ldp < N || ldx < K || ldy < width) return false;
    if (groupsize != 0 && groupsize != 32 && groupsize != 64 && groupsize != 128) return false;
    if (M > 0 && (!X || !Y || X == Y || x_rows < 1)) return false;
    // the kernels address an expert's words by 32-bit byte offsets
    if ((K * bits + 31) / 32 * ldp > ((int64_t)1 << 30)) return false;
    return tiles_ok(M, N, E);
}

}  // namespace

extern "C" {

size_t gptq_matmul_workspace_bytes(gptq_dtype_t dtype, int64_t M, int64_t K, int64_t N, int64_t experts,
                                   int64_t rank) {
    if (!dtype_ok(dtype) || M < 1 || M > kMaxRows || K < 1 || K > kMaxK || N < 1 || N > kMaxN) return 0;
    if (experts < 1 || experts > kMaxExperts || rank < 0 || rank > 128) return 0;
    if (!tiles_ok(M, N, experts)) return 0;
    return matmul_workspace_bytes(dtype == GPTQ_DTYPE_F32, M, K, N, experts, rank);
}

gptq_status_t gptq_route(const void* logits, gptq_dtype_t dtype, int64_t T, int64_t E, int64_t ld, int topk,
                         unsigned flags, float* weights, int32_t* experts, int32_t* offsets, int32_t* rows,
                         int32_t* positions, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dtype) || T < 0 || E < 1 || E > kRouteMaxExperts || ld < E) return GPTQ_ERR_ARG;
    if (topk < 1 || topk > kRouteMaxTopk || T > std::min(kMaxRows / topk, kMaxTokens) || !offsets) return GPTQ_ERR_ARG;
    if (flags & ~GPTQ_FLAG_RENORM) return GPTQ_ERR_ARG;
    if (T > 0 && (!logits || !weights || !experts || !rows || !positions)) return GPTQ_ERR_ARG;
    if (!ws_ok(workspace, workspace_bytes, route_workspace_bytes(T, E))) return GPTQ_ERR_WORKSPACE;
    TimerScope ts(static_cast<hipStream_t>(stream), GPTQ_TIMER_OTHER);
    return route(logits, dtype == GPTQ_DTYPE_F32, T, E, ld, topk, (flags & GPTQ_FLAG_RENORM) != 0, weights, experts,
                 offsets, rows, positions, workspace, static_cast<hipStream_t>(stream)) == hipSuccess
               ? GPTQ_OK
               : GPTQ_ERR_HIP;
}

gptq_status_t gptq_expert_matmul(const void* X, gptq_dtype_t dtype, int64_t x_rows, int64_t ldx, const int32_t* rows,
                                 int64_t M, const int32_t* offsets, int64_t E, const uint32_t* packed, int64_t ldp,
                                 int64_t p_stride, int64_t K, int64_t N, int bits, const float* scales,
                                 int64_t s_stride, int64_t groupsize, unsigned flags, void* Y, int64_t ldy,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    if (flags & ~GPTQ_FLAG_SWIGLU) return GPTQ_ERR_ARG;
    const bool swiglu = (flags & GPTQ_FLAG_SWIGLU) != 0;
    if (swiglu && N % 2 != 0) return GPTQ_ERR_ARG;
    if (!offsets || E < 1 || E > kMaxExperts || (!rows && x_rows < M)) return GPTQ_ERR_ARG;
    if (!layer_ok(X, dtype, x_rows, ldx, M, packed, ldp, K, N, bits, scales, groupsize, swiglu ? N / 2 : N, Y, ldy, E))
        return GPTQ_ERR_ARG;
    const int64_t groups = groupsize ? ceil_div(K, groupsize) : 1;
    if (E > 1 && (p_stride < (K * bits + 31) / 32 * ldp || s_stride < groups * N)) return GPTQ_ERR_ARG;
    if (M == 0) return GPTQ_OK;
    if (!ws_ok(workspace, workspace_bytes, matmul_workspace_bytes(dtype == GPTQ_DTYPE_F32, M, K, N, E, 0)))
        return GPTQ_ERR_WORKSPACE;
    MatmulArgs a;
    a.X = X; a.ldx = ldx; a.x_rows = x_rows; a.rows = rows; a.M = M;
    a.offsets = offsets; a.E = (int)E; a.f32 = dtype == GPTQ_DTYPE_F32;
    a.packed = packed; a.ldp = ldp; a.p_stride = p_stride; a.K = K; a.N = N; a.bits = bits;
    a.scales = scales; a.s_stride = s_stride; a.groupsize = (int)groupsize;
    a.swiglu = swiglu; a.Y = Y; a.ldy = ldy;
    TimerScope ts(static_cast<hipStream_t>(stream), GPTQ_TIMER_OTHER);
    return packed_matmul(a, workspace, static_cast<hipStream_t>(stream)) == hipSuccess ? GPTQ_OK : GPTQ_ERR_HIP;
}

gptq_status_t gptq_adapter_matmul(const void* X, gptq_dtype_t dtype, int64_t M, int64_t ldx, const uint32_t* packed,
                                  int64_t ldp, int64_t K, int64_t N, int bits, const float* scales, int64_t groupsize,
                                  const void* A, int64_t lda, int64_t a_stride, const void* B, int64_t ldb,
                                  int64_t b_stride, const float* alpha, int64_t n_adapters, int64_t rank,
                                  const int32_t* requests, const int32_t* adapter, int64_t n_requests, void* Y,
                                  int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
    if (!layer_ok(X, dtype, M, ldx, M, packed, ldp, K, N, bits, scales, groupsize, N, Y, ldy, 1)) return GPTQ_ERR_ARG;
    if (n_adapters < 0 || n_requests < 0 || n_requests > kMaxRequests || n_adapters > kMaxAdapters)
        return GPTQ_ERR_ARG;
    const bool lora = n_adapters > 0 && n_requests > 0;
    if (lora) {
        if (!A || !B || !alpha || !requests || !adapter || rank < 1 || rank > 128) return GPTQ_ERR_ARG;
        if (lda < K || ldb < rank) return GPTQ_ERR_ARG;
        if (n_adapters > 1 && (a_stride < rank * lda || b_stride < N * ldb)) return GPTQ_ERR_ARG;
    }
    if (M == 0) return GPTQ_OK;
    if (!ws_ok(workspace, workspace_bytes,
               matmul_workspace_bytes(dtype == GPTQ_DTYPE_F32, M, K, N, 1, lora ? rank : 0)))
        return GPTQ_ERR_WORKSPACE;
    MatmulArgs a;
    a.X = X; a.ldx = ldx; a.x_rows = M; a.M = M; a.f32 = dtype == GPTQ_DTYPE_F32;
    a.packed = packed; a.ldp = ldp; a.K = K; a.N = N; a.bits = bits;
    a.scales = scales; a.groupsize = (int)groupsize; a.Y = Y; a.ldy = ldy;
    if (lora) {
        a.A = static_cast<const uint16_t*>(A); a.lda = lda; a.a_stride = a_stride;
        a.B = static_cast<const uint16_t*>(B); a.ldb = ldb; a.b_stride = b_stride;
        a.alpha = alpha; a.n_adapters = n_adapters; a.rank = (int)rank;
        a.requests = requests; a.adapter = adapter; a.n_requests = n_requests;
    }
    TimerScope ts(static_cast<hipStream_t>(stream), GPTQ_TIMER_OTHER);
    return packed_matmul(a, workspace, static_cast<hipStream_t>(stream)) == hipSuccess ? GPTQ_OK : GPTQ_ERR_HIP;
}

gptq_status_t gptq_combine(const void* Y, gptq_dtype_t dtype, int64_t M, int64_t ldy, const int32_t* positions,
                           const float* weights, int64_t T, int topk, int64_t N, void* out, int64_t ldo, void* stream) {
    if (!dtype_ok(dtype) || M < 0 || M > kMaxRows || T < 0 || T > kMaxRows || topk < 1 || topk > kRouteMaxTopk)
        return GPTQ_ERR_ARG;
    if (N < 1 || N > kMaxN || ldy < N || ldo < N) return GPTQ_ERR_ARG;
    if (T > 0 && (!positions || !weights || !out || (M > 0 && !Y) || out == Y)) return GPTQ_ERR_ARG;
    if (T == 0) return GPTQ_OK;
    TimerScope ts(static_cast<hipStream_t>(stream), GPTQ_TIMER_OTHER);
    return combine(Y, dtype == GPTQ_DTYPE_F32, M, ldy, positions, weights, T, topk, N, out, ldo,
                   static_cast<hipStream_t>(stream)) == hipSuccess
               ? GPTQ_OK
               : GPTQ_ERR_HIP;
}

}  // extern "C"
