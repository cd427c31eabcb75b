// The inner half of the low-rank adapters: H[r] = alpha_a (A_a x_r) for every row r, a the adapter of r's request.
//
// What bounds it: for single tokens, the bytes of the adapters in use (rank x K of each) and latency; for prompts, the
// rows' bytes.  A workgroup takes 16 rows of one request at a time and the whole rank; its eight waves split K (each
// 32-k step one matrix product per 16 ranks: lane l holds row l % 16 and, of A, rank l % 16, eight consecutive k each,
// straight from memory) and the partial sums are joined in LDS in a fixed order.  Every request gets `slices`
// workgroups, so that the launch does not depend on the lengths, which only the device knows.  H stays in fp32.
#include <algorithm>

#include "matmul_launch.hpp"
#include "packed_frag.hpp"

namespace gptq {

namespace {

constexpr int kShrinkWaves = 8;

struct ShrinkArgs {
    const void* X;
    int64_t ldx, M, K;
    const uint16_t* A;
    int64_t lda, a_stride;
    const float* alpha;
    int64_t n_adapters;
    int rank, hrank;
    const int32_t* requests;
    const int32_t* adapter;
    int64_t n_requests;
    float* H;
    int32_t* row_adapter;
};

template <int PARTS, int NR>
__global__ __launch_bounds__(64 * kShrinkWaves) void shrink_kernel(ShrinkArgs p) {
    __shared__ float part[kShrinkWaves][NR * 4][64];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t req = blockIdx.x;
    if (req == p.n_requests) {                       // rows of no request
        if (blockIdx.y) return;
        int64_t head = p.requests[0], tail = p.requests[p.n_requests];
        head = head < 0 ? 0 : head > p.M ? p.M : head;
        tail = tail < head ? head : tail > p.M ? p.M : tail;
        for (int64_t r = tid; r < head; r += 64 * kShrinkWaves) p.row_adapter[r] = -1;
        for (int64_t r = tail + tid; r < p.M; r += 64 * kShrinkWaves) p.row_adapter[r] = -1;
        return;
    }
    int64_t lo = p.requests[req], hi = p.requests[req + 1];
    lo = lo < 0 ? 0 : lo;
    hi = hi > p.M ? p.M : hi;
    int a = p.adapter[req];
    if (a < 0 || a >= p.n_adapters) a = -1;
    const int64_t step = 16 * (int64_t)gridDim.y;
    for (int64_t r0 = lo + 16 * (int64_t)blockIdx.y; r0 < hi; r0 += step) {
        if (tid < 16 && r0 + tid < hi) p.row_adapter[r0 + tid] = a;
        if (a < 0) continue;
        int64_t r = r0 + (lane & 15);
        if (r >= hi) r = hi - 1;
        const char* xrow = static_cast<const char*>(p.X) + r * p.ldx * (PARTS == 1 ? 2 : 4);
        const uint16_t* arow[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            int rk = 16 * n + (lane & 15);
            if (rk >= p.rank) rk = p.rank - 1;       // ranks past the end are not stored
            arow[n] = p.A + a * p.a_stride + rk * p.lda;
        }
        f32x4 acc[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) acc[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int64_t k = wave * kStepK; k < p.K; k += kShrinkWaves * kStepK) {
            u32x4 x[PARTS], b[1];
            load_octet<PARTS>(xrow, k + 8 * q, p.K, x);
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                load_octet<1>(arow[n], k + 8 * q, p.K, b);
#pragma unroll
                for (int i = 0; i < PARTS; ++i) acc[n] = mfma16(x[i], __builtin_bit_cast(bf16x8, b[0]), acc[n]);
            }
        }
        __syncthreads();                             // the previous rows' partials have been read
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[wave][n * 4 + i][lane] = acc[n][i];
        __syncthreads();
        for (int v = wave; v < NR * 4; v += kShrinkWaves) {
            float s = 0.f;
#pragma unroll
            for (int u = 0; u < kShrinkWaves; ++u) s += part[u][v][lane];
            const int64_t row = r0 + 4 * q + (v & 3);
            const int rk = 16 * (v >> 2) + (lane & 15);
            if (row < hi && rk < p.hrank) p.H[row * p.hrank + rk] = rk < p.rank ? s * p.alpha[a] : 0.f;
        }
    }
}

}  // namespace

hipError_t adapter_shrink(const MatmulArgs& a, float* H, int hrank, int32_t* row_adapter, hipStream_t stream) {
    ShrinkArgs p;
    p.X = a.X; p.ldx = a.ldx; p.M = a.M; p.K = a.K;
    p.A = a.A; p.lda = a.lda; p.a_stride = a.a_stride;
    p.alpha = a.alpha; p.n_adapters = a.n_adapters;
    p.rank = a.rank; p.hrank = hrank;
    p.requests = a.requests; p.adapter = a.adapter; p.n_requests = a.n_requests;
    p.H = H; p.row_adapter = row_adapter;
    // Workgroups per request: about 1024 in all, no more than the longest request could use.
    const int64_t slices = std::max<int64_t>(1, std::min<int64_t>(ceil_div(a.M, 16), 1024 / std::max<int64_t>(1, a.n_requests)));
    const dim3 grid((unsigned)(a.n_requests + 1), (unsigned)slices), block(64 * kShrinkWaves);
#define GPTQ_SHRINK(PARTS, NR) hipLaunchKernelGGL((shrink_kernel<PARTS, NR>), grid, block, 0, stream, p)
    if (a.f32) {
        if (a.rank <= 16) GPTQ_SHRINK(3, 1);
        else if (a.rank <= 32) GPTQ_SHRINK(3, 2);
        else if (a.rank <= 64) GPTQ_SHRINK(3, 4);
        else GPTQ_SHRINK(3, 8);
    } else {
        if (a.rank <= 16) GPTQ_SHRINK(1, 1);
        else if (a.rank <= 32) GPTQ_SHRINK(1, 2);
        else if (a.rank <= 64) GPTQ_SHRINK(1, 4);
        else GPTQ_SHRINK(1, 8);
    }
#undef GPTQ_SHRINK
    return hipGetLastError();
}

}  // namespace gptq
