// Attention of new tokens over their pages: the launch, and the join of sums that several workgroups hold
// (kernels in attention_kernel.hpp).
#include <algorithm>
#include <cmath>

#include "attention.hpp"

namespace gptq {

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// Up to this many parts a workgroup joins all query heads of a segment, Dp / 4 threads each, which weigh the parts for
// themselves; beyond it each of the workgroups along y has one head, and each along z a slice of its dimensions.  Whole calls with
// 2, 4, 8 and 16: 256 requests of 1950 tokens in 16 bits 207, 199, 199, 199 us; 32 ragged ones of up to 1024 17.0, 17.0, 17.0, 19.2;
// 16 of 100 under a wide table 12.6, 10.2, 10.2, 10.2.
constexpr int kFewParts = 4, kThreads = 256;

template <typename E>
__device__ __forceinline__ void write_joined(const AttentionKernelArgs& a, const AttentionRecord& rec, int hq, int d, f32x4 sum,
                                             float top, float whole) {
    if (d >= a.D) return;
    E* to = static_cast<E*>(a.out) + rec.request * a.o_rs + hq * a.o_hs + d;
    const float inverse = 1.0f / whole;
    for (int z = 0; z < 4; ++z) to[z] = (E)(whole == 0.0f ? 0.0f : sum[z] * inverse);
    if (a.lse && d == 0) a.lse[(int64_t)rec.request * a.Hq + hq] = whole == 0.0f ? -INFINITY : top * kLn2 + logf(whole);
}

template <typename E>
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttentionKernelArgs a, int Dp) {
    __shared__ float weights[kMaxPieces], most[kThreads / 64], wholes[kThreads / 64];
    __shared__ f32x4 sums[kThreads];
    const AttentionRecord rec = a.records[blockIdx.x];
    const int tid = threadIdx.x, wave = tid >> 6;
    const bool few = rec.parts <= kFewParts;
    if (rec.parts == 0 || (few && blockIdx.y + blockIdx.z > 0)) return;
    const int h = rec.segment / a.tiles, tile = rec.segment - h * a.tiles;
    const int heads = min(kTileHeads, a.group - tile * kTileHeads), hq = h * a.group + tile * kTileHeads;
    const auto slot = [&](int i) { return (uint64_t)((2 * (rec.first + i) + (i == 0 ? 1 : 0)) * a.rows); };
    const int quads = Dp / 4 / (few ? 1 : (int)gridDim.z), at_once = kThreads / quads, line = tid / quads;
    const int quad = tid - line * quads + (few ? 0 : (int)blockIdx.z * quads);
    if (few) {
        for (int row = line; row < heads && line < at_once; row += at_once) {
            float top = -INFINITY, whole = 0.0f;
            for (int p = 0; p < rec.parts; ++p) top = fmaxf(top, a.partial_ml[(slot(p) + row) * 2]);
            const float ref = top == -INFINITY ? 0.0f : top;
            f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
            for (int p = 0; p < rec.parts; ++p) {
                const f32x2 ml = *reinterpret_cast<const f32x2*>(a.partial_ml + (slot(p) + row) * 2);
                const float keep = __builtin_amdgcn_exp2f(ml[0] - ref);
                whole += keep * ml[1];
                sum += keep * *reinterpret_cast<const f32x4*>(a.partial_o + (slot(p) + row) * Dp + 4 * quad);
            }
            write_joined<E>(a, rec, hq + row, 4 * quad, sum, top, whole);
        }
        return;
    }
    const int row = blockIdx.y;
    if (row >= heads) return;
    const auto place = [&](int i) { return slot(i) + row; };
    float top = -INFINITY;
    for (int p = tid; p < rec.parts; p += kThreads) {
        const float m = a.partial_ml[place(p) * 2];
        weights[p] = m;
        top = fmaxf(top, m);
    }
    for (int i = 32; i; i >>= 1) top = fmaxf(top, __shfl_xor(top, i));
    if ((tid & 63) == 0) most[wave] = top;
    __syncthreads();
    for (int w = 0; w < kThreads / 64; ++w) top = fmaxf(top, most[w]);
    const float ref = top == -INFINITY ? 0.0f : top;
    float whole = 0.0f;
    for (int p = tid; p < rec.parts; p += kThreads) {
        const float keep = __builtin_amdgcn_exp2f(weights[p] - ref);
        whole += keep * a.partial_ml[place(p) * 2 + 1];
        weights[p] = keep;
    }
    for (int i = 32; i; i >>= 1) whole += __shfl_xor(whole, i);
    if ((tid & 63) == 0) wholes[wave] = whole;
    __syncthreads();
    whole = 0.0f;
    for (int w = 0; w < kThreads / 64; ++w) whole += wholes[w];

    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    if (line < at_once) {
#pragma unroll 8
        for (int p = line; p < rec.parts; p += at_once)
            sum += weights[p] * *reinterpret_cast<const f32x4*>(a.partial_o + place(p) * Dp + 4 * quad);
    }
    sums[tid] = sum;
    __syncthreads();
    if (tid < quads) {
        for (int i = 1; i < at_once; ++i) sum += sums[tid + i * quads];
        write_joined<E>(a, rec, hq + row, 4 * quad, sum, top, whole);
    }
}

int rows_of(int64_t Hq, int64_t H) { return (int)std::min<int64_t>(Hq / H, kTileHeads); }

void carve(Carver& c, AttentionKernelArgs& k, int Dp) {
    const size_t pieces = most_pieces(Dp / 32);
    k.records = c.take<AttentionRecord>(pieces);
    k.partial_ml = c.take<float>(2 * pieces * k.rows * 2);
    k.partial_o = c.take<float>(2 * pieces * k.rows * Dp);
}

}  // namespace

bool attention_line_ok(int64_t R, int64_t Hq, int64_t H, int64_t max_tokens) {
    return R * (max_tokens / kBlockTokens + 8) * H * ceil_div(Hq / H, kTileHeads) < kMaxLine;
}

size_t attention_workspace_bytes(int64_t R, int64_t Hq, int64_t H, int64_t D) {
    AttentionKernelArgs k{};
    k.rows = rows_of(Hq, H);
    Carver c(nullptr);
    carve(c, k, stored_head_size(D));
    return c.bytes();
}

hipError_t cache_attention(const AttentionArgs& a, void* workspace, hipStream_t stream) {
    const int Dp = stored_head_size(a.D);
    AttentionKernelArgs k{};
    k.q = a.q.p, k.q_rs = a.q.ts, k.q_hs = a.q.hs;
    k.out = a.out.p, k.o_rs = a.out.ts, k.o_hs = a.out.hs;
    k.lse = a.lse;
    k.pages = a.pages.p, k.page_stride = a.pages.page_stride, k.head_stride = a.pages.head_stride;
    k.n_pages = (uint32_t)a.pages.n, k.page_size = a.pages.page_size;
    k.table = a.table, k.ld_table = a.ld_table;
    k.max_tokens = (uint32_t)(a.max_pages * a.pages.page_size);
    k.lengths = a.lengths;
    k.scale_log2e = std::frexp(a.scale, &k.scale_exponent) * kLog2e;
    k.window = a.window;
    k.R = a.R, k.Hq = a.Hq, k.H = a.H, k.D = a.D, k.group = a.Hq / a.H;
    k.tiles = (int)ceil_div(k.group, kTileHeads), k.segments = a.H * k.tiles;
    k.rows = rows_of(a.Hq, a.H);
    // no more pieces than the table's pages could fill
    const int64_t places = (int64_t)a.R * k.segments * (k.max_tokens / kBlockTokens + 2 + kBeginCost);
    const int pieces = (int)std::min<int64_t>(attention_pieces(Dp / 32, a.pages.bits, a.f32 ? 3 : 1), ceil_div(places, kLeastPiece));
    k.pieces = pieces;
    k.by_page = Divisor((uint32_t)k.page_size), k.by_segments = Divisor((uint32_t)k.segments);
    k.by_pieces = Divisor((uint32_t)pieces);
    Carver c(workspace);
    carve(c, k, Dp);
    const hipError_t e = a.pages.bits == 16  ? launch_attention<16>(k, Dp / 32, a.f32, stream)
                         : a.pages.bits == 8 ? launch_attention<8>(k, Dp / 32, a.f32, stream)
                                             : launch_attention<4>(k, Dp / 32, a.f32, stream);
    if (e != hipSuccess) return e;
    // one record per segment where that is not more than one per piece
    // Few rows of long requests have hundreds of parts each: a row goes to four workgroups (131072 tokens: 10.3 us without,
    // 7.9 with; one workgroup of 1024 threads for a row the same).  Whole calls without and with, 32 query heads on 8 of 128: one
    // request of 8192 tokens 14.9 and 15.5 us, of 16384 19.2 and 18.0, of 131072 66.3 and 63.5; ragged ones of up to 16384, 8 of
    // them 30.5 and 30.7, 32 (1024 rows) 76.4 and 79.1; 64 of up to 8192 92 and 98.  The lengths are on the device and the
    // table's width stands for them: 16 requests of 3000 tokens under a table of 131072 take 26.3 where 24.8 would do.
    const unsigned segments = (unsigned)std::min<int64_t>((int64_t)a.R * k.segments, pieces);
    const dim3 grid(segments, (unsigned)k.rows, segments * k.rows <= 512 && k.max_tokens >= 16384 ? 4 : 1);
    if (a.f32) attention_join_kernel<float><<<grid, kThreads, 0, stream>>>(k, Dp);
    else attention_join_kernel<__bf16><<<grid, kThreads, 0, stream>>>(k, Dp);
    return hipGetLastError();
}

}  // namespace gptq
