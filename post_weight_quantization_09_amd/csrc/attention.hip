// Attention of new tokens over their pages: the launch, and the join of sums that several workgroups hold
// (kernels in attention_kernel.hpp).
#include <algorithm>

#include "attention.hpp"

namespace gptq {

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// A wave joins one query head of the segment that begins in workgroup blockIdx.x and ends in a later one.
template <typename E>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionKernelArgs a, int Dp) {
    const AttentionRecord rec = a.records[blockIdx.x];
    if (rec.request < 0) return;
    const int lane = threadIdx.x & 63, row = blockIdx.y * 4 + (threadIdx.x >> 6);
    const int h = rec.segment / a.tiles, tile = rec.segment - h * a.tiles;
    const int heads = min(kTileHeads, a.group - tile * kTileHeads), hq = h * a.group + tile * kTileHeads + row;
    if (row >= heads) return;
    const int first = blockIdx.x, parts = rec.last - first + 1;
    const auto place = [&](int i) { return (2 * (int64_t)(first + i) + (i == 0 ? 1 : 0)) * a.rows + row; };
    float top = -INFINITY;
    for (int i = lane; i < parts; i += 64) top = fmaxf(top, a.partial_ml[place(i) * 2]);
    for (int i = 32; i; i >>= 1) top = fmaxf(top, __shfl_xor(top, i));
    const float from = top == -INFINITY ? 0.0f : top;
    float whole = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < parts; ++i) {
        const int64_t p = place(i);
        const float keep = __builtin_amdgcn_exp2f(a.partial_ml[p * 2] - from);
        whole += keep * a.partial_ml[p * 2 + 1];
        for (int z = 0; z < 4; ++z)
            if (lane + 64 * z < Dp) o[z] += keep * a.partial_o[p * Dp + lane + 64 * z];
    }
    E* to = static_cast<E*>(a.out) + rec.request * a.o_rs + hq * a.o_hs;
    for (int z = 0; z < 4; ++z)
        if (lane + 64 * z < a.D) to[lane + 64 * z] = (E)(whole == 0.0f ? 0.0f : o[z] / whole);
    if (a.lse && lane == 0) a.lse[(int64_t)rec.request * a.Hq + hq] = whole == 0.0f ? -INFINITY : top * kLn2 + logf(whole);
}

constexpr int kWorkgroups = 1024;

int rows_of(int64_t Hq, int64_t H) { return (int)std::min<int64_t>(Hq / H, kTileHeads); }

void carve(Carver& c, AttentionKernelArgs& k, int Dp) {
    k.records = c.take<AttentionRecord>(kWorkgroups);
    k.partial_ml = c.take<float>((size_t)2 * kWorkgroups * k.rows * 2);
    k.partial_o = c.take<float>((size_t)2 * kWorkgroups * k.rows * Dp);
}

}  // namespace

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
    while (((uint64_t)1 << k.page_shift) < (uint64_t)k.page_size) ++k.page_shift;
    k.page_mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << k.page_shift) - k.page_size)) / k.page_size + 1);
    k.table = a.table, k.ld_table = a.ld_table;
    k.max_tokens = (uint32_t)(a.max_pages * a.pages.page_size);
    k.lengths = a.lengths;
    k.scale_log2e = a.scale * kLog2e;
    k.window = a.window;
    k.R = a.R, k.Hq = a.Hq, k.H = a.H, k.D = a.D, k.group = a.Hq / a.H;
    k.tiles = (int)ceil_div(k.group, kTileHeads), k.segments = a.H * k.tiles;
    k.rows = rows_of(a.Hq, a.H);
    Carver c(workspace);
    carve(c, k, Dp);
    const hipError_t e = a.pages.bits == 16  ? launch_attention<16>(k, Dp / 32, a.f32, kWorkgroups, stream)
                         : a.pages.bits == 8 ? launch_attention<8>(k, Dp / 32, a.f32, kWorkgroups, stream)
                                             : launch_attention<4>(k, Dp / 32, a.f32, kWorkgroups, stream);
    if (e != hipSuccess) return e;
    const dim3 grid(kWorkgroups, (unsigned)ceil_div(k.rows, 4));
    if (a.f32) attention_join_kernel<float><<<grid, 256, 0, stream>>>(k, Dp);
    else attention_join_kernel<__bf16><<<grid, 256, 0, stream>>>(k, Dp);
    return hipGetLastError();
}

}  // namespace gptq
