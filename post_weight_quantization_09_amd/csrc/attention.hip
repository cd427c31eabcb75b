// Attention of one new token of every request over its pages.
//
// One pass over the tokens: with m the largest score so far, l = sum e^(score - m) and o = sum e^(score - m) v, a larger score
// rescales l and o by e^(old m - new m).  The waves of a workgroup take the tokens in turn and join their (m, l, o) in LDS.
#include "context.hpp"

namespace gptq {

namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct AttentionKernelArgs {
    const void* q;
    void* out;
    int64_t q_rs, q_hs, o_rs, o_hs;
    int R, Hq, H, D, Dp;
    const uint8_t* pages;
    int64_t n_pages, page_stride, head_stride;
    int page_size;
    const int32_t* table;
    int64_t ld_table, max_pages;
    const int32_t* lengths;
    float scale;
    int64_t window;
    float* lse;
};

template <typename E, int BITS>
__global__ __launch_bounds__(256) void attention_kernel(AttentionKernelArgs a) {
    __shared__ float part[4][256 + 2];
    const int hq = blockIdx.x, r = blockIdx.y, h = hq / (a.Hq / a.H);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t n = min((int64_t)max(a.lengths[r], 0), a.max_pages * a.page_size);
    const int64_t first = a.window > 0 && n > a.window ? n - a.window : 0;
    const E* q = static_cast<const E*>(a.q) + r * a.q_rs + hq * a.q_hs;
    float qv[4], o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0.0f;
    for (int i = 0; i < 4; ++i) qv[i] = lane + 64 * i < a.D ? (float)q[lane + 64 * i] * a.scale * kLog2e : 0.0f;
    for (int64_t t = first + wave; t < n; t += 4) {
        const int page = a.table[r * a.ld_table + t / a.page_size], slot = (int)(t % a.page_size);
        if ((uint32_t)page >= (uint64_t)a.n_pages) continue;
        const uint8_t* block = a.pages + page * a.page_stride + h * a.head_stride;
        const int size = a.page_size * a.Dp * BITS / 8;
        const float* scales = reinterpret_cast<const float*>(block + 2 * size);
        float sum = 0.0f, v[4];
        for (int i = 0; i < 4; ++i) {
            const int d = lane + 64 * i;
            v[i] = 0.0f;
            if (d >= a.D) continue;
            float k;
            if constexpr (BITS == 16) {
                k = (float)reinterpret_cast<const __bf16*>(block)[slot * a.Dp + d];
                v[i] = (float)reinterpret_cast<const __bf16*>(block + size)[((slot >> 3) * a.Dp + d) * 8 + (slot & 7)];
            } else if constexpr (BITS == 8) {
                k = (float)(int8_t)block[slot * a.Dp + d];
                v[i] = (float)(int8_t)block[size + ((slot >> 3) * a.Dp + d) * 8 + (slot & 7)];
            } else {
                k = (float)((int)((uint32_t)block[(slot * a.Dp + d) / 2] << (d & 1 ? 24 : 28)) >> 28);
                v[i] = (float)((int)((uint32_t)block[size + ((slot >> 3) * (a.Dp / 2) + d / 2) * 8 + (slot & 7)] << (d & 1 ? 24 : 28)) >> 28);
            }
            sum += qv[i] * k;
        }
        for (int i = 32; i; i >>= 1) sum += __shfl_xor(sum, i);
        float sv = 1.0f;
        if constexpr (BITS < 16) {
            sum *= scales[slot];
            sv = scales[a.page_size + slot];
        }
        const float top = sum == sum ? fmaxf(m, sum) : sum;
        const float base = top == -INFINITY ? 0.0f : top, keep = exp2f(m - base), p = exp2f(sum - base);
        m = top;
        l = l * keep + p;
        for (int i = 0; i < 4; ++i) o[i] = o[i] * keep + p * sv * v[i];
    }
    for (int i = 0; i < 4; ++i) part[wave][lane + 64 * i] = o[i];
    if (lane == 0) part[wave][256] = m, part[wave][257] = l;
    __syncthreads();
    float top = -INFINITY, whole = 0.0f;
    for (int w = 0; w < 4; ++w) top = part[w][256] == part[w][256] ? fmaxf(top, part[w][256]) : NAN;
    const float base = top == -INFINITY ? 0.0f : top;
    for (int w = 0; w < 4; ++w) whole += part[w][257] * exp2f(part[w][256] - base);
    if ((int)threadIdx.x < a.D) {
        float sum = 0.0f;
        for (int w = 0; w < 4; ++w) sum += part[w][threadIdx.x] * exp2f(part[w][256] - base);
        static_cast<E*>(a.out)[r * a.o_rs + hq * a.o_hs + threadIdx.x] = (E)(whole == 0.0f ? 0.0f : sum / whole);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(int64_t)r * a.Hq + hq] = whole == 0.0f ? -INFINITY : top * kLn2 + logf(whole);
}

}  // namespace

size_t attention_workspace_bytes(int64_t R, int64_t Hq, int64_t H, int64_t D) { return kAlign; }

hipError_t cache_attention(const AttentionArgs& a, void* workspace, hipStream_t stream) {
    AttentionKernelArgs k{a.q.p, a.out.p, a.q.ts, a.q.hs, a.out.ts, a.out.hs, a.R, a.Hq, a.H, a.D, stored_head_size(a.D),
                          a.pages.p, a.pages.n, a.pages.page_stride, a.pages.head_stride, a.pages.page_size,
                          a.table, a.ld_table, a.max_pages, a.lengths, a.scale, a.window, a.lse};
    auto pick = [&](auto e) {
        using E = decltype(e);
        return a.pages.bits == 16 ? attention_kernel<E, 16> : a.pages.bits == 8 ? attention_kernel<E, 8> : attention_kernel<E, 4>;
    };
    (a.f32 ? pick(0.0f) : pick((__bf16)0.0f))<<<dim3((unsigned)a.Hq, (unsigned)a.R), 256, 0, stream>>>(k);
    return hipGetLastError();
}

}  // namespace gptq
