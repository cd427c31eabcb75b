// Product of a few rows with packed weights: the single tokens of a decode step, an expert with few rows.
//
// What bounds it: the packed words are read once from HBM; for up to 16 rows per expert there are at most 32 operations
// per weight, far below what the matrix cores do in the time of its half byte.  So one workgroup owns 16 NT channels of
// one expert over all K, its W waves take the 128-k chunks in turn (each wave's words come straight into registers as
// MFMA operands, the next chunks' loads in flight while one is multiplied), and the W partial sums are joined in LDS in
// a fixed order: no second launch, no partials in memory, the same bits every time.  More than 16 rows loop.
// Measured: 16 rows of 8 experts x 28672 gated channels x 4096, 4 bits: 353 MB in 83 us, 4.3 TB/s (read
// once, by the counters); one row x 4096 x 4096: 7.6 us, latency.
#pragma once

#include "matmul.hpp"
#include "packed_frag.hpp"

namespace gptq {

// The rows [lo, hi) of expert e, clamped to [0, M].
__device__ __forceinline__ void expert_rows(const MatmulKernelArgs& p, int e, int64_t& lo, int64_t& hi) {
    if (!p.offsets) {
        lo = 0;
        hi = p.M;
        return;
    }
    const int64_t a = p.offsets[e], b = p.offsets[e + 1];
    lo = a < 0 ? 0 : a;
    hi = b > p.M ? p.M : b;
}

// The row of X behind product row r, or -1 where the caller's index is out of range (such a row is zero).
__device__ __forceinline__ int64_t source_row(const MatmulKernelArgs& p, int64_t r) {
    if (!p.rows) return r;
    const int64_t s = p.rows[r];
    return s >= 0 && s < p.x_rows ? s : -1;
}

// Writes NV consecutive values of a row, fp32 or bf16 (rounded to nearest even: the product's only rounding).
template <int PARTS, int NV>
__device__ __forceinline__ void store_values(void* Y, int64_t at, const float (&v)[NV]) {
    if constexpr (PARTS == 1) {
        __bf16* y = static_cast<__bf16*>(Y) + at;
        typedef __attribute__((ext_vector_type(NV))) __bf16 vec_t;
        typedef vec_t __attribute__((aligned(2))) vec_a2;
        vec_t t;
#pragma unroll
        for (int i = 0; i < NV; ++i) t[i] = (__bf16)v[i];
        *reinterpret_cast<vec_a2*>(y) = t;
    } else {
        float* y = static_cast<float*>(Y) + at;
        typedef __attribute__((ext_vector_type(NV))) float vec_t;
        typedef vec_t __attribute__((aligned(4))) vec_a4;
        vec_t t;
#pragma unroll
        for (int i = 0; i < NV; ++i) t[i] = v[i];
        *reinterpret_cast<vec_a4*>(y) = t;
    }
}

// Rows of no expert, [0, offsets[0]) and [offsets[E], M): zero, columns [c0, c0 + cols).
template <int PARTS>
__device__ __forceinline__ void zero_outside(const MatmulKernelArgs& p, int64_t c0, int64_t cols, int64_t width,
                                             int threads) {
    if (!p.offsets) return;
    int64_t head = p.offsets[0], tail = p.offsets[p.E];
    head = head < 0 ? 0 : head > p.M ? p.M : head;
    tail = tail < head ? head : tail > p.M ? p.M : tail;
    const int64_t n = head + p.M - tail, w = cols < width - c0 ? cols : width - c0;
    for (int64_t i = threadIdx.x; i < n * w; i += threads) {
        int64_t r = i / w;
        if (r >= head) r += tail - head;
        const float z[1] = {0.f};
        store_values<PARTS, 1>(p.Y, r * p.ldy + c0 + i % w, z);
    }
}

// NT neighbouring words of one row of the packed weight (at lane's channels), as one load.
// (a uniform address and a 32-bit offset of the lane: the load takes both as they are)
template <int NT>
struct WordLoad;
template <>
struct WordLoad<4> {
    static __device__ __forceinline__ void run(const uint32_t* row, uint32_t off, uint32_t (&w)[4]) {
        const u32x4 v = *reinterpret_cast<const u32x4_a4*>(reinterpret_cast<const char*>(row) + 4u * off);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = v[j];
    }
};
template <>
struct WordLoad<2> {
    static __device__ __forceinline__ void run(const uint32_t* row, uint32_t off, uint32_t (&w)[2]) {
        const u32x2 v = *reinterpret_cast<const u32x2_a4*>(reinterpret_cast<const char*>(row) + 4u * off);
        w[0] = v[0];
        w[1] = v[1];
    }
};

// Where a lane's NT channels are.  Plain: NT neighbours.  GATED: NT / 2 gate channels and the NT / 2 up channels N / 2
// further.  At the right edge the lane's base moves left so that its loads stay inside the row; lanes that share
// channels that way compute and write the same values.
template <int NT, bool GATED>
struct LaneChannels {
    static constexpr int kRun = GATED ? NT / 2 : NT;
    uint32_t c0;       // first channel (and first output column)
    uint32_t half;
    __device__ __forceinline__ LaneChannels(int tile0, int lane, int N) {
        half = GATED ? N / 2 : 0;
        const int width = GATED ? N / 2 : N;
        const int c = tile0 + kRun * (lane & 15);
        c0 = c > width - kRun ? width - kRun : c;
    }
    // NT words (or scales) of one row: `row` is uniform, `off` the lane's own offset into it (c0, or c0 and some rows)
    __device__ __forceinline__ void words(const uint32_t* row, uint32_t off, uint32_t (&w)[NT]) const {
        if constexpr (GATED) {
            uint32_t a[kRun], b[kRun];
            WordLoad<kRun>::run(row, off, a);
            WordLoad<kRun>::run(row + half, off, b);
#pragma unroll
            for (int j = 0; j < kRun; ++j) { w[j] = a[j]; w[kRun + j] = b[j]; }
        } else {
            WordLoad<NT>::run(row, off, w);
        }
    }
    __device__ __forceinline__ uint32_t channel(int j) const { return j < kRun ? c0 + j : half + c0 + (j - kRun); }
};

// y[j] += sum_k H[r][k] B_a[channel j][k] for one row: the adapter's own term where a row stands for itself (single
// tokens, each with an adapter of its own).
template <int NT, bool GATED>
__device__ __forceinline__ void add_adapter_row(const MatmulKernelArgs& p, int64_t r, const LaneChannels<NT, GATED>& ch,
                                                float (&y)[NT]) {
    const int a = p.row_adapter[r];
    if (a < 0) return;
    const float* h = p.H + r * p.hrank;
    const uint16_t* B = p.B + a * p.b_stride;
    const uint16_t* row[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) row[j] = B + ch.channel(j) * p.ldb;
    if (p.rank < 8) {
        for (int k = 0; k < p.rank; ++k)
#pragma unroll
            for (int j = 0; j < NT; ++j) y[j] = fmaf(h[k], __uint_as_float((uint32_t)row[j][k] << 16), y[j]);
        return;
    }
    // octets of ranks; the last one moves back to end with the rank, what it repeats counts as zero
#pragma unroll 4
    for (int k = 0; k < p.rank; k += 8) {
        const int at = min(k, p.rank - 8);
        float hv[8];
        const f32x4 u = *reinterpret_cast<const f32x4_a4*>(h + at), v = *reinterpret_cast<const f32x4_a4*>(h + at + 4);
#pragma unroll
        for (int d = 0; d < 8; ++d) hv[d] = at + d >= k ? (d < 4 ? u[d & 3] : v[d & 3]) : 0.f;
        u32x4 b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) b[j] = *reinterpret_cast<const u32x4_a2*>(row[j] + at);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                y[j] = fmaf(hv[2 * d], bf16lo_to_f32(b[j][d]), y[j]);
                y[j] = fmaf(hv[2 * d + 1], bf16hi_to_f32(b[j][d]), y[j]);
            }
    }
}

// FORM of a product: plain, gated pairs of channels, or plain with adapters.
enum { kPlain = 0, kGated = 1, kAdapters = 2 };

template <int BITS, int PARTS, int NT, int GS, int FORM, int W>
__global__ __launch_bounds__(64 * W, W == 16 ? 4 : W == 4 && GS == 4 && kLaneWords<BITS> == 1 ? 3 : 2)
void matmul_rows_kernel(MatmulKernelArgs p) {
    constexpr bool GATED = FORM == kGated;
    constexpr int kLW = kLaneWords<BITS>;
    constexpr int kXBytes = PARTS == 1 ? 2 : 4, kGroups = kChunkSteps / GS;
    __shared__ float part[W][4 * NT][64];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int width = GATED ? p.N / 2 : p.N;
    constexpr int kCols = LaneChannels<NT, GATED>::kRun * 16;
    const int tile0 = blockIdx.x * kCols;
    const int e = blockIdx.y;
    if (e == p.E) {
        zero_outside<PARTS>(p, tile0, kCols, width, 64 * W);
        return;
    }
    int64_t lo, hi;
    expert_rows(p, e, lo, hi);
    if (lo >= hi) return;

    const LaneChannels<NT, GATED> ch(tile0, lane, p.N);
    const int nfull = p.K / kChunkK;                 // whole chunks
    const int sh = lane_shift<BITS>(q);
    const uint32_t base = code_base();
    const uint32_t* words0 = p.packed + e * p.p_stride;
    const uint32_t off[2] = {lane_word<BITS>(q) * p.ldp + ch.c0, lane_word2<BITS>(q) * p.ldp + ch.c0};
    const float* scales = p.scales + e * p.s_stride;

    for (int64_t r0 = lo; r0 < hi; r0 += 16) {
        // words, scales and rows one of the wave's chunks ahead: each step's registers are loaded again as soon as they
        // have been used
        uint32_t w[kChunkSteps][kLW][NT], sc[kGroups][NT];
        RawOctet<PARTS> x[kChunkSteps];
        auto load_scales = [&](int step, uint32_t (&v)[NT]) {
            const int g = step / GS;
            const float* row = scales + (int64_t)(g < p.last_group ? g : p.last_group) * p.s_row;
            ch.words(reinterpret_cast<const uint32_t*>(row), ch.c0, v);
        };
        auto load_words = [&](int chunk, int s) {
            const int step = chunk * kChunkSteps + s;
            const uint32_t* row = words0 + (int64_t)(step * BITS) * p.ldp;
#pragma unroll
            for (int l = 0; l < kLW; ++l) ch.words(row, off[l], w[s][l]);
            if ((s + 1) % GS == 0) load_scales(step, sc[s / GS]);
        };
        int64_t mine = r0 + (lane & 15);
        if (mine >= hi) mine = hi - 1;               // a row past the end repeats the last one and is not stored
        const int64_t src = source_row(p, mine);
        const char* xrow = static_cast<const char*>(p.X) + ((src < 0 ? 0 : src) * p.ldx + 8 * q) * kXBytes;
        auto load_x = [&](int chunk, int s) { x[s].whole(xrow + (chunk * kChunkSteps + s) * (kStepK * kXBytes)); };
        if (wave < nfull) {                          // in the order of the loop: the waits count loads
#pragma unroll
            for (int s = 0; s < kChunkSteps; ++s) {
                load_x(wave, s);
                load_words(wave, s);
            }
        }

        f32x4 acc[NT], sum, prt[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        auto clear = [&] {
            sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < NT; ++j) prt[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        };
        auto multiply = [&](const RawOctet<PARTS>& rows, const uint32_t (&v)[kLW][NT]) {
            u32x4 a[PARTS];
            rows.parts(a);
#pragma unroll
            for (int i = 0; i < PARTS; ++i) a[i] = pair_order(a[i]);
            if constexpr (PARTS == 1) sum = mfma16(a[0], minus_excess_frag(), sum);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const bf16x8 b = PARTS == 1 ? codes_to_frag<BITS>(v[0][j], v[kLW - 1][j], sh, base)
                                            : codes_to_exact_frag<BITS>(v[0][j], v[kLW - 1][j], sh, base);
#pragma unroll
                for (int i = 0; i < PARTS; ++i) prt[j] = mfma16(a[i], b, prt[j]);
            }
        };
        auto add = [&](const uint32_t (&f)[NT]) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(__uint_as_float(f[j]), prt[j][i] + sum[i], acc[j][i]);
        };
        for (int c = wave; c < nfull; c += W) {
            const bool more = c + W < nfull;
#pragma unroll
            for (int s = 0; s < kChunkSteps; ++s) {
                if (s % GS == 0) clear();
                multiply(x[s], w[s]);
                if ((s + 1) % GS == 0) add(sc[s / GS]);
                __builtin_amdgcn_sched_barrier(0);   // loads moved up would need registers of their own
                if (more) {
                    load_x(c + W, s);
                    load_words(c + W, s);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        {   // the rest of K, a step for each of the next waves: past its end x is zero
            const int step = nfull * kChunkSteps + (wave + W - nfull % W) % W;
            if (step * kStepK < p.K) {
                const int last = p.nwords - 1;
                uint32_t v[kLW][NT], f[NT];
                RawOctet<PARTS> rows;
                rows.some(xrow + step * (kStepK * kXBytes), p.K - step * kStepK - 8 * q, p.K);
                ch.words(words0, min(step * BITS + lane_word<BITS>(q), last) * p.ldp + ch.c0, v[0]);
                if constexpr (kLW == 2)
                    ch.words(words0, min(step * BITS + lane_word2<BITS>(q), last) * p.ldp + ch.c0, v[1]);
                load_scales(step, f);
                clear();
                multiply(rows, v);
                add(f);
            }
        }

        if (r0 != lo) __syncthreads();               // the previous rows' partials have been read
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) part[wave][i * NT + j][lane] = acc[j][i];
        __syncthreads();
        if (wave < 4) {                              // row register `wave` of every lane
            float y[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) y[j] = 0.f;
#pragma unroll
            for (int s = 0; s < W; ++s)
#pragma unroll
                for (int j = 0; j < NT; ++j) y[j] += part[s][wave * NT + j][lane];
#pragma unroll
            for (int j = 0; j < NT; ++j) y[j] *= kCodeUnits<BITS>;
            const int64_t r = r0 + 4 * q + wave;
            if (r < hi) {
                if constexpr (FORM == kAdapters) add_adapter_row<NT, GATED>(p, r, ch, y);
                const bool real = source_row(p, r) >= 0;
                constexpr int NV = LaneChannels<NT, GATED>::kRun;
                float o[NV];
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    o[j] = y[j];
                    if constexpr (GATED) o[j] = gated(y[j], y[NV + j]);
                    o[j] = real ? o[j] : 0.f;
                }
                store_values<PARTS, NV>(p.Y, r * p.ldy + ch.c0, o);
            }
        }
    }
}

// Channels per workgroup: 32 while every such workgroup has a CU of its own, else 64 (one token x 4096, 4 bits, 8192
// channels: 6.6 us with 32, 8.6 with 64; 10240 channels: 10.8 and 8.8; 16 rows: 8.7 and 9.4, 15.1 and 9.6; fp32 rows and 3
// bits alike).  Waves that share K: 16 in the narrow kernel with one word per step and lane, whose registers allow it
// (latency counts); 8 in the others; 4 where there are many workgroups, several of which then share a CU and cover each
// other's start and end (experts' decode step 82 us with 4, 110 with 8).
template <int BITS, int PARTS, int NT, int FORM, int W>
hipError_t launch_rows_form(const MatmulKernelArgs& k, bool swiglu, hipStream_t stream) {
    const int width = swiglu ? k.N / 2 : k.N;
    const dim3 grid((unsigned)ceil_div(width, NT == 4 && !swiglu ? 64 : 32), (unsigned)(k.E + (k.offsets ? 1 : 0)));
    const dim3 block(64 * W);
    // a scale per step: 16 waves' registers spill (one token, 4096 x 4096, 4 bits in groups of 32: 20.4 us against 12.7)
    constexpr int W1 = W < 8 ? W : 8;
    if (k.lg_group == 0)
        hipLaunchKernelGGL((matmul_rows_kernel<BITS, PARTS, NT, 1, FORM, W1>), grid, dim3(64 * W1), 0, stream, k);
    else if (k.lg_group == 1)
        hipLaunchKernelGGL((matmul_rows_kernel<BITS, PARTS, NT, 2, FORM, W>), grid, block, 0, stream, k);
    else
        hipLaunchKernelGGL((matmul_rows_kernel<BITS, PARTS, NT, 4, FORM, W>), grid, block, 0, stream, k);
    return hipGetLastError();
}

template <int BITS, int PARTS, int WIDE, int NARROW>
hipError_t launch_rows_w(const MatmulKernelArgs& k, bool swiglu, hipStream_t stream) {
    if (swiglu) return launch_rows_form<BITS, PARTS, 4, kGated, WIDE>(k, swiglu, stream);
    if (ceil_div(k.N, 32) * k.E > 256) {
        if (k.H) return launch_rows_form<BITS, PARTS, 4, kAdapters, WIDE>(k, swiglu, stream);
        return launch_rows_form<BITS, PARTS, 4, kPlain, WIDE>(k, swiglu, stream);
    }
    if (k.H) return launch_rows_form<BITS, PARTS, 2, kAdapters, NARROW>(k, swiglu, stream);
    return launch_rows_form<BITS, PARTS, 2, kPlain, NARROW>(k, swiglu, stream);
}

template <int BITS>
hipError_t launch_rows(const MatmulKernelArgs& k, bool f32, bool swiglu, hipStream_t stream) {
    if (f32) return launch_rows_w<BITS, 3, 8, 8>(k, swiglu, stream);
    if (ceil_div(k.N, 64) * k.E >= 1024) return launch_rows_w<BITS, 1, 4, 4>(k, swiglu, stream);
    return launch_rows_w<BITS, 1, 8, kLaneWords<BITS> == 1 ? 16 : 8>(k, swiglu, stream);
}

}  // namespace gptq
