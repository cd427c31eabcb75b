// Product of a few rows with packed weights: the single tokens of a decode step, an expert with few rows.
//
// What bounds it: the packed words are read once from HBM; for up to 16 rows per expert there are at most 32 operations
// per weight, far below what the matrix cores do in the time of its half byte.  So one workgroup owns 16 NT channels of
// one expert over all K, its W waves take the 128-k chunks in turn (each wave's words come straight into registers as
// MFMA operands, the next chunk's loads in flight while one is multiplied), and the W partial sums are joined in LDS in
// a fixed order: no second launch, no partials in memory, the same bits every time.  MT row tiles of 16 share a wave's
// operands; more rows than 16 MT loop.
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
template <int NT>
struct WordLoad;
template <>
struct WordLoad<4> {
    static __device__ __forceinline__ void run(const uint32_t* p, uint32_t (&w)[4]) {
        const u32x4 v = *reinterpret_cast<const u32x4_a4*>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = v[j];
    }
};
template <>
struct WordLoad<2> {
    static __device__ __forceinline__ void run(const uint32_t* p, uint32_t (&w)[2]) {
        const u32x2 v = *reinterpret_cast<const u32x2_a4*>(p);
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
    int64_t c0;        // first channel (and first output column)
    int64_t half;
    __device__ __forceinline__ LaneChannels(int64_t tile0, int lane, int64_t N) {
        half = GATED ? N / 2 : 0;
        const int64_t width = GATED ? N / 2 : N;
        c0 = tile0 + kRun * (lane & 15);
        if (c0 > width - kRun) c0 = width - kRun;
    }
    __device__ __forceinline__ void words(const uint32_t* row, uint32_t (&w)[NT]) const {
        if constexpr (GATED) {
            uint32_t a[kRun], b[kRun];
            WordLoad<kRun>::run(row + c0, a);
            WordLoad<kRun>::run(row + half + c0, b);
#pragma unroll
            for (int j = 0; j < kRun; ++j) { w[j] = a[j]; w[kRun + j] = b[j]; }
        } else {
            WordLoad<NT>::run(row + c0, w);
        }
    }
    __device__ __forceinline__ int64_t channel(int j) const { return j < kRun ? c0 + j : half + c0 + (j - kRun); }
};

template <int BITS, int PARTS, int MT, int NT, bool GATED, int W>
__global__ __launch_bounds__(64 * W) void matmul_rows_kernel(MatmulKernelArgs p) {
    constexpr int kVals = MT * 4;                    // (row tile, register) items of NT channels
    __shared__ float part[W][kVals * NT][64];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t width = GATED ? p.N / 2 : p.N;
    constexpr int kCols = LaneChannels<NT, GATED>::kRun * 16;
    const int64_t tile0 = (int64_t)blockIdx.x * kCols;
    const int e = blockIdx.y;
    if (e == p.E) {
        zero_outside<PARTS>(p, tile0, kCols, width, 64 * W);
        return;
    }
    int64_t lo, hi;
    expert_rows(p, e, lo, hi);
    if (lo >= hi) return;

    const LaneChannels<NT, GATED> ch(tile0, lane, p.N);
    const uint32_t* words = p.packed + e * p.p_stride;
    const float* scales = p.scales + e * p.s_stride;
    const int nchunks = (int)((p.K + kChunkK - 1) / kChunkK);
    const int last_word = p.nwords - 1;
    const int wa = lane_word<BITS>(q), wb = lane_word2<BITS>(q), sh = lane_shift<BITS>(q);
    constexpr int kLW = kLaneWords<BITS>;

    auto load_words = [&](int chunk, uint32_t (&w)[kChunkSteps][kLW][NT]) {
#pragma unroll
        for (int s = 0; s < kChunkSteps; ++s) {
            const int at = (chunk * kChunkSteps + s) * BITS;
            const int a = min(at + wa, last_word);   // past the last word x is zero
            ch.words(words + (int64_t)a * p.ldp, w[s][0]);
            if constexpr (kLW == 2) {
                const int b = min(at + wb, last_word);
                ch.words(words + (int64_t)b * p.ldp, w[s][1]);
            }
        }
    };
    float s_ch[NT];
    if (p.per_channel) {
#pragma unroll
        for (int j = 0; j < NT; ++j) s_ch[j] = scales[ch.channel(j)];
    }

    for (int64_t r0 = lo; r0 < hi; r0 += 16 * MT) {
        const char* xrow[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            int64_t r = r0 + 16 * t + (lane & 15);
            if (r >= hi) r = hi - 1;                 // a row past the end repeats the last one and is not stored
            int64_t s = source_row(p, r);
            xrow[t] = static_cast<const char*>(p.X) + (s < 0 ? 0 : s) * p.ldx * (PARTS == 1 ? 2 : 4);
        }
        f32x4 acc[MT][NT];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};

        // y += H B^T of the rows' adapters: the runs of equal adapters among the tile's rows, dealt out to the waves
        if (p.H) {
            constexpr int HP = PARTS == 1 ? 2 : 3;   // parts of H: its error stays far below the output's rounding
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int64_t t0 = r0 + 16 * t;
                if (t0 >= hi) break;
                const int nrow = (int)(hi - t0 < 16 ? hi - t0 : 16);
                const int mine = (lane & 15) < nrow ? p.row_adapter[t0 + (lane & 15)] : -1;
                for (int f = 0, run = t; f < nrow; ++run) {
                    const int a = __builtin_amdgcn_readlane(mine, f);
                    int g = f + 1;
                    while (g < nrow && __builtin_amdgcn_readlane(mine, g) == a) ++g;
                    if (a >= 0 && run % W == wave) {
                        const bool in = (lane & 15) >= f && (lane & 15) < g;
                        const float* h = p.H + (t0 + (lane & 15)) * p.hrank;
                        for (int k = 0; k < p.rank; k += kStepK) {
                            float hv[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) hv[i] = 0.f;
                            const int kq = k + 8 * q;
                            if (in && kq < p.rank) {
                                const f32x4 u = *reinterpret_cast<const f32x4*>(h + kq);
                                const f32x4 v = *reinterpret_cast<const f32x4*>(h + kq + 4);
#pragma unroll
                                for (int i = 0; i < 4; ++i) { hv[i] = u[i]; hv[4 + i] = v[i]; }
                            }
                            u32x4 hp[3];
                            split3(hv, hp);
#pragma unroll
                            for (int j = 0; j < NT; ++j) {
                                u32x4 b[1] = {{0u, 0u, 0u, 0u}};
                                if (kq < p.rank)
                                    load_octet<1>(p.B + a * p.b_stride + ch.channel(j) * p.ldb, kq, p.rank, p.bvec, b);
#pragma unroll
                                for (int i = 0; i < HP; ++i)
                                    acc[t][j] = mfma16(hp[i], __builtin_bit_cast(bf16x8, b[0]), acc[t][j]);
                            }
                        }
                    }
                    f = g;
                }
            }
        }

        uint32_t w[kChunkSteps][kLW][NT];
        if (wave < nchunks) load_words(wave, w);
        for (int c = wave; c < nchunks; c += W) {
            // this chunk's rows
            u32x4 x[kChunkSteps][MT][PARTS];
#pragma unroll
            for (int s = 0; s < kChunkSteps; ++s)
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    load_octet<PARTS>(xrow[t], (int64_t)c * kChunkK + s * kStepK + 8 * q, p.K, p.vec, x[s][t]);
            uint32_t wn[kChunkSteps][kLW][NT];
            if (c + W < nchunks) load_words(c + W, wn);
            f32x4 sum[MT], prt[MT][NT];
#pragma unroll
            for (int s = 0; s < kChunkSteps; ++s) {
                if ((s & (p.group_steps - 1)) == 0) {
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        sum[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int j = 0; j < NT; ++j) prt[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
                    }
                }
                bf16x8 b[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    b[j] = PARTS == 1 ? codes_to_frag<BITS>(w[s][0][j], w[s][kLW - 1][j], sh)
                                      : codes_to_exact_frag<BITS>(w[s][0][j], w[s][kLW - 1][j], sh);
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int i = 0; i < PARTS; ++i) {
                        const u32x4 a = pair_order(x[s][t][i]);
                        if constexpr (PARTS == 1) sum[t] = mfma16(a, minus_excess_frag<BITS>(), sum[t]);
#pragma unroll
                        for (int j = 0; j < NT; ++j) prt[t][j] = mfma16(a, b[j], prt[t][j]);
                    }
                if (((s + 1) & (p.group_steps - 1)) == 0) {
                    float sc[NT];
                    if (p.per_channel) {
#pragma unroll
                        for (int j = 0; j < NT; ++j) sc[j] = s_ch[j];
                    } else {
                        const int64_t g = ((int64_t)c * kChunkSteps + s) / p.group_steps;
                        const int64_t last = (p.K - 1) / (kStepK * p.group_steps);
                        const float* srow = scales + (g < last ? g : last) * p.N;
#pragma unroll
                        for (int j = 0; j < NT; ++j) sc[j] = srow[ch.channel(j)];
                    }
#pragma unroll
                    for (int t = 0; t < MT; ++t)
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc[t][j][i] = fmaf(sc[j], prt[t][j][i] + sum[t][i], acc[t][j][i]);
                }
            }
#pragma unroll
            for (int s = 0; s < kChunkSteps; ++s)
#pragma unroll
                for (int l = 0; l < kLW; ++l)
#pragma unroll
                    for (int j = 0; j < NT; ++j) w[s][l][j] = wn[s][l][j];
        }

        __syncthreads();                             // the previous rows' partials have been read
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) part[wave][(t * 4 + i) * NT + j][lane] = acc[t][j][i];
        __syncthreads();
        for (int v = wave; v < kVals; v += W) {
            float y[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) y[j] = 0.f;
            for (int s = 0; s < W; ++s)
#pragma unroll
                for (int j = 0; j < NT; ++j) y[j] += part[s][v * NT + j][lane];
            const int64_t r = r0 + 16 * (v >> 2) + 4 * q + (v & 3);
            if (r < hi) {
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

// Channels per workgroup: 64, or 32 where 64 would leave more than half of the CUs without a workgroup.
template <int BITS, int PARTS, int MT, int W>
hipError_t launch_rows_mt(const MatmulKernelArgs& k, bool swiglu, hipStream_t stream) {
    const int64_t width = swiglu ? k.N / 2 : k.N;
    const unsigned ey = (unsigned)(k.E + (k.offsets ? 1 : 0));
    if (swiglu) {
        hipLaunchKernelGGL((matmul_rows_kernel<BITS, PARTS, MT, 4, true, W>), dim3((unsigned)ceil_div(width, 32), ey),
                           dim3(64 * W), 0, stream, k);
    } else if (ceil_div(width, 64) * k.E >= 256) {
        hipLaunchKernelGGL((matmul_rows_kernel<BITS, PARTS, MT, 4, false, W>), dim3((unsigned)ceil_div(width, 64), ey),
                           dim3(64 * W), 0, stream, k);
    } else {
        hipLaunchKernelGGL((matmul_rows_kernel<BITS, PARTS, MT, 2, false, W>), dim3((unsigned)ceil_div(width, 32), ey),
                           dim3(64 * W), 0, stream, k);
    }
    return hipGetLastError();
}

template <int BITS>
hipError_t launch_rows(const MatmulKernelArgs& k, bool f32, int row_tiles, bool swiglu, hipStream_t stream) {
    if (f32) {
        if (row_tiles <= 1) return launch_rows_mt<BITS, 3, 1, 8>(k, swiglu, stream);
        return launch_rows_mt<BITS, 3, 2, 8>(k, swiglu, stream);
    }
    if (row_tiles <= 1) return launch_rows_mt<BITS, 1, 1, 16>(k, swiglu, stream);
    if (row_tiles <= 2) return launch_rows_mt<BITS, 1, 2, 8>(k, swiglu, stream);
    return launch_rows_mt<BITS, 1, 4, 8>(k, swiglu, stream);
}

}  // namespace gptq
