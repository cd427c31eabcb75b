// Product of some tens of rows with packed weights: batches of single tokens, experts with a few dozen rows, and larger
// products with too few tiles for the tile kernel to fill the GPU.
//
// What bounds it: between the two others - every weight serves up to 64 rows, so the matrix cores and the conversion of
// codes take about as long as the words do from HBM (64 rows x 14336 channels x 4096, 4 bits: 19.5 us with rank 16
// adapters, 30 MB of words at 1.5 TB/s; 782 rows of 16 experts x 1411 x 1990, 3 bits in groups of 64: 29.5 us, 149 TFLOP/s).  One workgroup owns 16 MT
// rows of one expert and 64 channels over all K; its W waves take the 128-k chunks in turn and join their sums in LDS in
// a fixed order, as in the few-rows kernel, so a product of 64 rows and 4096 channels already has 64 workgroups of 8
// waves without partials in memory.
// Rows come from stage_kernel (matmul.hip) as whole operands: one contiguous kilobyte per 16 rows and 32 k, where the rows
// as they lie would be 64 pieces of 16 bytes.
#pragma once

#include "matmul_rows.hpp"

namespace gptq {

template <int BITS, int PARTS, int MT, int GS, int FORM, int W>
__global__ __launch_bounds__(64 * W, 2) void matmul_split_kernel(MatmulKernelArgs p) {
    constexpr bool GATED = FORM == kGated;
    constexpr int NT = 4, kVals = MT * 4, kGroups = kChunkSteps / GS;
    constexpr int XR = 2;                            // steps of rows in flight
    constexpr int kLW = kLaneWords<BITS>;
    __shared__ float part[W][kVals * NT][64];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int e = p.tiles[3 * blockIdx.y];
    if (e < 0) return;
    const int64_t r0 = p.tiles[3 * blockIdx.y + 1], r1 = p.tiles[3 * blockIdx.y + 2];
    constexpr int kRun = LaneChannels<NT, GATED>::kRun;
    const LaneChannels<NT, GATED> ch(blockIdx.x * (16 * kRun), lane, p.N);
    if (e == p.E) {                                  // rows of no expert
        float z[kRun];
#pragma unroll
        for (int j = 0; j < kRun; ++j) z[j] = 0.f;
        for (int64_t r = r0 + (tid >> 4); r < r1; r += 4 * W) store_values<PARTS, kRun>(p.Y, r * p.ldy + ch.c0, z);
        return;
    }
    const int nchunks = (p.K + kChunkK - 1) / kChunkK;
    const int sh = lane_shift<BITS>(q);
    const uint32_t base = code_base();
    const uint32_t* words0 = p.packed + e * p.p_stride;
    const uint32_t off[2] = {lane_word<BITS>(q) * p.ldp + ch.c0, lane_word2<BITS>(q) * p.ldp + ch.c0};
    const float* scales = p.scales + e * p.s_stride;
    const int last_word = p.nwords - 1;
    // operands of the rows: a uniform base and the lane's 16 bytes
    const char* rows0 = reinterpret_cast<const char*>(p.XT) + r0 * 16;
    const uint32_t row_off = (uint32_t)(q * p.Mp + (lane & 15)) * 16;
    const int64_t part_bytes = (int64_t)nchunks * (kChunkK / 8) * p.Mp * 16;
    const char* sums0 = reinterpret_cast<const char*>(p.sums) + r0 * 4;

    uint32_t w[kChunkSteps][kLW][NT], sc[kGroups][NT];
    u32x4 x[XR][MT][PARTS];
    f32x4 start[MT];
    auto load_words = [&](int chunk, int s) {
        const int step = chunk * kChunkSteps + s;
        if ((step + 1) * BITS <= p.nwords) {
            const uint32_t* row = words0 + (int64_t)(step * BITS) * p.ldp;
#pragma unroll
            for (int l = 0; l < kLW; ++l) ch.words(row, off[l], w[s][l]);
        } else {                                     // past the layer's last word x is zero
            ch.words(words0, min(step * BITS + lane_word<BITS>(q), last_word) * p.ldp + ch.c0, w[s][0]);
            if constexpr (kLW == 2)
                ch.words(words0, min(step * BITS + lane_word2<BITS>(q), last_word) * p.ldp + ch.c0, w[s][1]);
        }
        if ((s + 1) % GS == 0) {
            const int g = step / GS;
            const float* row = scales + (int64_t)(g < p.last_group ? g : p.last_group) * p.s_row;
            ch.words(reinterpret_cast<const uint32_t*>(row), ch.c0, sc[s / GS]);
        }
    };
    auto load_x = [&](int chunk, int s) {
        const char* at = rows0 + (int64_t)(chunk * kChunkSteps + s) * 4 * p.Mp * 16;
#pragma unroll
        for (int i = 0; i < PARTS; ++i)
#pragma unroll
            for (int t = 0; t < MT; ++t)
                x[s % XR][t][i] = *reinterpret_cast<const u32x4*>(at + i * part_bytes + row_off + t * 256);
    };
    auto load_start = [&](int chunk, int g) {
        if constexpr (PARTS == 1) {
            const char* at = sums0 + (int64_t)(chunk * kGroups + g) * p.Mp * 4;
#pragma unroll
            for (int t = 0; t < MT; ++t) start[t] = *reinterpret_cast<const f32x4_a4*>(at + 16u * q + 64 * t);
        }
    };

    f32x4 acc[MT][NT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        start[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (wave < nchunks) {
        load_start(wave, 0);
#pragma unroll
        for (int s = 0; s < XR; ++s) load_x(wave, s);
#pragma unroll
        for (int s = 0; s < kChunkSteps; ++s) load_words(wave, s);
    }
    for (int c = wave; c < nchunks; c += W) {
        const int next = c + W < nchunks ? c + W : c;            // the last chunk loads itself again
        f32x4 prt[MT][NT];
#pragma unroll
        for (int s = 0; s < kChunkSteps; ++s) {
            bf16x8 b[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                b[j] = PARTS == 1 ? codes_to_frag<BITS>(w[s][0][j], w[s][kLW - 1][j], sh, base)
                                  : codes_to_exact_frag<BITS>(w[s][0][j], w[s][kLW - 1][j], sh, base);
            float f[NT];
            if ((s + 1) % GS == 0) {
#pragma unroll
                for (int j = 0; j < NT; ++j) f[j] = __uint_as_float(sc[s / GS][j]);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int i = 0; i < PARTS; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        prt[t][j] = mfma16(x[s % XR][t][i], b[j], s % GS == 0 && i == 0 ? start[t] : prt[t][j]);
            load_words(next, s);
            if (s + XR < kChunkSteps) load_x(c, s + XR);
            else load_x(next, s + XR - kChunkSteps);
            if (s % GS == 0) {
                if (s / GS + 1 < kGroups) load_start(c, s / GS + 1);
                else load_start(next, 0);
            }
            if ((s + 1) % GS == 0) {
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[t][j][i] = fmaf(f[j], prt[t][j][i], acc[t][j][i]);
            }
        }
    }

#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) part[wave][(t * 4 + i) * NT + j][lane] = acc[t][j][i];
    __syncthreads();
#pragma unroll
    for (int v = wave; v < kVals; v += W) {
        float y[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) y[j] = 0.f;
#pragma unroll
        for (int s = 0; s < W; ++s)
#pragma unroll
            for (int j = 0; j < NT; ++j) y[j] += part[s][v * NT + j][lane];
#pragma unroll
        for (int j = 0; j < NT; ++j) y[j] *= kCodeUnits<BITS>;
        const int64_t r = r0 + 16 * (v >> 2) + 4 * q + (v & 3);
        if (r < r1) {
            if constexpr (FORM == kAdapters) add_adapter_row<NT, GATED>(p, r, ch, y);
            const bool real = source_row(p, r) >= 0;
            float o[kRun];
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                o[j] = y[j];
                if constexpr (GATED) o[j] = gated(y[j], y[kRun + j]);
                o[j] = real ? o[j] : 0.f;
            }
            store_values<PARTS, kRun>(p.Y, r * p.ldy + ch.c0, o);
        }
    }
}

template <int BITS, int PARTS, int MT, int GS, int W>
hipError_t launch_split_waves(const MatmulKernelArgs& k, int ntm, bool swiglu, hipStream_t stream) {
    const dim3 grid((unsigned)ceil_div(swiglu ? k.N / 2 : k.N, swiglu ? 32 : 64), (unsigned)ntm), block(64 * W);
#define GPTQ_SPLIT(FORM) \
    hipLaunchKernelGGL((matmul_split_kernel<BITS, PARTS, MT, GS, FORM, W>), grid, block, 0, stream, k)
    if (swiglu) GPTQ_SPLIT(kGated);
    else if (k.H) GPTQ_SPLIT(kAdapters);
    else GPTQ_SPLIT(kPlain);
#undef GPTQ_SPLIT
    return hipGetLastError();
}

// Eight waves share K while every CU has one workgroup at most; beyond that four do, so that more workgroups share a CU
// and fewer partial sums are joined (87 rows x 3552 channels x 9496, 168 workgroups: 45 us with eight waves, 67 with
// four; 1127 rows of 23 experts x 24256 x 128: 275 against 117; 782 rows of 16 experts x 1411 x 1990: the same).
template <int BITS, int PARTS, int MT, int GS>
hipError_t launch_split_gs(const MatmulKernelArgs& k, int ntm, bool swiglu, hipStream_t stream) {
    const int64_t groups = ceil_div(swiglu ? k.N / 2 : k.N, swiglu ? 32 : 64) * (ceil_div(k.M, 16 * MT) + k.E / 2);
    if (groups > 256) return launch_split_waves<BITS, PARTS, MT, GS, 4>(k, ntm, swiglu, stream);
    return launch_split_waves<BITS, PARTS, MT, GS, 8>(k, ntm, swiglu, stream);
}

// row_tiles: 2, or 4 as split_row_tiles() allows.
template <int BITS>
hipError_t launch_split(const MatmulKernelArgs& k, bool f32, int row_tiles, int ntm, bool swiglu, hipStream_t stream) {
    if (f32) {
        if (k.lg_group == 0) return launch_split_gs<BITS, 3, 2, 1>(k, ntm, swiglu, stream);
        if (k.lg_group == 1) return launch_split_gs<BITS, 3, 2, 2>(k, ntm, swiglu, stream);
        return launch_split_gs<BITS, 3, 2, 4>(k, ntm, swiglu, stream);
    }
    if constexpr (kLaneWords<BITS> == 1) {
        if (row_tiles == 4) return launch_split_gs<BITS, 1, 4, 4>(k, ntm, swiglu, stream);
    }
    if (k.lg_group == 0) return launch_split_gs<BITS, 1, 2, 1>(k, ntm, swiglu, stream);
    if (k.lg_group == 1) return launch_split_gs<BITS, 1, 2, 2>(k, ntm, swiglu, stream);
    return launch_split_gs<BITS, 1, 2, 4>(k, ntm, swiglu, stream);
}

}  // namespace gptq
