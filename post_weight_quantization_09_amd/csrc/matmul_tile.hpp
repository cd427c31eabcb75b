// Product of many rows with packed weights: a prompt's rows, an expert with many rows.
//
// What bounds it: the matrix cores (2 M K N operations against half a byte per weight).  One workgroup of four waves owns
// 16 RT rows of one expert and 256 channels; every wave holds its own 64 channels for all the rows, so no code is
// converted twice in a workgroup: the words of a 128-k chunk come straight from global memory into registers as operands
// (nothing of the weights passes through LDS) and serve RT row tiles.  Seven of them (four for small experts and for codes
// of two words an operand, see big_tile_rows in matmul.hip): the 256 registers that two waves
// per SIMD leave each then hold the sums, the chunk's operands and the next step's rows; eight leave no room to read rows
// ahead (experts 8192 x 28672 x 4096: 1.91 ms against 2.05; adapters 4096 x 8192 x 28672: 2.06 against 2.80), and one
// wave per SIMD with 512 registers is slower (3.1 ms: half of them are accumulation registers, which cost moves).  That is
// 1.0 PFLOP/s: the matrix units are busy 48% of the cycles at 2.0 GHz.  The rows are laid out once per call by
// stage_kernel: octets of k in the converted operand's order, [K / 8][row], so that a chunk is 16 contiguous
// pieces, copied to LDS by DMA and read back as 16-byte operands without bank conflicts; rows are gathered and fp32 rows
// split in the same pass, and it leaves the row sums that take the codes' excess off again as the accumulators' start (bf16 rows).
#pragma once

#include "matmul_rows.hpp"

namespace gptq {

typedef __attribute__((address_space(3))) void lds_dma_t;

// 64 lanes x BYTES from global memory (a uniform address and the lane's byte offset) into LDS at `lds` + BYTES * lane.
// The instruction itself and not the compiler's builtin: after the builtin every LDS read waits until the copy has landed,
// also one from the other buffer (2.05 against 1.80 ms without any copy, 8192 rows x 28672 channels x 4096).  It has no
// result registers; the kernel waits for it (vmcnt(0) before the barrier after which the buffer is read).  M0, which the
// compiler may be using, is put back.
template <int BYTES>
__device__ __forceinline__ void copy_to_lds(const void* src, uint32_t off, void* lds) {
    const uint32_t at = (uint32_t)(uintptr_t)(lds_dma_t*)lds;
    uint32_t m0;
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\ts_mov_b32 m0, %0"
                     : "=&s"(m0) : "s"(at), "v"(off), "s"(src) : "memory");
    else
        asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %2, %3\n\ts_mov_b32 m0, %0"
                     : "=&s"(m0) : "s"(at), "v"(off), "s"(src) : "memory");
}

constexpr int kTileCols = 256;         // channels of a workgroup (outputs: half of them when gated)
constexpr int kTileGroup = 8;          // row tiles that neighbouring workgroups share a weight tile for

// acc += H B^T for the rows r0 .. r0 + nrow - 1: one product per run of rows with the same adapter, added to the rows of
// the run alone (zero rows of H would not do: an infinite or NaN value of B would reach the other rows as 0 * inf).
template <int RT, int NT, bool GATED>
__device__ __forceinline__ void add_adapter_runs(const MatmulKernelArgs& p, const LaneChannels<NT, GATED>& ch, int64_t r0,
                                                 int nrow, int lane, f32x4 (&acc)[RT][NT]) {
    constexpr int HP = 3;                            // parts of H: exactly its fp32 value
    const int q = lane >> 4;
    for (int f = 0; f < nrow;) {
        const int a = __builtin_amdgcn_readfirstlane(p.row_adapter[r0 + f]);
        int g = f + 1;                               // end of the run, 64 rows at a time
        while (g < nrow) {
            const int mine = g + lane < nrow ? p.row_adapter[r0 + g + lane] : -2;
            const uint64_t other = __ballot(mine != a);
            if (other) {
                g += __builtin_ctzll(other);
                break;
            }
            g += 64;
        }
        if (g > nrow) g = nrow;
        for (int k = 0; a >= 0 && k < p.rank; k += kStepK) {
            const int kq = k + 8 * q;
            bf16x8 b[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                u32x4 v[1];
                load_octet<1>(p.B + a * p.b_stride + ch.channel(j) * p.ldb, kq, p.rank, v);
                b[j] = __builtin_bit_cast(bf16x8, v[0]);
            }
            const bool has = kq < p.rank;
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                if (16 * t >= g || 16 * t + 16 <= f) continue;
                const int row = 16 * t + (lane & 15);
                const bool in = has && row >= f && row < g;
                const f32x4* h = reinterpret_cast<const f32x4*>(p.H + (r0 + (in ? row : f)) * p.hrank + (has ? kq : 0));
                f32x4 u = h[0], v = h[1];
                for (int z = 1; z < p.h_parts; ++z) {
                    const f32x4* hz = h + (int64_t)z * p.M * p.hrank / 4;
                    u += hz[0];
                    v += hz[1];
                }
                float hv[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    hv[i] = in ? u[i] : 0.f;
                    hv[4 + i] = in ? v[i] : 0.f;
                }
                u32x4 hp[3];
                split3(hv, hp);
                f32x4 sum[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) sum[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < HP; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) sum[j] = mfma16(hp[i], b[j], sum[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int to = 16 * t + 4 * q + i;
#pragma unroll
                    for (int j = 0; j < NT; ++j) acc[t][j][i] += to >= f && to < g ? sum[j][i] : 0.f;
                }
            }
        }
        f = g;
    }
}

template <int BITS, int PARTS, int RT, int GS, int FORM>
__global__ __launch_bounds__(256, PARTS == 1 ? 2 : 1) void matmul_tile_kernel(MatmulKernelArgs p, int ntn, int ntm) {
    constexpr bool GATED = FORM == kGated;
    constexpr int NT = 4, TM = (16 * RT + 63) / 64 * 64, kGroups = kChunkSteps / GS;
    constexpr int kOctets = kChunkK / 8;
    __shared__ __attribute__((aligned(1024))) uint16_t xs[2][PARTS][kOctets][TM][8];
    __shared__ __attribute__((aligned(1024))) float ss[2][kGroups][PARTS == 1 ? TM : 1];
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    // Workgroup b runs on XCD b % 8: each XCD takes a contiguous share of an order in which kTileGroup row tiles sweep
    // the channels together, so that the tiles in flight on one XCD share rows and words in its L2.
    const int total = ntn * ntm, share = (total + 7) / 8;
    const int lin = (int)(blockIdx.x & 7) * share + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= share || lin >= total) return;
    const int grp = lin / (kTileGroup * ntn), in_grp = lin - grp * kTileGroup * ntn;
    const int gm = min(kTileGroup, ntm - grp * kTileGroup);
    const int tm = grp * kTileGroup + in_grp % gm, tn = in_grp / gm;

    const int e = p.tiles[3 * tm];
    if (e < 0) return;
    const int64_t r0 = p.tiles[3 * tm + 1], r1 = p.tiles[3 * tm + 2];
    constexpr int kRun = LaneChannels<NT, GATED>::kRun;
    const int col0 = tn * (64 * kRun) + wave * (16 * kRun);
    const LaneChannels<NT, GATED> ch(col0, lane, p.N);
    if (e == p.E) {                                  // rows of no expert
        float z[kRun];
#pragma unroll
        for (int j = 0; j < kRun; ++j) z[j] = 0.f;
        for (int64_t r = r0 + q; r < r1; r += 4) store_values<PARTS, kRun>(p.Y, r * p.ldy + ch.c0, z);
        return;
    }
    const uint32_t* words = p.packed + e * p.p_stride;
    const float* scales = p.scales + e * p.s_stride;
    const int nchunks = (p.K + kChunkK - 1) / kChunkK;
    const int last_word = p.nwords - 1;
    const int sh = lane_shift<BITS>(q);
    const uint32_t off[2] = {lane_word<BITS>(q) * p.ldp + ch.c0, lane_word2<BITS>(q) * p.ldp + ch.c0};
    constexpr int kLW = kLaneWords<BITS>;
    const uint32_t base = code_base();
    uint32_t w[kChunkSteps][kLW][NT];
    uint32_t sc[kGroups][NT];
    auto load_words = [&](int chunk) {
        if ((chunk + 1) * kChunkSteps * BITS <= p.nwords) {
#pragma unroll
            for (int s = 0; s < kChunkSteps; ++s) {
                const uint32_t* row = words + (int64_t)((chunk * kChunkSteps + s) * BITS) * p.ldp;
#pragma unroll
                for (int l = 0; l < kLW; ++l) ch.words(row, off[l], w[s][l]);
            }
        } else {                                     // past the layer's last word x is zero
#pragma unroll
            for (int s = 0; s < kChunkSteps; ++s) {
                const int at = (chunk * kChunkSteps + s) * BITS;
                ch.words(words, min(at + lane_word<BITS>(q), last_word) * p.ldp + ch.c0, w[s][0]);
                if constexpr (kLW == 2)
                    ch.words(words, min(at + lane_word2<BITS>(q), last_word) * p.ldp + ch.c0, w[s][1]);
            }
        }
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int at = chunk * kGroups + g;
            const float* row = scales + (int64_t)(at < p.last_group ? at : p.last_group) * p.s_row;
            ch.words(reinterpret_cast<const uint32_t*>(row), ch.c0, sc[g]);
        }
    };
    const int64_t noct = (int64_t)nchunks * kOctets;
    constexpr int kRowPieces = TM / 64;              // 64 rows of 16 bytes per DMA instruction
    constexpr int kPieces = PARTS * kOctets * kRowPieces;
    auto stage = [&](int chunk, int buf) {
#pragma unroll
        for (int i = 0; i < kPieces / 4; ++i) {
            const int pc = wave * (kPieces / 4) + i;
            const int part = pc / (kOctets * kRowPieces), rest = pc % (kOctets * kRowPieces);
            const int o = rest / kRowPieces, h = rest % kRowPieces;
            const uint16_t* src =
                p.XT + ((part * noct + (int64_t)chunk * kOctets + o) * p.Mp + r0 + 64 * h) * 8;
            copy_to_lds<16>(src, 16 * lane, &xs[buf][part][o][64 * h][0]);
        }
        constexpr int kSumPieces = PARTS == 1 ? kGroups * kRowPieces : 0;
#pragma unroll
        for (int i = 0; i < (kSumPieces + 3) / 4; ++i) {
            const int pc = wave + 4 * i;
            if (pc < kSumPieces) {
                const int g = pc / kRowPieces, h = pc % kRowPieces;
                const float* src = p.sums + ((int64_t)chunk * kGroups + g) * p.Mp + r0 + 64 * h;
                copy_to_lds<4>(src, 4 * lane, &ss[buf][g][PARTS == 1 ? 64 * h : 0]);
            }
        }
    };

    f32x4 acc[RT][NT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    stage(0, 0);
    load_words(0);

    for (int c = 0; c < nchunks; ++c) {
        const int buf = c & 1;
        // this chunk's rows are in LDS for every wave, and every wave has left the other buffer
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        bf16x8 b[kChunkSteps][NT];
#pragma unroll
        for (int s = 0; s < kChunkSteps; ++s)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                b[s][j] = PARTS == 1 ? codes_to_frag<BITS>(w[s][0][j], w[s][kLW - 1][j], sh, base)
                                     : codes_to_exact_frag<BITS>(w[s][0][j], w[s][kLW - 1][j], sh, base);
        float f[kGroups][NT];
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int j = 0; j < NT; ++j) f[g][j] = __uint_as_float(sc[g][j]);
        if (c + 1 < nchunks) {
            stage(c + 1, buf ^ 1);
            load_words(c + 1);
        }
        // one step of one row tile after the other, its successor's rows on their way out of LDS meanwhile; the order is
        // pinned (left alone, the scheduler puts every read right before its use)
        u32x4 a[2][PARTS];
        f32x4 start[2], prt[NT];
        auto read_rows = [&](int k, int set) {
#pragma unroll
            for (int i = 0; i < PARTS; ++i)
                a[set][i] = *reinterpret_cast<const u32x4*>(&xs[buf][i][4 * (k % kChunkSteps) + q][16 * (k / kChunkSteps) + (lane & 15)][0]);
        };
        auto read_start = [&](int u, int set) {      // of group u, row tile by row tile
            start[set] = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (PARTS == 1)
                start[set] = *reinterpret_cast<const f32x4*>(&ss[buf][u % kGroups][16 * (u / kGroups) + 4 * q]);
        };
        read_rows(0, 0);
        read_start(0, 0);
#pragma unroll
        for (int k = 0; k < RT * kChunkSteps; ++k) {
            const int t = k / kChunkSteps, s = k % kChunkSteps, u = k / GS;
            __builtin_amdgcn_sched_barrier(0);
            if (k + 1 < RT * kChunkSteps) read_rows(k + 1, (k + 1) & 1);
            if (k % GS == GS - 1 && u + 1 < RT * kGroups) read_start(u + 1, (u + 1) & 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < PARTS; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    prt[j] = mfma16(a[k & 1][i], b[s][j], k % GS == 0 && i == 0 ? start[u & 1] : prt[j]);
            if (k % GS == GS - 1) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[t][j][i] = fmaf(f[s / GS][j], prt[j][i], acc[t][j][i]);
            }
        }
    }

#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][j][i] *= kCodeUnits<BITS>;
    if constexpr (FORM == kAdapters) {
        if (!p.Z) add_adapter_runs<RT, NT, GATED>(p, ch, r0, (int)(r1 - r0), lane, acc);
    }
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = r0 + 16 * t + 4 * q + i;
            if (r < r1) {
                const bool real = source_row(p, r) >= 0;
                float o[kRun];
#pragma unroll
                for (int j = 0; j < kRun; ++j) {
                    o[j] = acc[t][j][i];
                    if constexpr (FORM == kAdapters) o[j] += p.Z ? p.Z[r * p.N + ch.channel(j)] : 0.f;
                    if constexpr (GATED) o[j] = gated(acc[t][j][i], acc[t][kRun + j][i]);
                    o[j] = real ? o[j] : 0.f;
                }
                store_values<PARTS, kRun>(p.Y, r * p.ldy + ch.c0, o);
            }
        }
}

template <int BITS, int PARTS, int RT>
hipError_t launch_tile_rt(const MatmulKernelArgs& k, int ntm, bool swiglu, hipStream_t stream) {
    const int64_t width = swiglu ? k.N / 2 : k.N;
    const int ntn = (int)ceil_div(width, swiglu ? kTileCols / 2 : kTileCols);
    const unsigned grid = (unsigned)(ceil_div((int64_t)ntn * ntm, 8) * 8);
#define GPTQ_TILE(GS, FORM) \
    hipLaunchKernelGGL((matmul_tile_kernel<BITS, PARTS, RT, GS, FORM>), dim3(grid), dim3(256), 0, stream, k, ntn, ntm)
#define GPTQ_TILE_FORM(FORM)                        \
    do {                                            \
        if (k.lg_group == 0) GPTQ_TILE(1, FORM); \
        else if (k.lg_group == 1) GPTQ_TILE(2, FORM); \
        else GPTQ_TILE(4, FORM);                    \
    } while (0)
    if (swiglu) GPTQ_TILE_FORM(kGated);
    else if (k.H) GPTQ_TILE_FORM(kAdapters);
    else GPTQ_TILE_FORM(kPlain);
#undef GPTQ_TILE_FORM
#undef GPTQ_TILE
    return hipGetLastError();
}

// row_tiles: 4, or 7 as big_tile_rows() allows.
template <int BITS>
hipError_t launch_tile(const MatmulKernelArgs& k, bool f32, int row_tiles, int ntm, bool swiglu, hipStream_t stream) {
    if (f32) return launch_tile_rt<BITS, 3, 4>(k, ntm, swiglu, stream);
    if constexpr (kLaneWords<BITS> == 1) {
        if (row_tiles == 7) return launch_tile_rt<BITS, 1, 7>(k, ntm, swiglu, stream);
    }
    return launch_tile_rt<BITS, 1, 4>(k, ntm, swiglu, stream);
}

}  // namespace gptq
