// Routing of tokens to experts and joining their results on gfx950.
//
// Routing, per token t: p = softmax(logits_t); the topk experts with the largest p (ties: the lowest index), weights p
// or p over their sum; then a stable counting sort of the (token, choice) pairs by expert.  The data are a few hundred
// bytes per token: single tokens are bound by the launch and the chain of choices, prompts by the instructions of the
// choices.  So a wave takes four tokens, 16 lanes each, where 16 lanes hold the logits (8 per lane; more experts or
// choices: one token); logits stay in registers as integers in the order of the values, and every choice is one maximum
// over the lanes (data-parallel moves, no LDS) and the first lane that holds it (16384 tokens, 128 experts, 8 choices:
// 13.0 us with one token per wave, 7.4 with four).  The sort needs, per block of kBlockTokens tokens and expert,
// which tokens chose it: a bitmap in LDS, whose popcounts are both the block's count and the token's rank, whatever order
// the waves ran in.  Up to one block of tokens everything is one launch (one token: 3.4 us); else a second launch adds up
// the blocks' counts, a byte each (each block for itself, from L2: 6.8 us with 32-bit counts, 5.6 with bytes), and places
// the rows.  That grows with the square of the tokens, so many blocks are first added up by groups of 64, whose sums are
// scanned (2^20 tokens, 128 experts, 8 choices: 462 us).
#include "route.hpp"

#include <algorithm>

namespace gptq {

namespace {

constexpr int kBlockTokens = 64;
constexpr int kRouteWaves = 16;
constexpr int kGroupBlocks = 64;        // blocks whose counts are summed together where there are many

struct RouteArgs {
    const void* logits;
    int64_t T, ld;
    int E, topk, renorm;
    float* weights;
    int32_t* experts;
    int32_t* offsets;
    int32_t* rows;
    int32_t* positions;
    DevStatus* status;
    uint8_t* counts;        // [block][E, rounded up to 4]
    uint32_t* bad;          // [block]
    int nblocks;
    int32_t* before;        // [group][E]: an expert's tokens in the groups of blocks before; only where grouped
    int32_t* whole;         // [E]: an expert's tokens
};

// Maximum over 16 lanes (in all of them), or over the wave, by data-parallel moves.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#define GPTQ_DPP_MAX(CTRL) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false))
    if constexpr (LANES == 16) {
        GPTQ_DPP_MAX(0x128);   // rotated by 8, 4, 2, 1 lanes within each 16
        GPTQ_DPP_MAX(0x124);
        GPTQ_DPP_MAX(0x122);
        GPTQ_DPP_MAX(0x121);
        return v;
    } else {
        GPTQ_DPP_MAX(0x111);   // from 1, 2, 4, 8 lanes below
        GPTQ_DPP_MAX(0x112);
        GPTQ_DPP_MAX(0x114);
        GPTQ_DPP_MAX(0x118);
        GPTQ_DPP_MAX(0x142);   // lane 15 of each row to the next row
        GPTQ_DPP_MAX(0x143);   // lane 31 to the upper half; lane 63 has it
        return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
    }
#undef GPTQ_DPP_MAX
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int d = LANES / 2; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
// The token's lanes of a ballot, from bit 0.
template <int LANES>
__device__ __forceinline__ auto lanes_of(uint64_t mask, int lane) {
    if constexpr (LANES == 16) {
        const uint32_t half = lane & 32 ? (uint32_t)(mask >> 32) : (uint32_t)mask;
        return (lane & 16 ? half >> 16 : half) & 0xFFFFu;
    } else {
        return mask;
    }
}
__device__ __forceinline__ int first_bit(uint32_t v) { return __builtin_ctz(v); }
__device__ __forceinline__ int first_bit(uint64_t v) { return __builtin_ctzll(v); }

// fp32 bits in the order of the values; both zeros alike.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// Inclusive sum over the threads of a workgroup of kRouteWaves waves.
__device__ __forceinline__ int block_scan(int v, int* scratch) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    if (lane == 63) scratch[wave] = v;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < wave; ++w) before += scratch[w];
    return v + before;
}

// LANES lanes a token, V consecutive experts a lane.
template <int LANES, int V, bool F32>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs p) {
    constexpr int kTokens = 64 / LANES, kTurns = kBlockTokens / (kRouteWaves * kTokens);
    __shared__ uint64_t chosen[V * LANES];            // per expert: the block's tokens that chose it
    __shared__ int first[V * LANES + 1];
    __shared__ int16_t choice[kBlockTokens][LANES == 16 ? 16 : kRouteMaxTopk];
    __shared__ int scratch[kRouteWaves];
    __shared__ uint32_t bad;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane & (LANES - 1);
    for (int e = tid; e < p.E; e += 64 * kRouteWaves) chosen[e] = 0;
    if (tid == 0) bad = 0;
    const int64_t t0 = (int64_t)blockIdx.x * kBlockTokens;
    const int nt = (int)(p.T - t0 < kBlockTokens ? p.T - t0 : kBlockTokens);
    float all[kTurns][V];                             // the wave's tokens, loaded together
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
        const int64_t at = (t0 + min((wave + u * kRouteWaves) * kTokens + lane / LANES, nt - 1)) * p.ld + V * l;
        const float* xf = static_cast<const float*>(p.logits) + at;
        const uint16_t* xb = static_cast<const uint16_t*>(p.logits) + at;
        if (V * l + V <= p.E) {
            typedef __attribute__((ext_vector_type(V))) float vecf_t;
            typedef __attribute__((ext_vector_type(V))) uint16_t vecb_t;
            typedef vecf_t __attribute__((aligned(4))) vecf_a4;
            typedef vecb_t __attribute__((aligned(2))) vecb_a2;
            if constexpr (F32) {
                const vecf_t x = *reinterpret_cast<const vecf_a4*>(xf);
#pragma unroll
                for (int v = 0; v < V; ++v) all[u][v] = x[v];
            } else {
                const vecb_t x = *reinterpret_cast<const vecb_a2*>(xb);
#pragma unroll
                for (int v = 0; v < V; ++v) all[u][v] = __uint_as_float((uint32_t)x[v] << 16);
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                all[u][v] = -INFINITY;
                if (V * l + v < p.E) {
                    if constexpr (F32) all[u][v] = xf[v];
                    else all[u][v] = __uint_as_float((uint32_t)xb[v] << 16);
                }
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
        const int i0 = (wave + u * kRouteWaves) * kTokens, i = i0 + lane / LANES;
        if (i0 >= nt) break;
        const bool real = i < nt;
        const int64_t t = t0 + i;
        const float (&x)[V] = all[u];
        uint32_t key[V];                              // 0: not to be chosen (any more)
        bool wrong = false;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            wrong |= !(x[v] < INFINITY);
            key[v] = x[v] > -INFINITY && real ? ordered(x[v]) : 0u;
        }
        if (lanes_of<LANES>(__ballot(wrong), lane)) { // NaN or +infinity: reported, and the token chooses nothing
            if (l == 0) atomicOr(&bad, 1u);
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = 0;
        }
        // the value of choice j ends up in lane j, its expert in LDS
        uint32_t mine_key = 0, top_key = 0;
        for (int j = 0; j < p.topk; ++j) {
            uint32_t own = key[0];
#pragma unroll
            for (int v = 1; v < V; ++v) own = max(own, key[v]);
            const uint32_t k = lanes_max<LANES>(own);
            if (LANES == 64 && k == 0) break;
            if (j == 0) top_key = k;
            if (l == j) mine_key = k;
            const auto has = lanes_of<LANES>(__ballot(own == k && k), lane);
            if (has && l == first_bit(has)) {         // the first expert with this logit is this lane's
                int e = 0;
                bool open = true;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const bool is = open && key[v] == k;
                    e = is ? v : e;
                    key[v] = is ? 0 : key[v];
                    open = open && !is;
                }
                choice[i][j] = (int16_t)(V * l + e);
            }
        }
        const float top = unordered(top_key);
        const float weight = mine_key ? expf(unordered(mine_key) - top) : 0.f;
        float sum = weight;
        if (!p.renorm) {
            sum = 0.f;
            if (top_key) {
#pragma unroll
                for (int v = 0; v < V; ++v) sum += expf(x[v] - top);
            }
        }
        sum = lanes_sum<LANES>(sum);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (real && l < p.topk) {
            const int mine = mine_key ? choice[i][l] : -1;
            if (!mine_key) choice[i][l] = -1;
            p.experts[t * p.topk + l] = mine;
            p.weights[t * p.topk + l] = mine_key ? weight / sum : 0.f;
            if (mine_key) atomicOr(reinterpret_cast<unsigned long long*>(&chosen[mine]), 1ull << i);
        }
    }
    __syncthreads();
    const bool alone = p.nblocks == 1;
    if (alone) {
        const int n = tid < p.E ? __popcll(chosen[tid]) : 0;      // E <= 1024 threads
        const int upto = block_scan(n, scratch);
        if (tid < p.E) first[tid] = upto - n;
        if (tid == p.E - 1) first[p.E] = upto;
        __syncthreads();
        for (int e = tid; e <= p.E; e += 64 * kRouteWaves) p.offsets[e] = first[e];
        for (int64_t i = first[p.E] + tid; i < p.T * p.topk; i += 64 * kRouteWaves) p.rows[i] = -1;
        if (tid == 0) p.status->flags = bad ? kDevNonFinite : kDevOk;
    } else {
        const int Ep = (p.E + 3) & ~3;
        for (int e = tid; e < Ep; e += 64 * kRouteWaves)
            p.counts[(int64_t)blockIdx.x * Ep + e] = (uint8_t)(e < p.E ? __popcll(chosen[e]) : 0);
        if (tid == 0) p.bad[blockIdx.x] = bad;
    }
    // rank of every choice among the block's (alone: its row)
    for (int i = tid; i < nt * p.topk; i += 64 * kRouteWaves) {
        const int64_t at = t0 * p.topk + i;
        const int tk = i / p.topk, e = choice[tk][i - tk * p.topk];
        int pos = -1;
        if (e >= 0) {
            pos = __popcll(chosen[e] & ((1ull << tk) - 1ull));
            if (alone) {
                pos += first[e];
                p.rows[pos] = (int)(t0 + tk);
            }
        }
        p.positions[at] = pos;
    }
}

// Many blocks: an expert's tokens in every group of kGroupBlocks blocks.  A thread takes four experts.
__global__ __launch_bounds__(256) void group_counts_kernel(RouteArgs p) {
    const int words = (p.E + 3) >> 2, word = threadIdx.x;
    if (word >= words) return;
    const int64_t k0 = (int64_t)blockIdx.x * kGroupBlocks;
    const int n = (int)min((int64_t)kGroupBlocks, p.nblocks - k0);
    const uint32_t* counts = reinterpret_cast<const uint32_t*>(p.counts) + k0 * words + word;
    uint32_t w[2] = {0, 0};                           // experts 0 and 2, 1 and 3: 64 counts of at most 64 fit 16 bits
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
        const uint32_t c = counts[(int64_t)k * words];
        w[0] += c & 0x00FF00FFu;
        w[1] += (c >> 8) & 0x00FF00FFu;
    }
    int32_t* to = p.before + (int64_t)blockIdx.x * p.E + 4 * word;
    for (int i = 0; i < 4 && 4 * word + i < p.E; ++i) to[i] = (int)(w[i & 1] >> (i & 2 ? 16 : 0) & 0xFFFFu);
}

// Then, for 32 experts a workgroup, their sums over the groups before, in place, and over all.
__global__ __launch_bounds__(1024) void scan_groups_kernel(RouteArgs p) {
    constexpr int kParts = 32, kAhead = 8;
    __shared__ int sums[kParts][32];
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    const int ngroups = (p.nblocks + kGroupBlocks - 1) / kGroupBlocks, per = (ngroups + kParts - 1) / kParts;
    const int g0 = min(part * per, ngroups), g1 = e < p.E ? min(g0 + per, ngroups) : g0;
    int sum = 0;
#pragma unroll 8
    for (int g = g0; g < g1; ++g) sum += p.before[(int64_t)g * p.E + e];
    sums[part][lane] = sum;
    __syncthreads();
    int at = 0;
    for (int q = 0; q < part; ++q) at += sums[q][lane];
    for (int g = g0; g < g1; g += kAhead) {
        int v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) v[i] = g + i < g1 ? p.before[(int64_t)(g + i) * p.E + e] : 0;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (g + i < g1) {
                p.before[(int64_t)(g + i) * p.E + e] = at;
                at += v[i];
            }
    }
    if (part == kParts - 1 && e < p.E) p.whole[e] = at;
}

// Last launch: the first row of every expert for this block, then the rows of its tokens.  It adds up the counts of all
// blocks or, GROUPED, those of its group's blocks before it.
template <bool GROUPED>
__global__ __launch_bounds__(64 * kRouteWaves) void place_kernel(RouteArgs p) {
    __shared__ int before[kRouteMaxExperts], whole[kRouteMaxExperts];
    __shared__ int scratch[kRouteWaves];
    __shared__ int valid;
    const int tid = threadIdx.x, nthreads = 64 * kRouteWaves;
    const int64_t t0 = (int64_t)blockIdx.x * kBlockTokens;
    const int nt = (int)(p.T - t0 < kBlockTokens ? p.T - t0 : kBlockTokens);
    constexpr int kMine = kBlockTokens * kRouteMaxTopk / (64 * kRouteWaves);
    int expert[kMine], rank[kMine];                   // this thread's choices, on their way meanwhile
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
        const int i = tid + u * nthreads;
        expert[u] = rank[u] = -1;
        if (i < nt * p.topk) {
            expert[u] = p.experts[t0 * p.topk + i];
            rank[u] = p.positions[t0 * p.topk + i];
        }
    }
    const int64_t group = blockIdx.x / kGroupBlocks;
    const int begin = GROUPED ? (int)group * kGroupBlocks : 0, blocks_end = GROUPED ? (int)blockIdx.x : p.nblocks;
    for (int e = tid; e < kRouteMaxExperts; e += nthreads) {
        before[e] = GROUPED && e < p.E ? p.before[group * p.E + e] : 0;
        whole[e] = 0;
    }
    __syncthreads();
    // threads side by side take four experts each; what is left of the workgroup splits the blocks
    const int words = (p.E + 3) >> 2, parts = nthreads / words, part = tid / words, word = tid - part * words;
    const uint32_t* counts = reinterpret_cast<const uint32_t*>(p.counts) + word;
    constexpr int kSum = 512;                         // bytes of at most 64 that 16 bits hold the sum of
    if (part < parts) {
        for (int k0 = begin + part; k0 < blocks_end; k0 += kSum * parts) {
            uint32_t w[2] = {0, 0}, b[2] = {0, 0};    // experts 0 and 2, 1 and 3
            const int end = (int)min((int64_t)blocks_end, k0 + (int64_t)kSum * parts);
#pragma unroll 8
            for (int k = k0; k < end; k += parts) {
                const uint32_t c = counts[(int64_t)k * words], c0 = c & 0x00FF00FFu, c1 = (c >> 8) & 0x00FF00FFu;
                const bool ahead = k < (int)blockIdx.x;
                w[0] += c0;
                w[1] += c1;
                b[0] += ahead ? c0 : 0u;
                b[1] += ahead ? c1 : 0u;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                atomicAdd(&before[4 * word + i], (int)(b[i & 1] >> (i & 2 ? 16 : 0) & 0xFFFFu));
                atomicAdd(&whole[4 * word + i], (int)(w[i & 1] >> (i & 2 ? 16 : 0) & 0xFFFFu));
            }
        }
    }
    __syncthreads();
    const int n = tid < p.E ? GROUPED ? p.whole[tid] : whole[tid] : 0;      // E <= 1024 threads
    const int upto = block_scan(n, scratch);
    if (tid < p.E) {
        before[tid] += upto - n;
        if (blockIdx.x == 0) {
            p.offsets[tid] = upto - n;
            if (tid == p.E - 1) p.offsets[p.E] = upto;
        }
        if (tid == p.E - 1) valid = upto;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
        if (expert[u] >= 0) {
            const int i = tid + u * nthreads, pos = before[expert[u]] + rank[u];
            p.positions[t0 * p.topk + i] = pos;
            p.rows[pos] = (int)(t0 + i / p.topk);
        }
    }
    for (int64_t i = valid + (int64_t)blockIdx.x * nthreads + tid; i < p.T * p.topk;
         i += (int64_t)gridDim.x * nthreads)
        p.rows[i] = -1;
    if (blockIdx.x == 0) {
        uint32_t any = 0;
        for (int k = tid; k < p.nblocks; k += nthreads) any |= p.bad[k];
        const int found = __syncthreads_or((int)any);
        if (tid == 0) p.status->flags = found ? kDevNonFinite : kDevOk;
    }
}

__global__ void route_nothing_kernel(int32_t* offsets, int E, DevStatus* status) {
    for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = 0;
    if (threadIdx.x == 0) status->flags = kDevOk;
}

// out_t = sum_j weights_tj Y[positions_tj], in the order of j, in fp32.  Bound by HBM: a thread takes eight (bf16) or
// four (fp32) columns of one token, its topk pieces in flight together (16384 tokens, 8 choices, some dropped, 4096 bf16
// columns: 1.15 GB in 228 us, 5.0 TB/s; 8 tokens, 2 choices: 3 us, the launch).
template <bool F32, bool VEC>
__global__ __launch_bounds__(256) void combine_kernel(const void* Y, int64_t M, int64_t ldy, const int32_t* positions,
                                                      const float* weights, int topk, int64_t N, void* out,
                                                      int64_t ldo) {
    constexpr int C = VEC ? (F32 ? 4 : 8) : 1;
    const int64_t t = blockIdx.x;
    const int64_t c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * C;
    if (c >= N) return;
    const int32_t* pos = positions + t * topk;
    const float* w = weights + t * topk;
    float acc[C];
#pragma unroll
    for (int i = 0; i < C; ++i) acc[i] = 0.f;
#pragma unroll 8
    for (int j = 0; j < topk; ++j) {
        const int64_t r = pos[j];
        if (r < 0 || r >= M) continue;
        const float wj = w[j];
        if constexpr (VEC && F32) {
            const f32x4 y = *reinterpret_cast<const f32x4*>(static_cast<const float*>(Y) + r * ldy + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = fmaf(wj, y[i], acc[i]);
        } else if constexpr (VEC) {
            const u32x4 y = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(Y) + r * ldy + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[2 * i] = fmaf(wj, bf16lo_to_f32(y[i]), acc[2 * i]);
                acc[2 * i + 1] = fmaf(wj, bf16hi_to_f32(y[i]), acc[2 * i + 1]);
            }
        } else if constexpr (F32) {
            acc[0] = fmaf(wj, static_cast<const float*>(Y)[r * ldy + c], acc[0]);
        } else {
            acc[0] = fmaf(wj, __uint_as_float((uint32_t) static_cast<const uint16_t*>(Y)[r * ldy + c] << 16), acc[0]);
        }
    }
    if constexpr (VEC && F32) {
        *reinterpret_cast<f32x4*>(static_cast<float*>(out) + t * ldo + c) = f32x4{acc[0], acc[1], acc[2], acc[3]};
    } else if constexpr (VEC) {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2_rne(acc[2 * i], acc[2 * i + 1]);
        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + t * ldo + c) = o;
    } else if constexpr (F32) {
        static_cast<float*>(out)[t * ldo + c] = acc[0];
    } else {
        static_cast<__bf16*>(out)[t * ldo + c] = (__bf16)acc[0];
    }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether the blocks' counts are first added up by groups, two short launches more, or by every block for itself, which
// reads blocks^2 E bytes from L2 (1024 blocks, 64 experts: 24 us the second way, 31 the first; 256 experts: 77 and 71;
// 2048 blocks, 8 experts: 54 and 42; 16384 blocks, 128 experts: 2785 and 462).
bool counts_by_groups(int64_t blocks, int64_t E) { return blocks > 1024 || blocks * blocks * E > (int64_t)1 << 27; }

struct RouteBuffers {
    DevStatus* status;
    uint8_t* counts;
    uint32_t* bad;
    int32_t *before, *whole;
    size_t bytes;
    RouteBuffers(int64_t T, int64_t E, void* ws) {
        const size_t blocks = (size_t)ceil_div(T, kBlockTokens);
        Carver c(ws);
        status = c.take<DevStatus>(1);
        counts = c.take<uint8_t>(blocks > 1 ? blocks * align_up((size_t)E, 4) : 0);
        bad = c.take<uint32_t>(blocks > 1 ? blocks : 0);
        const bool grouped = counts_by_groups(blocks, E);
        before = grouped ? c.take<int32_t>((blocks + kGroupBlocks - 1) / kGroupBlocks * (size_t)E) : nullptr;
        whole = grouped ? c.take<int32_t>((size_t)E) : nullptr;
        bytes = c.bytes();
    }
};

}  // namespace

size_t route_workspace_bytes(int64_t T, int64_t E) { return RouteBuffers(T, E, nullptr).bytes; }

hipError_t route(const void* logits, bool f32, int64_t T, int64_t E, int64_t ld, int topk, bool renorm, float* weights,
                 int32_t* experts, int32_t* offsets, int32_t* rows, int32_t* positions, void* workspace,
                 hipStream_t stream) {
    const RouteBuffers buf(T, E, workspace);
    if (T == 0) {
        hipLaunchKernelGGL(route_nothing_kernel, dim3(1), dim3(256), 0, stream, offsets, (int)E, buf.status);
        return hipGetLastError();
    }
    RouteArgs p;
    p.logits = logits; p.T = T; p.ld = ld; p.E = (int)E; p.topk = topk; p.renorm = renorm;
    p.weights = weights; p.experts = experts; p.offsets = offsets; p.rows = rows; p.positions = positions;
    p.status = buf.status; p.counts = buf.counts; p.bad = buf.bad;
    p.nblocks = (int)ceil_div(T, kBlockTokens);
    p.before = buf.before; p.whole = buf.whole;
    const dim3 grid((unsigned)p.nblocks), block(64 * kRouteWaves);
#define GPTQ_ROUTE(LANES, V)                                                                      \
    do {                                                                                          \
        if (f32) hipLaunchKernelGGL((route_kernel<LANES, V, true>), grid, block, 0, stream, p);   \
        else hipLaunchKernelGGL((route_kernel<LANES, V, false>), grid, block, 0, stream, p);      \
    } while (0)
    if (E <= 128 && topk <= 16) {                     // a lane keeps a choice: 16 lanes hold 16
        if (E <= 16) GPTQ_ROUTE(16, 1);
        else if (E <= 32) GPTQ_ROUTE(16, 2);
        else if (E <= 64) GPTQ_ROUTE(16, 4);
        else GPTQ_ROUTE(16, 8);
    } else if (E <= 256) {
        GPTQ_ROUTE(64, 4);
    } else {
        GPTQ_ROUTE(64, 16);
    }
#undef GPTQ_ROUTE
    if (p.nblocks > 1) {
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (p.before) {
            hipLaunchKernelGGL(group_counts_kernel, dim3((unsigned)ceil_div(p.nblocks, kGroupBlocks)), dim3(256), 0, stream, p);
            hipLaunchKernelGGL(scan_groups_kernel, dim3((unsigned)ceil_div(E, 32)), dim3(1024), 0, stream, p);
        }
        if (p.before) hipLaunchKernelGGL(place_kernel<true>, grid, block, 0, stream, p);
        else hipLaunchKernelGGL(place_kernel<false>, grid, block, 0, stream, p);
    }
    return hipGetLastError();
}

hipError_t combine(const void* Y, bool f32, int64_t M, int64_t ldy, const int32_t* positions, const float* weights,
                   int64_t T, int topk, int64_t N, void* out, int64_t ldo, hipStream_t stream) {
    const int c = f32 ? 4 : 8;
    const bool vec = N % c == 0 && ldy % c == 0 && ldo % c == 0 && aligned16(Y) && aligned16(out);
    constexpr int64_t kMost = 1 << 23;                // a launch has fewer than 2^32 threads along x
    for (int64_t t0 = 0; t0 < T; t0 += kMost) {
        const dim3 grid((unsigned)std::min(T - t0, kMost), (unsigned)ceil_div(N, (int64_t)256 * (vec ? c : 1)));
        const int32_t* pos = positions + t0 * topk;
        const float* w = weights + t0 * topk;
        void* to = static_cast<char*>(out) + t0 * ldo * (f32 ? 4 : 2);
#define GPTQ_COMBINE(F, V) \
    hipLaunchKernelGGL((combine_kernel<F, V>), grid, dim3(256), 0, stream, Y, M, ldy, pos, w, topk, N, to, ldo)
        if (f32) {
            if (vec) GPTQ_COMBINE(true, true);
            else GPTQ_COMBINE(true, false);
        } else {
            if (vec) GPTQ_COMBINE(false, true);
            else GPTQ_COMBINE(false, false);
        }
#undef GPTQ_COMBINE
    }
    return hipGetLastError();
}

}  // namespace gptq
