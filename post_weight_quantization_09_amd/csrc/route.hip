// Routing of tokens to experts and joining their results on gfx950.
//
// Routing, per token t: p = softmax(logits_t); the topk experts with the largest p (ties: the lowest index), weights p
// or p over their sum; then a stable counting sort of the (token, choice) pairs by expert.  Bound by latency: the data
// are a few hundred bytes per token.  One wave takes a token: its logits stay in registers (E / 64 per lane) as
// integers in the order of the values, and every choice is one maximum over the wave (six DPP steps, no LDS) and the
// first lane that holds it.  The sort
// needs, per block of kBlockTokens tokens and expert, which tokens chose it: a bitmap in LDS, whose popcounts are both
// the block's count and the token's rank, whatever order the waves ran in.  Up to one block of tokens everything is one
// launch; else a second launch adds up the blocks' counts (each block for itself, from L2) and places the rows.
#include "route.hpp"

#include <algorithm>

namespace gptq {

namespace {

constexpr int kBlockTokens = 64;
constexpr int kRouteWaves = 16;

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
    int32_t* counts;        // [block][E]
    uint32_t* bad;          // [block]
    int nblocks;
};

// Maximum over the wave, by data-parallel moves: within rows of 16 lanes, then across them; lane 63 has it.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define GPTQ_DPP_MAX(CTRL) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false))
    GPTQ_DPP_MAX(0x111);   // from 1, 2, 4, 8 lanes below
    GPTQ_DPP_MAX(0x112);
    GPTQ_DPP_MAX(0x114);
    GPTQ_DPP_MAX(0x118);
    GPTQ_DPP_MAX(0x142);   // lane 15 of each row to the next row
    GPTQ_DPP_MAX(0x143);   // lane 31 to the upper half
#undef GPTQ_DPP_MAX
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

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

template <int V, bool F32>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs p) {
    __shared__ uint64_t chosen[V * 64];               // per expert: the block's tokens that chose it
    __shared__ int first[V * 64 + 1];
    __shared__ int scratch[kRouteWaves];
    __shared__ uint32_t bad;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < p.E; e += 64 * kRouteWaves) chosen[e] = 0;
    if (tid == 0) bad = 0;
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * kBlockTokens;
    const int nt = (int)(p.T - t0 < kBlockTokens ? p.T - t0 : kBlockTokens);
    constexpr int kTurns = kBlockTokens / kRouteWaves;
    float all[kTurns][V];                             // the wave's tokens, loaded together
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
        const int64_t t = t0 + min(wave + u * kRouteWaves, nt - 1);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = 64 * v + lane;
            all[u][v] = -INFINITY;
            if (e < p.E) {
                if (F32) all[u][v] = static_cast<const float*>(p.logits)[t * p.ld + e];
                else all[u][v] = __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.logits)[t * p.ld + e] << 16);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
        const int i = wave + u * kRouteWaves;
        if (i >= nt) break;
        const int64_t t = t0 + i;
        const float (&x)[V] = all[u];
        uint32_t key[V];                              // 0: not to be chosen (any more)
        bool wrong = false;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            wrong |= !(x[v] < INFINITY);
            key[v] = x[v] > -INFINITY ? ordered(x[v]) : 0u;
        }
        if (__any(wrong)) {                           // NaN or +infinity: reported, and the token chooses nothing
            if (lane == 0) atomicOr(&bad, 1u);
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = 0;
        }
        // choice j ends up in lane j, its exponential is taken there at the end
        int mine = -1;
        uint32_t mine_key = 0, top_key = 0;
        for (int j = 0; j < p.topk; ++j) {
            uint32_t k = key[0];
#pragma unroll
            for (int v = 1; v < V; ++v) k = max(k, key[v]);
            k = wave_max(k);
            if (k == 0) break;
            if (j == 0) top_key = k;
            int e = -1;                               // the first expert with this logit
#pragma unroll
            for (int v = V - 1; v >= 0; --v) {
                const uint64_t has = __ballot(key[v] == k);
                if (has) e = 64 * v + __builtin_ctzll(has);
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (64 * v + lane == e) key[v] = 0;
            if (lane == j) {
                mine = e;
                mine_key = k;
            }
        }
        const float top = unordered(top_key);
        const float weight = mine >= 0 ? expf(unordered(mine_key) - top) : 0.f;
        float sum = weight;
        if (!p.renorm) {
            sum = 0.f;
            if (top_key) {
#pragma unroll
                for (int v = 0; v < V; ++v) sum += expf(x[v] - top);
            }
        }
        sum = wave_sum(sum);
        if (lane < p.topk) {
            p.experts[t * p.topk + lane] = mine;
            p.weights[t * p.topk + lane] = mine >= 0 ? weight / sum : 0.f;
            if (mine >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&chosen[mine]), 1ull << i);
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
        for (int e = tid; e < p.E; e += 64 * kRouteWaves)
            p.counts[(int64_t)blockIdx.x * p.E + e] = __popcll(chosen[e]);
        if (tid == 0) p.bad[blockIdx.x] = bad;
    }
    // rank of every choice among the block's (alone: its row)
    for (int i = tid; i < nt * p.topk; i += 64 * kRouteWaves) {
        const int64_t at = t0 * p.topk + i;
        const int e = p.experts[at], tk = i / p.topk;
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

// Second launch: the first row of every expert for this block, then the rows of its tokens.
__global__ __launch_bounds__(64 * kRouteWaves) void place_kernel(RouteArgs p) {
    __shared__ int before[kRouteMaxExperts], whole[kRouteMaxExperts];
    __shared__ int scratch[kRouteWaves];
    __shared__ int valid;
    const int tid = threadIdx.x, nthreads = 64 * kRouteWaves;
    for (int e = tid; e < p.E; e += nthreads) before[e] = whole[e] = 0;
    __syncthreads();
    // threads side by side take experts side by side; what is left of the workgroup splits the blocks
    const int parts = nthreads / p.E > 0 ? nthreads / p.E : 1;
    for (int i = tid; i < parts * p.E; i += nthreads) {
        const int e = i % p.E, part = i / p.E;
        int b = 0, w = 0;
#pragma unroll 8
        for (int k = part; k < p.nblocks; k += parts) {
            const int c = p.counts[(int64_t)k * p.E + e];
            w += c;
            b += k < (int)blockIdx.x ? c : 0;
        }
        atomicAdd(&before[e], b);
        atomicAdd(&whole[e], w);
    }
    __syncthreads();
    const int n = tid < p.E ? whole[tid] : 0;         // E <= 1024 threads
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
    const int64_t t0 = (int64_t)blockIdx.x * kBlockTokens;
    const int nt = (int)(p.T - t0 < kBlockTokens ? p.T - t0 : kBlockTokens);
    for (int i = tid; i < nt * p.topk; i += nthreads) {
        const int64_t at = t0 * p.topk + i;
        const int e = p.experts[at];
        if (e >= 0) {
            const int pos = before[e] + p.positions[at];
            p.positions[at] = pos;
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
// four (fp32) columns of one token, its topk pieces in flight together.
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

struct RouteBuffers {
    DevStatus* status;
    int32_t* counts;
    uint32_t* bad;
    size_t bytes;
    RouteBuffers(int64_t T, int64_t E, void* ws) {
        const size_t blocks = (size_t)ceil_div(T, kBlockTokens);
        Carver c(ws);
        status = c.take<DevStatus>(1);
        counts = c.take<int32_t>(blocks > 1 ? blocks * (size_t)E : 0);
        bad = c.take<uint32_t>(blocks > 1 ? blocks : 0);
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
    const dim3 grid((unsigned)p.nblocks), block(64 * kRouteWaves);
#define GPTQ_ROUTE(V)                                                                          \
    do {                                                                                       \
        if (f32) hipLaunchKernelGGL((route_kernel<V, true>), grid, block, 0, stream, p);       \
        else hipLaunchKernelGGL((route_kernel<V, false>), grid, block, 0, stream, p);          \
    } while (0)
    if (E <= 64) GPTQ_ROUTE(1);
    else if (E <= 128) GPTQ_ROUTE(2);
    else if (E <= 256) GPTQ_ROUTE(4);
    else GPTQ_ROUTE(16);
#undef GPTQ_ROUTE
    if (p.nblocks > 1) {
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(place_kernel, grid, block, 0, stream, p);
    }
    return hipGetLastError();
}

hipError_t combine(const void* Y, bool f32, int64_t M, int64_t ldy, const int32_t* positions, const float* weights,
                   int64_t T, int topk, int64_t N, void* out, int64_t ldo, hipStream_t stream) {
    const int c = f32 ? 4 : 8;
    const bool vec = N % c == 0 && ldy % c == 0 && ldo % c == 0 && aligned16(Y) && aligned16(out);
    const dim3 grid((unsigned)T, (unsigned)ceil_div(N, (int64_t)256 * (vec ? c : 1)));
#define GPTQ_COMBINE(F, V)                                                                                   \
    hipLaunchKernelGGL((combine_kernel<F, V>), grid, dim3(256), 0, stream, Y, M, ldy, positions, weights, topk, N, \
                       out, ldo)
    if (f32) {
        if (vec) GPTQ_COMBINE(true, true);
        else GPTQ_COMBINE(true, false);
    } else {
        if (vec) GPTQ_COMBINE(false, true);
        else GPTQ_COMBINE(false, false);
    }
#undef GPTQ_COMBINE
    return hipGetLastError();
}

}  // namespace gptq
