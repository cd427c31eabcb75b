// Products with packed weights: the pass that lays the rows out for the tile kernel, workspace, choice of kernel.
#include <algorithm>

#include "matmul_launch.hpp"
#include "matmul_rows.hpp"

namespace gptq {

namespace {

constexpr int kMaxTileRows = 128;

// Row tiles of at most `tile` rows: one list entry (expert, first row, end) per tile, the rows of no expert as expert E,
// the rest of the list expert -1.  One workgroup.
__device__ void list_tiles(const MatmulKernelArgs& p, int tile, int cap, int32_t* tiles) {
    __shared__ int counts[256];
    __shared__ int base;
    const int tid = threadIdx.x;
    if (tid == 0) base = 0;
    __syncthreads();
    const int ranges = p.offsets ? p.E + 2 : 1;
    for (int f = 0; f < ranges; f += 256) {
        const int i = f + tid;
        int64_t lo = 0, hi = 0;
        int e = i;
        if (i < ranges) {
            if (!p.offsets) {
                hi = p.M;
            } else if (i < p.E) {
                expert_rows(p, i, lo, hi);
            } else {
                e = p.E;
                int64_t head = p.offsets[0], tail = p.offsets[p.E];
                head = head < 0 ? 0 : head > p.M ? p.M : head;
                tail = tail < head ? head : tail > p.M ? p.M : tail;
                lo = i == p.E ? 0 : tail;
                hi = i == p.E ? head : p.M;
            }
        }
        const int n = hi > lo ? (int)((hi - lo + tile - 1) / tile) : 0;
        counts[tid] = n;
        __syncthreads();
        for (int d = 1; d < 256; d <<= 1) {
            const int v = tid >= d ? counts[tid - d] : 0;
            __syncthreads();
            counts[tid] += v;
            __syncthreads();
        }
        const int first = base + counts[tid] - n;
        for (int t = 0; t < n && first + t < cap; ++t) {
            tiles[3 * (first + t)] = e;
            tiles[3 * (first + t) + 1] = (int32_t)(lo + (int64_t)t * tile);
            tiles[3 * (first + t) + 2] = (int32_t)(lo + (int64_t)(t + 1) * tile < hi ? lo + (int64_t)(t + 1) * tile : hi);
        }
        __syncthreads();
        if (tid == 255) base += counts[255];
        __syncthreads();
    }
    for (int t = base + tid; t < cap; t += 256) tiles[3 * t] = -1;
}

// Rows -> [part][K / 8][Mp] octets in the operand's order of k, with each row's sums over the scale groups times
// -1.5 2^b.  64 rows x 128 k per workgroup: rows are read in 16-byte pieces along k and written in 16-byte pieces along
// the rows, turned in LDS.  Bound by HBM: every row is read once and written once.
template <int PARTS>
__global__ __launch_bounds__(256) void stage_rows_kernel(MatmulKernelArgs p, uint16_t* XT, float* sums, float excess,
                                                         int tile, int cap, int32_t* tiles) {
    constexpr int kOctets = kChunkK / 8;
    __shared__ u32x4 xt[PARTS][kOctets][65];
    __shared__ float os[kOctets][65];
    if (blockIdx.x == 0 && blockIdx.y == 0) list_tiles(p, tile, cap, tiles);
    const int tid = threadIdx.x;
    const int64_t r0 = (int64_t)blockIdx.x * 64;
    const int chunk = blockIdx.y;
    const int64_t noct = (int64_t)gridDim.y * kOctets;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = (tid >> 4) + 16 * i, o = tid & 15;
        const int64_t r = r0 + row;
        u32x4 part[PARTS];
#pragma unroll
        for (int j = 0; j < PARTS; ++j) part[j] = u32x4{0u, 0u, 0u, 0u};
        const int64_t s = r < p.M ? source_row(p, r) : -1;
        if (s >= 0)
            load_octet<PARTS>(static_cast<const char*>(p.X) + s * p.ldx * (PARTS == 1 ? 2 : 4),
                              (int64_t)chunk * kChunkK + 8 * o, p.K, part);
        float sum = 0.f;
#pragma unroll
        for (int d = 0; d < 4; ++d) sum += bf16lo_to_f32(part[0][d]) + bf16hi_to_f32(part[0][d]);
#pragma unroll
        for (int j = 0; j < PARTS; ++j) xt[j][o][row] = pair_order(part[j]);
        os[o][row] = sum;
    }
    __syncthreads();
    const int row = tid & 63;
    if (r0 + row >= p.M) return;
#pragma unroll
    for (int j = 0; j < PARTS; ++j)
#pragma unroll
        for (int i = 0; i < kOctets / 4; ++i) {
            const int o = (tid >> 6) + 4 * i;
            reinterpret_cast<u32x4*>(XT)[(j * noct + (int64_t)chunk * kOctets + o) * p.Mp + r0 + row] = xt[j][o][row];
        }
    if (PARTS > 1) return;                           // fp32 rows: the codes come without the excess
    const int groups = kChunkSteps / p.group_steps;
    for (int g = tid >> 6; g < groups; g += 4) {
        float s = 0.f;
        for (int o = 0; o < 4 * p.group_steps; ++o) s += os[g * 4 * p.group_steps + o][row];
        sums[((int64_t)chunk * groups + g) * p.Mp + r0 + row] = excess * s;
    }
}

// Z = H B^T for many rows of short requests (single tokens beside each other): one thread per row and four channels.
__global__ __launch_bounds__(256) void adapter_expand_kernel(MatmulKernelArgs p, float* Z) {
    const int lane = threadIdx.x & 63;
    const int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), c0 = ((int64_t)blockIdx.y * 64 + lane) * 4;
    if (r >= p.M || c0 >= p.N) return;
    LaneChannels<4, false> ch(0, 0, p.N);
    ch.c0 = c0 < p.N - 4 ? c0 : p.N - 4;
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    add_adapter_row<4, false>(p, r, ch, y);
    *reinterpret_cast<f32x4_a4*>(Z + r * p.N + ch.c0) = f32x4{y[0], y[1], y[2], y[3]};
}

// Rows an expert is expected to have; the kernels hold for any split, this only chooses.
int64_t rows_per_expert(int64_t M, int64_t experts) { return ceil_div(M, std::max<int64_t>(1, experts)); }

bool use_tiles(int64_t M, int64_t experts) { return rows_per_expert(M, experts) > 64; }

int tile_rows(bool f32, int64_t M, int64_t N, int64_t experts) {
    if (f32 || ceil_div(M, 128) * ceil_div(N, 256) < 256) return 64;
    return 128;
}

struct Plan {
    bool tiles;
    int tile;
    int cap;               // entries of the tile list
    int64_t Mp;
    int nchunks;
    size_t xt_elems, sum_floats;
    int hrank;
};

Plan make_plan(bool f32, int64_t M, int64_t K, int64_t N, int64_t experts, int64_t rank) {
    Plan p;
    p.tiles = use_tiles(M, experts);
    p.tile = tile_rows(f32, M, N, experts);
    p.cap = (int)(M / p.tile + std::min<int64_t>(experts + 2, M) + 1);
    p.Mp = (int64_t)align_up((size_t)M + kMaxTileRows, 64);
    p.nchunks = (int)ceil_div(K, kChunkK);
    p.xt_elems = (size_t)(f32 ? 3 : 1) * p.nchunks * kChunkK * p.Mp;
    p.sum_floats = (size_t)p.nchunks * kChunkSteps * p.Mp;
    p.hrank = (int)align_up((size_t)rank, 8);
    return p;
}

struct Buffers {
    float* H;
    int32_t* row_adapter;
    uint16_t* XT;
    float* sums;
    int32_t* tiles;
    size_t bytes;
    float* Z;
    Buffers(const Plan& p, int64_t M, int64_t N, void* ws) {
        Carver c(ws);
        H = p.hrank ? c.take<float>((size_t)M * p.hrank) : nullptr;
        row_adapter = p.hrank ? c.take<int32_t>((size_t)M) : nullptr;
        XT = p.tiles ? c.take<uint16_t>(p.xt_elems) : nullptr;
        sums = p.tiles ? c.take<float>(p.sum_floats) : nullptr;
        tiles = p.tiles ? c.take<int32_t>(3 * (size_t)p.cap) : nullptr;
        Z = p.tiles && p.hrank ? c.take<float>((size_t)M * N) : nullptr;
        bytes = c.bytes();
    }
};

// A tile takes one small product per run of rows with the same adapter: about 1 us each, against M N fp32 values written
// and read again for Z.  Runs of 32 rows and more (prompts) go the first way, single tokens the second.
bool short_requests(int64_t M, int64_t n_requests) { return M < 32 * n_requests; }

}  // namespace

size_t matmul_workspace_bytes(bool f32, int64_t M, int64_t K, int64_t N, int64_t experts, int64_t rank) {
    return Buffers(make_plan(f32, M, K, N, experts, rank), M, N, nullptr).bytes;
}

hipError_t packed_matmul(const MatmulArgs& a, void* workspace, hipStream_t stream) {
    const bool lora = a.n_requests > 0 && a.n_adapters > 0;
    const Plan plan = make_plan(a.f32, a.M, a.K, a.N, a.E, lora ? a.rank : 0);
    const Buffers buf(plan, a.M, a.N, workspace);
    MatmulKernelArgs k;
    k.X = a.X; k.ldx = a.ldx; k.x_rows = a.x_rows; k.rows = a.rows; k.M = a.M;
    k.offsets = a.offsets; k.E = a.E;
    k.packed = a.packed; k.ldp = a.ldp; k.p_stride = a.p_stride; k.K = a.K; k.N = a.N;
    k.nwords = (int)((a.K * a.bits + 31) / 32);
    k.scales = a.scales; k.s_stride = a.s_stride;
    k.group_steps = a.groupsize ? a.groupsize / kStepK : kChunkSteps;
    k.s_row = a.groupsize ? a.N : 0;
    k.last_group = a.groupsize ? (a.K - 1) / a.groupsize : 0;
    k.Y = a.Y; k.ldy = a.ldy;
    k.H = lora ? buf.H : nullptr;
    k.hrank = plan.hrank; k.row_adapter = buf.row_adapter;
    k.B = a.B; k.ldb = a.ldb; k.b_stride = a.b_stride; k.rank = a.rank;
    k.Z = lora && plan.tiles && short_requests(a.M, a.n_requests) ? buf.Z : nullptr;
    k.XT = buf.XT; k.sums = buf.sums; k.Mp = plan.Mp; k.tiles = buf.tiles;
    if (lora) {
        const hipError_t e = adapter_shrink(a, buf.H, plan.hrank, buf.row_adapter, stream);
        if (e != hipSuccess) return e;
        if (k.Z) {
            const dim3 grid((unsigned)ceil_div(a.M, 4), (unsigned)ceil_div(a.N, 256));
            hipLaunchKernelGGL(adapter_expand_kernel, grid, dim3(256), 0, stream, k, buf.Z);
            const hipError_t x = hipGetLastError();
            if (x != hipSuccess) return x;
        }
    }
    if (plan.tiles) {
        const dim3 grid((unsigned)ceil_div(a.M, 64), (unsigned)plan.nchunks);
        const float excess = -1.5f * (float)(1 << a.bits);
        if (a.f32)
            hipLaunchKernelGGL((stage_rows_kernel<3>), grid, dim3(256), 0, stream, k, buf.XT, buf.sums, excess,
                               plan.tile, plan.cap, buf.tiles);
        else
            hipLaunchKernelGGL((stage_rows_kernel<1>), grid, dim3(256), 0, stream, k, buf.XT, buf.sums, excess,
                               plan.tile, plan.cap, buf.tiles);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        switch (a.bits) {
            case 2: return tile_b2(k, a.f32, plan.tile / 16, plan.cap, a.swiglu, stream);
            case 3: return tile_b3(k, a.f32, plan.tile / 16, plan.cap, a.swiglu, stream);
            case 4: return tile_b4(k, a.f32, plan.tile / 16, plan.cap, a.swiglu, stream);
            case 5: return tile_b5(k, a.f32, plan.tile / 16, plan.cap, a.swiglu, stream);
            default: return tile_b6(k, a.f32, plan.tile / 16, plan.cap, a.swiglu, stream);
        }
    }
    const int row_tiles = (int)ceil_div(rows_per_expert(a.M, a.E), 16);
    switch (a.bits) {
        case 2: return rows_b2(k, a.f32, row_tiles, a.swiglu, stream);
        case 3: return rows_b3(k, a.f32, row_tiles, a.swiglu, stream);
        case 4: return rows_b4(k, a.f32, row_tiles, a.swiglu, stream);
        case 5: return rows_b5(k, a.f32, row_tiles, a.swiglu, stream);
        default: return rows_b6(k, a.f32, row_tiles, a.swiglu, stream);
    }
}

}  // namespace gptq
