// Products with packed weights: the pass that prepares the rows, workspace, choice of kernel.
#include <algorithm>
#include <type_traits>

#include "matmul_launch.hpp"
#include "matmul_rows.hpp"

namespace gptq {

namespace {

constexpr int kMaxTileRows = 128;
constexpr int kStageThreads = 512;
constexpr int kStageRows = 64;
constexpr int kMaxKParts = 8;

// What stage_kernel writes.
struct StageArgs {
    uint16_t* XT;
    float* sums;
    int tile, cap;         // rows of a tile, entries of the list
    int32_t* tiles;
    int row_blocks;        // workgroups of the rows: row_blocks x nchunks (0: rows are not laid out)
    int nchunks;
    int64_t workgroups;    // of the launch, counted along x, then y
    // adapters
    const uint16_t* A;
    int64_t lda, a_stride;
    const float* alpha;
    int64_t n_adapters;
    const int32_t* requests;
    const int32_t* adapter;
    int64_t n_requests;
    int slices;            // workgroups of a request along its rows (0: no adapters)
    int k_parts;           // and along K: part z of H is at z * M * hrank
    int64_t windows;       // of one pass's rows, for what is longer (0: no request can be)
    float* H;
    int32_t* row_adapter;
};

// Row tiles of at most `tile` rows: one list entry (expert, first row, end) per tile, the rows of no expert as expert E,
// the rest of the list expert -1.  One workgroup.  Offsets out of order give more tiles than the list has entries, up to E
// times the rows' tiles: they are counted in 64 bits, so that what is left out is what comes past the end.
__device__ void list_tiles(const MatmulKernelArgs& p, const StageArgs& a) {
    constexpr int T = kStageThreads;
    __shared__ int64_t counts[T];
    __shared__ int64_t base;
    const int tid = threadIdx.x;
    if (tid == 0) base = 0;
    __syncthreads();
    const int ranges = p.offsets ? p.E + 2 : 1;
    for (int f = 0; f < ranges; f += T) {
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
        const int n = hi > lo ? (int)((hi - lo + a.tile - 1) / a.tile) : 0;
        counts[tid] = n;
        __syncthreads();
        for (int d = 1; d < T; d <<= 1) {
            const int64_t v = tid >= d ? counts[tid - d] : 0;
            __syncthreads();
            counts[tid] += v;
            __syncthreads();
        }
        const int64_t first = base + counts[tid] - n;
        for (int t = 0; t < n && first + t < a.cap; ++t) {
            const int64_t r = lo + (int64_t)t * a.tile;
            a.tiles[3 * (first + t)] = e;
            a.tiles[3 * (first + t) + 1] = (int32_t)r;
            a.tiles[3 * (first + t) + 2] = (int32_t)(r + a.tile < hi ? r + a.tile : hi);
        }
        __syncthreads();
        if (tid == T - 1) base += counts[T - 1];
        __syncthreads();
    }
    for (int64_t t = base + tid; t < a.cap; t += T) a.tiles[3 * t] = -1;
}

// Rows -> [part][K / 8][Mp] octets in the operand's order of k, with each row's sums over the scale groups times -1.5 2^-8,
// the codes' excess.  64 rows x 128 k per workgroup: rows are read in 16-byte pieces along k and written in 16-byte pieces
// along the rows, turned in LDS.  Bound by HBM: every row is read once and written once (8192 gathered rows x 4096, bf16:
// 27.5 us, 4.9 TB/s).
template <int PARTS>
__device__ void lay_out_rows(const MatmulKernelArgs& p, const StageArgs& a, int64_t r0, int chunk, int nchunks, char* lds) {
    constexpr int kOctets = kChunkK / 8, kPitch = kStageRows + 1;
    u32x4* xt = reinterpret_cast<u32x4*>(lds);                          // [part][octet][row]
    float* os = reinterpret_cast<float*>(xt + PARTS * kOctets * kPitch);
    constexpr float kMinusExcess = -1.5f / (float)(1 << -kCodeExponent);
    const int tid = threadIdx.x;
    const int64_t noct = (int64_t)nchunks * kOctets;
#pragma unroll
    for (int i = 0; i < kStageRows * kOctets / kStageThreads; ++i) {
        const int row = (tid >> 4) + (kStageThreads / 16) * i, o = tid & 15;
        const int64_t r = r0 + row;
        u32x4 part[PARTS];
#pragma unroll
        for (int j = 0; j < PARTS; ++j) part[j] = u32x4{0u, 0u, 0u, 0u};
        const int64_t s = r < p.M ? source_row(p, r) : -1;
        if (s >= 0)
            load_octet<PARTS>(static_cast<const char*>(p.X) + s * p.ldx * (PARTS == 1 ? 2 : 4),
                              chunk * kChunkK + 8 * o, p.K, part);
        float sum = 0.f;
#pragma unroll
        for (int d = 0; d < 4; ++d) sum += kMinusExcess * bf16lo_to_f32(part[0][d]) + kMinusExcess * bf16hi_to_f32(part[0][d]);
#pragma unroll
        for (int j = 0; j < PARTS; ++j) xt[(j * kOctets + o) * kPitch + row] = pair_order(part[j]);
        os[o * kPitch + row] = sum;
    }
    __syncthreads();
    const int row = tid & 63;
    if (r0 + row >= p.M) return;
#pragma unroll
    for (int j = 0; j < PARTS; ++j)
#pragma unroll
        for (int i = 0; i < kOctets / (kStageThreads / 64); ++i) {
            const int o = (tid >> 6) + (kStageThreads / 64) * i;
            reinterpret_cast<u32x4*>(a.XT)[(j * noct + (int64_t)chunk * kOctets + o) * p.Mp + r0 + row] =
                xt[(j * kOctets + o) * kPitch + row];
        }
    if (PARTS > 1) return;                           // fp32 rows: the codes come without the excess
    const int per = 4 << p.lg_group, groups = kOctets / per;             // octets of a group
    for (int g = tid >> 6; g < groups; g += kStageThreads / 64) {
        float s = 0.f;
        for (int o = 0; o < per; ++o) s += os[(g * per + o) * kPitch + row];
        a.sums[((int64_t)chunk * groups + g) * p.Mp + r0 + row] = s;
    }
}

// H of one row: two ranks of a wave at a time, 4096 k with all their loads in flight.
template <int PARTS>
__device__ void single_row(const MatmulKernelArgs& p, const StageArgs& a, int64_t row, int id, float alpha, int lane,
                           int wave) {
    constexpr int W = kStageThreads / 64, kLoads = PARTS == 1 ? 8 : 4, kXBytes = PARTS == 1 ? 2 : 4;
    const char* xrow = static_cast<const char*>(p.X) + row * p.ldx * kXBytes;
    for (int n0 = wave; n0 < p.hrank; n0 += 2 * W) {
        const char* arow[2];
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < 2; ++n) arow[n] = reinterpret_cast<const char*>(a.A + id * a.a_stride + min(n0 + n * W, p.rank - 1) * a.lda);
        for (int k0 = 0; k0 < p.K; k0 += kLoads * 512) {
            RawOctet<PARTS> x[kLoads];
            RawOctet<1> b[2][kLoads];
            auto add = [&](auto masked) {
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    const int k = k0 + u * 512 + 8 * lane, skip = k - min(k, p.K - 8);
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        float x0, x1;
                        if constexpr (PARTS == 1) {
                            x0 = bf16lo_to_f32(x[u].v[0][d]);
                            x1 = bf16hi_to_f32(x[u].v[0][d]);
                        } else {
                            x0 = __uint_as_float(x[u].v[d >> 1][2 * (d & 1)]);
                            x1 = __uint_as_float(x[u].v[d >> 1][2 * (d & 1) + 1]);
                        }
                        if constexpr (decltype(masked)::value) {
                            x0 = 2 * d >= skip ? x0 : 0.f;
                            x1 = 2 * d + 1 >= skip ? x1 : 0.f;
                        }
#pragma unroll
                        for (int n = 0; n < 2; ++n)
                            sum[n] = fmaf(x1, bf16hi_to_f32(b[n][u].v[0][d]), fmaf(x0, bf16lo_to_f32(b[n][u].v[0][d]), sum[n]));
                    }
                }
            };
            if (k0 + kLoads * 512 <= p.K) {
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    const int k = k0 + u * 512 + 8 * lane;
                    x[u].whole(xrow + k * kXBytes);
#pragma unroll
                    for (int n = 0; n < 2; ++n) b[n][u].whole(arow[n] + k * 2);
                }
                add(std::integral_constant<bool, false>{});
            } else if (p.K >= 8) {                   // the last octet is read from further left, what is another's masked
#pragma unroll
                for (int u = 0; u < kLoads; ++u) {
                    const int at = min(k0 + u * 512 + 8 * lane, p.K - 8);
                    x[u].whole(xrow + at * kXBytes);
#pragma unroll
                    for (int n = 0; n < 2; ++n) b[n][u].whole(arow[n] + at * 2);
                }
                add(std::integral_constant<bool, true>{});
            } else if (lane == 0) {                  // rows shorter than an octet
                for (int k = 0; k < p.K; ++k) {
                    float xv;
                    if constexpr (PARTS == 1) xv = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(xrow)[k] << 16);
                    else xv = reinterpret_cast<const float*>(xrow)[k];
#pragma unroll
                    for (int n = 0; n < 2; ++n)
                        sum[n] = fmaf(xv, __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(arow[n])[k] << 16), sum[n]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) sum[n] += __shfl_xor(sum[n], d);
            const int rk = n0 + n * W;
            if (lane == 0 && rk < p.hrank) a.H[row * p.hrank + rk] = rk < p.rank ? alpha * sum[n] : 0.f;
        }
    }
}

// The inner half of the low-rank adapters: H[r] = alpha_a (A_a x_r) for the rows r of one request, a its adapter, and
// the adapter of every row.  Bound by latency and the adapters' bytes for single tokens, by the rows' bytes for prompts.
// A workgroup takes 16 RS rows at a time and the whole rank; its waves split K (each 32-k step one matrix product per 16
// ranks: lane l holds row l % 16 and, of A, rank l % 16, eight consecutive k each, straight from memory; a wave has the
// loads of kAhead steps in flight) and the partial sums are joined in LDS in a fixed order.  One to four tokens are no
// matrix product: there a wave takes a rank and reads its row of A in whole kilobytes (as operands it would be 64 pieces of 16
// bytes), products and sums in fp32 (one token, 4096 features, rank 16: 4.6 against 7.4 us).  Prompts take 64 rows at a
// time, since every pass reads A again, and split K over k_parts workgroups; their sums are added where H is used (4096
// rows x 28672, rank 64, rows laid out beside it: 240 us against 333 with 16 rows and no split).  H stays in fp32.
//
// The launch cannot depend on the lengths, which only the device knows.  Every request gets `slices` workgroups, which
// take one pass each; what is longer is left to `windows` workgroups, one per 16 RS rows of X, which look up the requests
// that reach into theirs (one request of 3841 rows beside 255 of one, 4096 features, rank 16: 53 us; 494 with the
// request's own workgroups alone).

// One pass: the rows r0 .. min(r0 + 16 RS, hi) - 1, for adapter `id`, over this workgroup's part z of K.
template <int PARTS, int NR, int RS>
__device__ void shrink_pass(const MatmulKernelArgs& p, const StageArgs& a, int id, float alpha, int64_t r0, int64_t hi, int z,
                            char* lds) {
    constexpr int W = kStageThreads / 64, kXBytes = PARTS == 1 ? 2 : 4;
    float* part = reinterpret_cast<float*>(lds);     // [wave][rank and row register][lane]
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int whole = p.K / kStepK, per = ((whole + a.k_parts - 1) / a.k_parts + 1) & ~1;
    const int s_begin = min(z * per, whole), s_end = min(s_begin + per, whole);
    float* H = a.H + (int64_t)z * p.M * p.hrank;
    const char* xrow[RS];
#pragma unroll
    for (int t = 0; t < RS; ++t) {
        int64_t r = r0 + 16 * t + (lane & 15);
        if (r >= hi) r = hi - 1;
        xrow[t] = static_cast<const char*>(p.X) + (r * p.ldx + 8 * q) * kXBytes;
    }
    const uint16_t* arow[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        int rk = 16 * n + (lane & 15);
        if (rk >= p.rank) rk = p.rank - 1;           // ranks past the end are not stored
        arow[n] = a.A + id * a.a_stride + rk * a.lda + 8 * q;
    }
    f32x4 acc[RS][NR];
#pragma unroll
    for (int t = 0; t < RS; ++t)
#pragma unroll
        for (int n = 0; n < NR; ++n) acc[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    // pairs of steps (128 bytes of a bf16 row) are dealt out to the waves, kAhead steps at a time
    constexpr int kAhead = RS > 1 || NR * PARTS > 4 ? 2 : 8;
    constexpr int kTurn = 2 * W;
    for (int s0 = s_begin + 2 * wave; s0 < s_end; s0 += kTurn * (kAhead / 2)) {
        RawOctet<PARTS> x[kAhead][RS];
        RawOctet<1> b[kAhead][NR];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            int s = s0 + (u >> 1) * kTurn + (u & 1);
            s = s < s_end ? s : s0;                  // beyond the end: loaded again and not used
#pragma unroll
            for (int t = 0; t < RS; ++t) x[u][t].whole(xrow[t] + s * (kStepK * kXBytes));
#pragma unroll
            for (int n = 0; n < NR; ++n) b[u][n].whole(reinterpret_cast<const char*>(arow[n] + s * kStepK));
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (s0 + (u >> 1) * kTurn + (u & 1) < s_end) {
#pragma unroll
                for (int t = 0; t < RS; ++t) {
                    u32x4 xp[PARTS];
                    x[u][t].parts(xp);
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int i = 0; i < PARTS; ++i)
                            acc[t][n] = mfma16(xp[i], __builtin_bit_cast(bf16x8, b[u][n].v[0]), acc[t][n]);
                }
            }
        }
    }
    if (z == a.k_parts - 1 && wave == W - 1 && whole * kStepK < p.K) {   // the rest of K
        u32x4 x[PARTS], b[1];
        const int k = whole * kStepK, left = p.K - k - 8 * q;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            load_octet<1>(arow[n], k, k + left, b);
#pragma unroll
            for (int t = 0; t < RS; ++t) {
                load_octet<PARTS>(xrow[t], k, k + left, x);
#pragma unroll
                for (int i = 0; i < PARTS; ++i) acc[t][n] = mfma16(x[i], __builtin_bit_cast(bf16x8, b[0]), acc[t][n]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < RS; ++t) {
        __syncthreads();                             // the partials before these have been read
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[(wave * NR * 4 + n * 4 + i) * 64 + lane] = acc[t][n][i];
        __syncthreads();
        for (int v = wave; v < NR * 4; v += W) {
            float s = 0.f;
#pragma unroll
            for (int u = 0; u < W; ++u) s += part[(u * NR * 4 + v) * 64 + lane];
            const int64_t row = r0 + 16 * t + 4 * q + (v & 3);
            const int rk = 16 * (v >> 2) + (lane & 15);
            if (row < hi && rk < p.hrank) H[row * p.hrank + rk] = rk < p.rank ? s * alpha : 0.f;
        }
    }
}

// The rows of request `req`: their adapter, and one pass of A x per workgroup (single tokens: all of it).
template <int PARTS, int NR, int RS>
__device__ void shrink_rows(const MatmulKernelArgs& p, const StageArgs& a, int64_t req, int slice, int z, char* lds) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (req == a.n_requests) {                       // rows of no request
        if (slice || z) return;
        int64_t head = a.requests[0], tail = a.requests[a.n_requests];
        head = head < 0 ? 0 : head > p.M ? p.M : head;
        tail = tail < head ? head : tail > p.M ? p.M : tail;
        for (int64_t r = tid; r < head; r += kStageThreads) a.row_adapter[r] = -1;
        for (int64_t r = tail + tid; r < p.M; r += kStageThreads) a.row_adapter[r] = -1;
        return;
    }
    int64_t lo = a.requests[req], hi = a.requests[req + 1];
    lo = lo < 0 ? 0 : lo;
    hi = hi > p.M ? p.M : hi;
    int id = a.adapter[req];
    if (id < 0 || id >= a.n_adapters) id = -1;
    const float alpha = id < 0 ? 0.f : a.alpha[id];
    if (hi - lo <= 4 && a.k_parts == 1) {
        for (int64_t r = lo + slice; r < hi; r += a.slices) {
            if (tid == 0) a.row_adapter[r] = id;
            if (id >= 0) single_row<PARTS>(p, a, r, id, alpha, lane, wave);
        }
        return;
    }
    if (z == 0)
        for (int64_t r = lo + slice * kStageThreads + tid; r < hi; r += (int64_t)a.slices * kStageThreads) a.row_adapter[r] = id;
    const int64_t r0 = lo + 16 * RS * (int64_t)slice;
    if (id >= 0 && r0 < hi) shrink_pass<PARTS, NR, RS>(p, a, id, alpha, r0, hi, z, lds);
}

// The rows of one window that their requests' own workgroups do not reach.  The requests are looked through side by side, from
// the one that the window's first row belongs to (found by halving) where they are many.
template <int PARTS, int NR, int RS>
__device__ void shrink_window(const MatmulKernelArgs& p, const StageArgs& a, int64_t window, int z, char* lds) {
    constexpr int T = kStageThreads;
    __shared__ int list[T], count;
    const int tid = threadIdx.x;
    const int64_t w0 = window * 16 * RS, w1 = w0 + 16 * RS < p.M ? w0 + 16 * RS : p.M;
    const int64_t reach = 16 * RS * (int64_t)a.slices;
    int64_t q = 0;
    if (a.n_requests > T) {
        int64_t past = a.n_requests;
        while (past - q > 1) {
            const int64_t mid = (q + past) / 2;
            if (a.requests[mid] <= w0) q = mid;
            else past = mid;
        }
    }
    for (; q < a.n_requests; q += T) {
        if (tid == 0) count = 0;
        __syncthreads();
        auto span = [&](int64_t req, int64_t& begin, int64_t& end) {
            int64_t lo = a.requests[req], hi = a.requests[req + 1];
            lo = lo < 0 ? 0 : lo;
            begin = lo + reach > w0 ? lo + reach : w0;
            end = hi < w1 ? hi : w1;
        };
        int64_t begin = 0, end = 0;
        if (q + tid < a.n_requests) span(q + tid, begin, end);
        if (begin < end) list[atomicAdd(&count, 1)] = (int)(q + tid);    // in any order: each has rows of its own
        __syncthreads();
        const int n = count;
        for (int i = 0; i < n; ++i) {
            const int64_t req = list[i];
            span(req, begin, end);
            const int id = a.adapter[req];
            if (id < 0 || id >= a.n_adapters) continue;
            shrink_pass<PARTS, NR, RS>(p, a, id, a.alpha[id], begin, end, z, lds);
        }
        if (q + T < a.n_requests && a.requests[q + T] >= w1) return;
        __syncthreads();                             // the list has been read
    }
}

// One launch before the product: workgroups of the adapters first (their chains of loads are the longest), then of the
// rows.  NR 0: no adapters.
template <int PARTS, int NR, int RS>
__global__ __launch_bounds__(kStageThreads, 2) void stage_kernel(MatmulKernelArgs p, StageArgs a) {
    constexpr int kLayBytes = PARTS * (kChunkK / 8) * (kStageRows + 1) * 16 + (kChunkK / 8) * (kStageRows + 1) * 4;
    constexpr int kShrinkBytes = (kStageThreads / 64) * NR * 4 * 64 * 4;
    __shared__ __attribute__((aligned(16))) char lds[kLayBytes > kShrinkBytes ? kLayBytes : kShrinkBytes];
    int64_t b = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
    if (b >= a.workgroups) return;
    if constexpr (NR > 0) {
        const int64_t per = (int64_t)a.slices * a.k_parts, n = (a.n_requests + 1) * per;
        if (b < n) {
            const int in = (int)(b % per);
            shrink_rows<PARTS, NR, RS>(p, a, b / per, in / a.k_parts, in % a.k_parts, lds);
            return;
        }
        b -= n;
        if (b < a.windows * a.k_parts) {
            shrink_window<PARTS, NR, RS>(p, a, b / a.k_parts, (int)(b % a.k_parts), lds);
            return;
        }
        b -= a.windows * a.k_parts;
    }
    const int nchunks = a.nchunks;
    if (b == (int64_t)a.row_blocks * nchunks) {
        list_tiles(p, a);
        return;
    }
    lay_out_rows<PARTS>(p, a, b / nchunks * kStageRows, (int)(b % nchunks), nchunks, lds);
}

// Z = H B^T for many rows of short requests (single tokens beside each other).  A wave takes 64 rows and 64 channels: for
// every adapter among the rows, wherever they are, one matrix product of which its rows are kept (and not one with other
// rows of H zero: an infinite or NaN value of B would reach them), so that B is read once for all of them (row by row it
// is read again for every token: 266 tokens of 13 adapters, rank 68, 15296 channels: 200 us against 55).  The next
// operands are on their way while one set is multiplied.
__global__ __launch_bounds__(256, 2) void adapter_expand_kernel(MatmulKernelArgs p, float* Z) {
    constexpr int HP = 3;                            // parts of H: exactly its fp32 value
    constexpr int RT = 4, NT = 4, kMaxOctets = 16;
    __shared__ u32x4 hs[HP][kMaxOctets][64];         // H of the rows as operands
    __shared__ int list[64];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t r0 = (int64_t)blockIdx.x * 64;
    const int mine = r0 + lane < p.M ? p.row_adapter[r0 + lane] : -1;   // adapter of row `lane`
    if (wave == 0) {                                 // the distinct adapters, in the order of their first rows
        bool first = mine >= 0;
        for (int i = 0; i < 63; ++i) first = first && !(i < lane && __builtin_amdgcn_readlane(mine, i) == mine);
        const uint64_t m = __ballot(first);
        if (first) list[__popcll(m & ((1ull << lane) - 1))] = mine;
        if (lane == 0) count = __popcll(m);
    }
    for (int o = wave; o < p.hrank / 8; o += 4) {
        float hv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) hv[i] = mine >= 0 ? p.H[(r0 + lane) * p.hrank + 8 * o + i] : 0.f;
        u32x4 part[3];
        split3(hv, part);
#pragma unroll
        for (int i = 0; i < HP; ++i) hs[i][o][lane] = part[i];
    }
    __syncthreads();
    const LaneChannels<NT, false> ch((blockIdx.y * 4 + wave) * 64, lane, p.N);
    const int n = __builtin_amdgcn_readfirstlane(count);
    int ids[RT][4];                                  // adapters of the rows that this lane has sums of
    f32x4 acc[RT][NT], out[RT][NT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) ids[t][i] = __shfl(mine, 16 * t + 4 * q + i);
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[t][j] = out[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const char* Bc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) Bc[j] = reinterpret_cast<const char*>(p.B + ch.channel(j) * p.ldb + 8 * q);
    const int steps = (p.rank + kStepK - 1) / kStepK, items = n * steps;
    int which = 0, step = 0;                         // of the next item
    RawOctet<1> b[NT];
    auto load = [&] {
        const int64_t id = __builtin_amdgcn_readfirstlane(list[which]);
#pragma unroll
        for (int j = 0; j < NT; ++j)
            b[j].some(Bc[j] + (id * p.b_stride + step * kStepK) * 2, p.rank - step * kStepK - 8 * q, p.rank);
        if (++step == steps) {
            step = 0;
            ++which;
        }
    };
    if (items) load();
    for (int item = 0, id = 0, at = 0, now = 0; item < items; ++item) {
        id = __builtin_amdgcn_readfirstlane(list[now]);
        bf16x8 bv[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) bv[j] = __builtin_bit_cast(bf16x8, b[j].v[0]);
        if (item + 1 < items) load();
        const int o = min(4 * at + q, p.hrank / 8 - 1);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const bool in = 4 * at + q < p.hrank / 8;
#pragma unroll
            for (int i = 0; i < HP; ++i) {
                u32x4 a = hs[i][o][16 * t + (lane & 15)];
#pragma unroll
                for (int d = 0; d < 4; ++d) a[d] = in ? a[d] : 0u;
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[t][j] = mfma16(a, bv[j], acc[t][j]);
            }
        }
        if (++at == steps) {
            at = 0;
            ++now;
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) out[t][j][i] = ids[t][i] == id ? acc[t][j][i] : out[t][j][i];
                    acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
        }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = r0 + 16 * t + 4 * q + i;
            if (r < p.M)
                *reinterpret_cast<f32x4_a4*>(Z + r * p.N + ch.c0) = f32x4{out[t][0][i], out[t][1][i], out[t][2][i], out[t][3][i]};
        }
}

enum Kernel { kRows, kSplit, kTile };

struct Plan {
    Kernel kernel;
    int tile;              // rows of a tile
    int cap;               // entries of the tile list
    int64_t Mp;
    int nchunks;
    size_t xt_elems, sum_floats;
    int hrank;
    int k_parts;
};

// Row tiles of the split kernel: 64 rows fit its registers with one word per step and lane and one scale per 128 k, and
// halve the conversions of codes; else 32 (64 rows of 3-bit codes in groups of 64 spill: 56 us against 28).
int split_row_tiles(bool f32, int64_t mean, int bits, int groupsize) {
    return !f32 && mean > 32 && (bits == 2 || bits == 4) && (groupsize == 0 || groupsize == 128) ? 4 : 2;
}

// Rows of the tile kernel's tiles: 112 where an expert fills several such tiles (the last one is half empty on average)
// and a lane's operand is one word; else 64 (fp32 rows take three operands; with two words per operand seven row tiles
// spill: 4096 rows of 4 experts x 14336 x 2048, 3 bits in groups of 32: 606 us against 393; per channel 402 against 323).
int big_tile_rows(bool f32, int64_t mean, int bits) {
    return !f32 && mean >= 256 && (bits == 2 || bits == 4) ? 112 : 64;
}

// Which kernel: by the rows an expert has on average (all hold for any split of the rows).  Up to 16 (one operand's
// rows) the few-rows kernel; then the tile kernel where it has work for every CU, else the split kernel (1531 rows x
// 4099 channels, 408 tiles of 64 x 256: 120 us against 193; 512 x 2048, 64 tiles: 83 against 44).
Plan make_plan(bool f32, int64_t M, int64_t K, int64_t N, int64_t experts, int64_t rank, int64_t n_requests, int bits,
               int groupsize) {
    Plan p;
    const int64_t mean = ceil_div(M, experts);
    const int big = big_tile_rows(f32, mean, bits);
    if (mean <= 16) {
        p.kernel = kRows;
        p.tile = 16;
    } else if (mean > 64 && ceil_div(M, 64) * ceil_div(N, 256) >= 256) {
        p.kernel = kTile;
        p.tile = ceil_div(M, big) * ceil_div(N, 256) >= 256 ? big : 64;
    } else {
        p.kernel = kSplit;
        p.tile = 16 * split_row_tiles(f32, mean, bits, groupsize);
    }
    p.cap = (int)(M / p.tile + std::min<int64_t>(experts + 2, M) + 1);
    p.Mp = (int64_t)align_up((size_t)M + kMaxTileRows, 64);
    p.nchunks = (int)ceil_div(K, kChunkK);
    p.xt_elems = (size_t)(f32 ? 3 : 1) * p.nchunks * kChunkK * p.Mp;
    p.sum_floats = f32 ? 0 : (size_t)p.nchunks * kChunkSteps * p.Mp;
    p.hrank = (int)align_up((size_t)rank, 8);
    // H in parts of K: for prompts, where 64-row passes alone would leave most of the GPU without one
    p.k_parts = 1;
    if (p.kernel == kTile && M >= 64 * n_requests)
        p.k_parts = (int)std::max<int64_t>(1, std::min<int64_t>({(int64_t)kMaxKParts, 512 / ceil_div(M, 64), K / 1024}));
    return p;
}

struct Buffers {
    float* H;
    int32_t* row_adapter;
    uint16_t* XT;
    float* sums;
    int32_t* tiles;
    float* Z;
    size_t bytes;
    Buffers(const Plan& p, int64_t M, int64_t N, void* ws) {
        Carver c(ws);
        const bool staged = p.kernel != kRows;
        H = p.hrank ? c.take<float>((size_t)M * p.hrank * p.k_parts) : nullptr;
        row_adapter = p.hrank ? c.take<int32_t>((size_t)M) : nullptr;
        XT = staged ? c.take<uint16_t>(p.xt_elems) : nullptr;
        sums = staged ? c.take<float>(p.sum_floats) : nullptr;
        tiles = staged ? c.take<int32_t>(3 * (size_t)p.cap) : nullptr;
        Z = p.kernel == kTile && p.hrank ? c.take<float>((size_t)M * N) : nullptr;
        bytes = c.bytes();
    }
};

// The tile kernel takes one small product per run of rows with the same adapter, about 1 us each, or Z, M N fp32 values
// written and read again.  Runs of 32 rows and more on average (prompts) go the first way, single tokens the second.
bool short_requests(int64_t M, int64_t n_requests) { return M < 32 * n_requests; }

template <int PARTS>
hipError_t launch_stage(const MatmulKernelArgs& k, const StageArgs& a, bool long_rows, hipStream_t stream) {
    constexpr int64_t kMost = 1 << 22;               // a launch has fewer than 2^32 threads along x
    const int64_t turns = ceil_div(a.workgroups, kMost);
    if (turns > 65535) return hipErrorInvalidValue;
    const dim3 grid((unsigned)std::min(a.workgroups, kMost), (unsigned)turns);
#define GPTQ_STAGE(NR, RS) hipLaunchKernelGGL((stage_kernel<PARTS, NR, RS>), grid, dim3(kStageThreads), 0, stream, k, a)
#define GPTQ_STAGE_RS(NR)             \
    do {                              \
        if (long_rows) GPTQ_STAGE(NR, 4); \
        else GPTQ_STAGE(NR, 1);       \
    } while (0)
    if (!a.slices) GPTQ_STAGE(0, 1);
    else if (k.rank <= 16) GPTQ_STAGE_RS(1);
    else if (k.rank <= 32) GPTQ_STAGE_RS(2);
    else if (k.rank <= 64) GPTQ_STAGE_RS(4);
    else GPTQ_STAGE_RS(8);
#undef GPTQ_STAGE_RS
#undef GPTQ_STAGE
    return hipGetLastError();
}

}  // namespace

// For any width, group size and requests: the smaller tiles' list is the longer one, one request has the most parts of H.
size_t matmul_workspace_bytes(bool f32, int64_t M, int64_t K, int64_t N, int64_t experts, int64_t rank) {
    return Buffers(make_plan(f32, M, K, N, experts, rank, 1, 3, 32), M, N, nullptr).bytes;
}

hipError_t packed_matmul(const MatmulArgs& a, void* workspace, hipStream_t stream) {
    const bool lora = a.n_requests > 0 && a.n_adapters > 0;
    const Plan plan = make_plan(a.f32, a.M, a.K, a.N, a.E, lora ? a.rank : 0, lora ? a.n_requests : 1, a.bits, a.groupsize);
    const Buffers buf(plan, a.M, a.N, workspace);
    if (buf.bytes > matmul_workspace_bytes(a.f32, a.M, a.K, a.N, a.E, lora ? a.rank : 0)) return hipErrorInvalidValue;
    MatmulKernelArgs k;
    k.X = a.X; k.ldx = a.ldx; k.x_rows = a.x_rows; k.rows = a.rows; k.M = a.M;
    k.offsets = a.offsets; k.E = a.E;
    k.packed = a.packed; k.ldp = (uint32_t)a.ldp; k.p_stride = a.p_stride; k.K = (int)a.K; k.N = (int)a.N;
    k.nwords = (int)((a.K * a.bits + 31) / 32);
    k.scales = a.scales; k.s_stride = a.s_stride;
    k.lg_group = a.groupsize == 32 ? 0 : a.groupsize == 64 ? 1 : 2;
    k.s_row = a.groupsize ? (int)a.N : 0;
    k.last_group = a.groupsize ? (int)((a.K - 1) / a.groupsize) : 0;
    k.Y = a.Y; k.ldy = a.ldy;
    k.H = lora ? buf.H : nullptr;
    k.h_parts = plan.k_parts; k.hrank = plan.hrank; k.row_adapter = buf.row_adapter;
    k.Z = lora && plan.kernel == kTile && short_requests(a.M, a.n_requests) ? buf.Z : nullptr;
    k.B = a.B; k.ldb = a.ldb; k.b_stride = a.b_stride; k.rank = a.rank;
    k.XT = buf.XT; k.sums = buf.sums; k.Mp = plan.Mp; k.tiles = buf.tiles;

    if (lora || plan.kernel != kRows) {
        StageArgs s = {};
        s.XT = buf.XT; s.sums = buf.sums;
        s.tile = plan.tile; s.cap = plan.cap; s.tiles = buf.tiles;
        bool long_rows = false;
        if (plan.kernel != kRows) {
            s.row_blocks = (int)ceil_div(a.M, kStageRows);
            s.nchunks = plan.nchunks;
            s.workgroups = (int64_t)s.row_blocks * plan.nchunks + 1;
        }
        if (lora) {
            s.A = a.A; s.lda = a.lda; s.a_stride = a.a_stride; s.alpha = a.alpha; s.n_adapters = a.n_adapters;
            s.requests = a.requests; s.adapter = a.adapter; s.n_requests = a.n_requests;
            s.H = buf.H; s.row_adapter = buf.row_adapter;
            // workgroups for the requests: about 1024 in all, no more than the longest could use
            long_rows = plan.k_parts > 1;
            const int rows = long_rows ? 64 : 16;
            s.k_parts = plan.k_parts;
            s.slices = (int)std::max<int64_t>(1, std::min<int64_t>(std::max<int64_t>(ceil_div(a.M, rows), std::min<int64_t>(a.M, 4)),
                                                                     1024 / (a.n_requests * s.k_parts)));
            s.windows = (int64_t)rows * s.slices < a.M ? ceil_div(a.M, rows) : 0;
            s.workgroups += ((a.n_requests + 1) * s.slices + s.windows) * s.k_parts;
        }
        hipError_t e = a.f32 ? launch_stage<3>(k, s, long_rows, stream) : launch_stage<1>(k, s, long_rows, stream);
        if (e != hipSuccess) return e;
        if (k.Z) {
            const dim3 zgrid((unsigned)ceil_div(a.M, 64), (unsigned)ceil_div(a.N, 256));
            hipLaunchKernelGGL(adapter_expand_kernel, zgrid, dim3(256), 0, stream, k, buf.Z);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
#define GPTQ_WIDTH(B)                                                                                      \
    do {                                                                                                   \
        if (plan.kernel == kRows) return rows_b##B(k, a.f32, a.swiglu, stream);                            \
        if (plan.kernel == kSplit) return split_b##B(k, a.f32, plan.tile / 16, plan.cap, a.swiglu, stream); \
        return tile_b##B(k, a.f32, plan.tile / 16, plan.cap, a.swiglu, stream);                            \
    } while (0)
    switch (a.bits) {
        case 2: GPTQ_WIDTH(2);
        case 3: GPTQ_WIDTH(3);
        case 4: GPTQ_WIDTH(4);
        case 5: GPTQ_WIDTH(5);
        default: GPTQ_WIDTH(6);
    }
#undef GPTQ_WIDTH
}

}  // namespace gptq
