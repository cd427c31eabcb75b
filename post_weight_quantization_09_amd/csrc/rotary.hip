// Rotary positions: every pair of a head's elements turned by position * frequency.
//
// The angle is taken in turns, position * f / 2 pi, in two 64-bit numbers (both products with what their rounding leaves off,
// and 1 / 2 pi in two parts), and loses its whole turns there: what the sine and cosine see is a fraction of a turn within 2^-53
// at any 32-bit position and any f up to 2^20, rounded to fp32.  (In one number it is off by 2^-24 of a turn at position 2^31 for f
// near 1, by 2^-4 for f near 2^20.)  They are evaluated in fp32, once for a
// token's pair whatever the number of heads, and wait in LDS.  What is left is a copy: a workgroup takes some tokens' rows of
// some heads, 16 bytes a load where the pairs allow it (units of V pairs), and is bound by memory traffic.
//
// Measured on MI355X: 8192 tokens x 40 heads x 128 in bf16, 168 MB, 36 to 39 us (4.3 to 4.6 TB/s; a copy moves 4.9); with an angle per head
// and single elements 72 us.  One token 2.0 us (a launch).
#include "context.hpp"

namespace gptq {

namespace {

constexpr int kThreads = 256, kMaxPairs = 1024;     // pairs of a workgroup's tokens, in LDS

struct RotaryArgs {
    const void* x;
    void* y;
    int64_t x_ts, x_hs, y_ts, y_hs;
    const int32_t* positions;
    const double* freqs;
    float factor;
    int T, H, D, half;
    int tokens, heads;              // of a workgroup
    int turned, units;              // units of a row that are turned, and all of them
    Divisor by_units, by_heads;
};

// cos and sin of position * f, times the factor
__device__ __forceinline__ f32x2 turn(int position, double f, float factor) {
    constexpr double kPerTurn = 0.15915494309189533577, kPerTurnRest = -9.839338337591243e-18;      // 1 / 2 pi
    const double angle = position * f, angle_rest = fma((double)position, f, -angle);
    const double whole = rint(angle * kPerTurn);
    const float part = (float)(fma(angle, kPerTurn, -whole) + (angle * kPerTurnRest + angle_rest * kPerTurn));
    f32x2 cs;
    cs[0] = factor * cospif(2.0f * part);
    cs[1] = factor * sinpif(2.0f * part);
    return cs;
}

// N elements of any alignment that their type has.
template <int N>
__device__ __forceinline__ void load(const float* p, float (&x)[N]) {
    typedef float __attribute__((ext_vector_type(N))) vec;
    typedef vec __attribute__((aligned(4))) any;
    if constexpr (N == 1) {
        x[0] = *p;
    } else {
        const vec v = *reinterpret_cast<const any*>(p);
        for (int i = 0; i < N; ++i) x[i] = v[i];
    }
}
template <int N>
__device__ __forceinline__ void load(const __bf16* p, float (&x)[N]) {
    if constexpr (N == 1) {
        x[0] = (float)*p;
    } else {
        typedef uint32_t __attribute__((ext_vector_type(N / 2))) vec;
        typedef vec __attribute__((aligned(2))) any;
        const vec v = *reinterpret_cast<const any*>(p);
        for (int i = 0; i < N; ++i) x[i] = i % 2 ? bf16hi_to_f32(v[i / 2]) : bf16lo_to_f32(v[i / 2]);
    }
}
template <int N>
__device__ __forceinline__ void store(float* p, const float (&x)[N]) {
    typedef float __attribute__((ext_vector_type(N))) vec;
    typedef vec __attribute__((aligned(4))) any;
    if constexpr (N == 1) {
        *p = x[0];
    } else {
        vec v;
        for (int i = 0; i < N; ++i) v[i] = x[i];
        *reinterpret_cast<any*>(p) = v;
    }
}
template <int N>
__device__ __forceinline__ void store(__bf16* p, const float (&x)[N]) {
    if constexpr (N == 1) {
        *p = (__bf16)x[0];
    } else {
        typedef uint32_t __attribute__((ext_vector_type(N / 2))) vec;
        typedef vec __attribute__((aligned(2))) any;
        vec v;
        for (int i = 0; i < N / 2; ++i) v[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
        *reinterpret_cast<any*>(p) = v;
    }
}

// N elements as they are (N even).
template <int N, typename E>
__device__ __forceinline__ void copy(const E* p, E* q) {
    typedef uint32_t __attribute__((ext_vector_type(N * sizeof(E) / 4))) vec;
    typedef vec __attribute__((aligned(sizeof(E)))) any;
    *reinterpret_cast<any*>(q) = *reinterpret_cast<const any*>(p);
}

// A unit: V pairs to be turned, or up to 2 V elements to be copied.
template <typename E, int V, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a) {
    __shared__ f32x2 turns[kMaxPairs];
    const int t0 = blockIdx.x * a.tokens, h0 = blockIdx.y * a.heads;
    const int tokens = min(a.tokens, a.T - t0), heads = min(a.heads, a.H - h0);
    for (int i = threadIdx.x; i < tokens * a.half; i += kThreads) {
        const int t = i / a.half, j = i - t * a.half;
        turns[i] = turn(a.positions[t0 + t], a.freqs[j], a.factor);
    }
    __syncthreads();
    const int all = tokens * a.heads * a.units;
    for (int i = threadIdx.x; i < all; i += kThreads) {
        const int row = (int)a.by_units.quotient((uint32_t)i), u = i - row * a.units;
        const int t = (int)a.by_heads.quotient((uint32_t)row), h = row - t * a.heads;
        if (h >= heads) continue;
        const E* x = static_cast<const E*>(a.x) + (t0 + t) * a.x_ts + (h0 + h) * a.x_hs;
        E* y = static_cast<E*>(a.y) + (t0 + t) * a.y_ts + (h0 + h) * a.y_hs;
        if (u < a.turned) {
            const f32x2* cs = &turns[t * a.half + u * V];
            float p[V], q[V];
            if constexpr (INTERLEAVED) {
                float w[2 * V];
                load<2 * V>(x + 2 * V * u, w);
                for (int k = 0; k < V; ++k) {
                    p[k] = w[2 * k] * cs[k][0] - w[2 * k + 1] * cs[k][1];
                    q[k] = w[2 * k + 1] * cs[k][0] + w[2 * k] * cs[k][1];
                }
                for (int k = 0; k < V; ++k) w[2 * k] = p[k], w[2 * k + 1] = q[k];
                store<2 * V>(y + 2 * V * u, w);
            } else {
                load<V>(x + V * u, p);
                load<V>(x + a.half + V * u, q);
                for (int k = 0; k < V; ++k) {
                    const float r = p[k] * cs[k][0] - q[k] * cs[k][1];
                    q[k] = q[k] * cs[k][0] + p[k] * cs[k][1];
                    p[k] = r;
                }
                store<V>(y + V * u, p);
                store<V>(y + a.half + V * u, q);
            }
        } else {
            const int d = 2 * a.half + 2 * V * (u - a.turned);
            if (d + 2 * V <= a.D) {
                copy<2 * V>(x + d, y + d);
            } else {
                for (int k = d; k < a.D; ++k) y[k] = x[k];
            }
        }
    }
}

template <typename E, int V>
void launch(RotaryArgs a, bool interleaved, hipStream_t stream) {
    const bool copies = a.x != a.y;
    a.turned = a.half / V;
    a.units = a.turned + (copies ? (int)ceil_div(a.D - 2 * a.half, 2 * V) : 0);
    // Workgroups of up to 2048 units, or fewer where there would not be two for every CU: first some heads of a token (whose
    // sines each of its workgroups then finds for itself), then more tokens.  With one, two and four for every CU: 512 tokens, 40
    // heads of 128 3.7, 3.5 and 3.3 us; 2111 tokens, 11 heads of 80, 32 neighbours turned, fp32 6.7, 4.4 and 4.3.  With 1024, 2048,
    // 4096 and 8192 units: 8192 tokens, 40 heads of 128 33, 37, 35 and 33 us, fp32 62, 70, 73 and 70 (in a graph; no order in them).
    const int64_t total = (int64_t)a.T * a.H * a.units;
    const int64_t each = total / 512 < kThreads ? kThreads : total / 512 > 2048 ? 2048 : total / 512;
    a.heads = (int)(ceil_div(each, a.units) < a.H ? ceil_div(each, a.units) : a.H);
    a.tokens = 1;
    if (a.heads == a.H) {
        const int64_t by_units = each / ((int64_t)a.H * a.units), by_pairs = kMaxPairs / a.half;
        a.tokens = (int)(by_units < by_pairs ? by_units : by_pairs);
        if (a.tokens < 1) a.tokens = 1;
    }
    a.by_units = Divisor((uint32_t)a.units);
    a.by_heads = Divisor((uint32_t)a.heads);
    const dim3 grid((unsigned)ceil_div(a.T, a.tokens), (unsigned)ceil_div(a.H, a.heads));
    if (interleaved) rotary_kernel<E, V, true><<<grid, kThreads, 0, stream>>>(a);
    else rotary_kernel<E, V, false><<<grid, kThreads, 0, stream>>>(a);
}

}  // namespace

hipError_t rotary(HeadRows x, bool f32, int64_t T, int H, int D, const int32_t* positions, const double* freqs, int rot,
                  float factor, bool interleaved, HeadRows y, hipStream_t stream) {
    RotaryArgs a{};
    a.x = x.p, a.y = y.p, a.x_ts = x.ts, a.x_hs = x.hs, a.y_ts = y.ts, a.y_hs = y.hs;
    a.positions = positions, a.freqs = freqs, a.factor = factor;
    a.T = (int)T, a.H = H, a.D = D, a.half = rot / 2;
    // 16 bytes a load in halves, 16 or 32 of neighbours; pairs that are no multiple of that go by two or one.  8192 tokens, 40
    // heads, bf16, by eights 128: 37 us (168 MB); by twos 72: 17.6 (94 MB), 104: 29.6 (136 MB), 80 with 40 turned: 20.6 (105 MB); by
    // ones 96 with 18 turned: 37.9 (126 MB)
    if (f32) {
        if (a.half % 4 == 0) launch<float, 4>(a, interleaved, stream);
        else if (a.half % 2 == 0) launch<float, 2>(a, interleaved, stream);
        else launch<float, 1>(a, interleaved, stream);
    } else {
        if (a.half % 8 == 0) launch<__bf16, 8>(a, interleaved, stream);
        else if (a.half % 2 == 0) launch<__bf16, 2>(a, interleaved, stream);
        else launch<__bf16, 1>(a, interleaved, stream);
    }
    return hipGetLastError();
}

}  // namespace gptq
