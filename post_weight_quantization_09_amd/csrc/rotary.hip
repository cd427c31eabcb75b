// Rotary positions: every pair of a head's elements turned by position * frequency.
//
// The angle is taken in turns and in 64 bits: position * f / 2 pi loses its whole turns there, so that what the sine and
// cosine see is a fraction of a turn with 2^-32 or better at any 32-bit position; they are evaluated in fp32.
#include "context.hpp"

namespace gptq {

namespace {

struct RotaryArgs {
    const void* x;
    void* y;
    int64_t x_ts, x_hs, y_ts, y_hs;
    const int32_t* positions;
    const double* freqs;
    float factor;
    int T, H, D, rot;
};

template <typename E>
__device__ __forceinline__ float as_float(E v) { return (float)v; }

// cos and sin of position * f, times the factor
__device__ __forceinline__ f32x2 turn(int position, double f, float factor) {
    constexpr double kPerTurn = 0.15915494309189533577;   // 1 / 2 pi
    const double turns = (double)position * f * kPerTurn;
    const float part = (float)(turns - rint(turns));
    f32x2 cs;
    cs[0] = factor * cospif(2.0f * part);
    cs[1] = factor * sinpif(2.0f * part);
    return cs;
}

template <typename E, bool INTERLEAVED>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a) {
    const int t = blockIdx.x, half = a.rot / 2;
    const int position = a.positions[t];
    for (int i = threadIdx.x; i < a.H * (a.D - half); i += 256) {
        const int h = i / (a.D - half), j = i % (a.D - half);
        const E* x = static_cast<const E*>(a.x) + t * a.x_ts + h * a.x_hs;
        E* y = static_cast<E*>(a.y) + t * a.y_ts + h * a.y_hs;
        if (j < half) {
            const f32x2 cs = turn(position, a.freqs[j], a.factor);
            const int d0 = INTERLEAVED ? 2 * j : j, d1 = INTERLEAVED ? 2 * j + 1 : j + half;
            const float u = as_float(x[d0]), w = as_float(x[d1]);
            y[d0] = (E)(u * cs[0] - w * cs[1]);
            y[d1] = (E)(w * cs[0] + u * cs[1]);
        } else {
            y[j + half] = x[j + half];
        }
    }
}

}  // namespace

hipError_t rotary(HeadRows x, bool f32, int64_t T, int H, int D, const int32_t* positions, const double* freqs, int rot,
                  float factor, bool interleaved, HeadRows y, hipStream_t stream) {
    RotaryArgs a{x.p, y.p, x.ts, x.hs, y.ts, y.hs, positions, freqs, factor, (int)T, H, D, rot};
    auto* kernel = f32 ? (interleaved ? rotary_kernel<float, true> : rotary_kernel<float, false>)
                       : (interleaved ? rotary_kernel<__bf16, true> : rotary_kernel<__bf16, false>);
    kernel<<<dim3((unsigned)T), 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace gptq
