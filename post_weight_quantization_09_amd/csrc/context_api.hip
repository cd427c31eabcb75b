// C ABI of rotary positions, the paged cache and the attention over it (see include/gptq.h).
#include <algorithm>
#include <cmath>

#include "context.hpp"
#include "timer.hpp"

using namespace gptq;

namespace {

bool dtype_ok(gptq_dtype_t d) { return d == GPTQ_DTYPE_F32 || d == GPTQ_DTYPE_BF16; }

constexpr int64_t kMaxTokens = (int64_t)1 << 22, kMaxHeads = 1024, kMaxRotaryHead = 1024;
constexpr int64_t kMaxRequests = 65536, kMaxPageSize = 65536, kMaxStride = (int64_t)1 << 40;

bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride; }

// Rows that are written: none of their D elements is shared with another row.
bool apart(int64_t T, int64_t H, int64_t D, int64_t ts, int64_t hs) {
    if (!stride_ok(ts) || !stride_ok(hs)) return false;
    if (T <= 1 && H <= 1) return true;
    if (T <= 1) return hs >= D;
    if (H <= 1) return ts >= D;
    return (hs >= D && ts >= (H - 1) * hs + D) || (ts >= D && hs >= (T - 1) * ts + D);
}

bool bits_ok(int bits) { return bits == 4 || bits == 8 || bits == 16; }

bool head_ok(int64_t D) { return D >= 8 && D <= kMaxHeadSize && D % 8 == 0; }

// The pages themselves: sizes, alignment, heads that do not overlap, slots that are int32.
bool pages_ok(const void* pages, int64_t n, int64_t page_stride, int64_t head_stride, int64_t page_size, int64_t H,
              int64_t D, int bits) {
    if (!bits_ok(bits) || !head_ok(D) || H < 1 || H > kMaxHeads) return false;
    if (page_size < 16 || page_size > kMaxPageSize || page_size % 16 != 0) return false;
    if (!pages || reinterpret_cast<uintptr_t>(pages) % 16 != 0 || n < 1 || n > (((int64_t)1 << 31) - 1) / page_size) return false;
    if (page_stride % 16 != 0 || head_stride % 16 != 0) return false;
    return apart(n, H, cache_block_bytes(page_size, D, bits), page_stride, head_stride);
}

}  // namespace

extern "C" {

gptq_status_t gptq_rotary_frequencies(int64_t rot, double base, int scaling, double factor, double original, double low,
                                      double high, double* freqs, float* magnitude) {
    if (!freqs || rot < 2 || rot > kMaxRotaryHead || rot % 2 != 0 || !(base > 1.0) || !std::isfinite(base)) return GPTQ_ERR_ARG;
    if (scaling < GPTQ_ROTARY_PLAIN || scaling > GPTQ_ROTARY_BANDS) return GPTQ_ERR_ARG;
    if (scaling != GPTQ_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return GPTQ_ERR_ARG;
    const bool banded = scaling == GPTQ_ROTARY_RAMP || scaling == GPTQ_ROTARY_BANDS;
    if (banded && (!(original >= 1.0) || !std::isfinite(original) || !(low > 0.0) || !(high > low) || !std::isfinite(high)))
        return GPTQ_ERR_ARG;
    if (scaling == GPTQ_ROTARY_BASE) base *= std::pow(factor, (double)rot / (double)std::max<int64_t>(rot - 2, 1));
    if (!std::isfinite(base)) return GPTQ_ERR_ARG;
    const double two_pi = 2.0 * M_PI;
    double first = 0.0, last = 0.0;
    if (scaling == GPTQ_ROTARY_RAMP) {
        // the pair that makes n turns over `original` positions
        const auto pair = [&](double n) { return (double)rot * std::log(original / (n * two_pi)) / (2.0 * std::log(base)); };
        first = std::max(std::floor(pair(high)), 0.0);
        last = std::min(std::ceil(pair(low)), (double)rot - 1.0);
    }
    for (int64_t i = 0; i < rot / 2; ++i) {
        const double f = std::pow(base, -2.0 * (double)i / (double)rot);
        double keep = 1.0;                     // share of f that is not stretched
        if (scaling == GPTQ_ROTARY_LINEAR) keep = 0.0;
        if (scaling == GPTQ_ROTARY_RAMP)
            keep = last <= 0.0 ? 0.0             // no pair makes more than `low` turns
                               : 1.0 - std::min(std::max(((double)i - first) / std::max(last - first, 0.001), 0.0), 1.0);
        if (scaling == GPTQ_ROTARY_BANDS)
            keep = std::min(std::max((original * f / two_pi - low) / (high - low), 0.0), 1.0);
        freqs[i] = keep == 1.0 ? f : f * keep + f / factor * (1.0 - keep);
    }
    if (magnitude) *magnitude = scaling == GPTQ_ROTARY_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return GPTQ_OK;
}

gptq_status_t gptq_rotary(const void* X, gptq_dtype_t dtype, int64_t T, int64_t H, int64_t D, int64_t x_ts, int64_t x_hs,
                          const int32_t* positions, const double* freqs, int64_t rot, float factor, unsigned flags,
                          void* Y, int64_t y_ts, int64_t y_hs, void* stream) {
    if (!dtype_ok(dtype) || T < 0 || T > kMaxTokens || H < 1 || H > kMaxHeads || D < 1 || D > kMaxRotaryHead)
        return GPTQ_ERR_ARG;
    if (rot < 2 || rot > D || rot % 2 != 0 || (flags & ~GPTQ_FLAG_INTERLEAVED)) return GPTQ_ERR_ARG;
    if (!stride_ok(x_ts) || !stride_ok(x_hs) || !apart(T, H, D, y_ts, y_hs)) return GPTQ_ERR_ARG;
    if (T == 0) return GPTQ_OK;
    if (!X || !Y || !positions || !freqs || (X == Y && ((T > 1 && x_ts != y_ts) || (H > 1 && x_hs != y_hs))))
        return GPTQ_ERR_ARG;
    TimerScope ts(static_cast<hipStream_t>(stream), GPTQ_TIMER_OTHER);
    return rotary({const_cast<void*>(X), x_ts, x_hs}, dtype == GPTQ_DTYPE_F32, T, (int)H, (int)D, positions, freqs,
                  (int)rot, factor, (flags & GPTQ_FLAG_INTERLEAVED) != 0, {Y, y_ts, y_hs},
                  static_cast<hipStream_t>(stream)) == hipSuccess
               ? GPTQ_OK
               : GPTQ_ERR_HIP;
}

size_t gptq_cache_block_bytes(int64_t page_size, int64_t D, int bits) {
    if (!bits_ok(bits) || !head_ok(D) || page_size < 16 || page_size > kMaxPageSize || page_size % 16 != 0) return 0;
    return (size_t)cache_block_bytes(page_size, D, bits);
}

gptq_status_t gptq_cache_write(const void* K, const void* V, gptq_dtype_t dtype, int64_t T, int64_t H, int64_t D,
                               int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs, const int32_t* slots, int bits,
                               void* pages, int64_t n_pages, int64_t page_stride, int64_t head_stride,
                               int64_t page_size, void* stream) {
    if (!dtype_ok(dtype) || T < 0 || T > kMaxTokens || !pages_ok(pages, n_pages, page_stride, head_stride, page_size, H, D, bits))
        return GPTQ_ERR_ARG;
    if (!stride_ok(k_ts) || !stride_ok(k_hs) || !stride_ok(v_ts) || !stride_ok(v_hs)) return GPTQ_ERR_ARG;
    if (T == 0) return GPTQ_OK;
    if (!K || !V || !slots) return GPTQ_ERR_ARG;
    TimerScope ts(static_cast<hipStream_t>(stream), GPTQ_TIMER_OTHER);
    const Pages p{static_cast<uint8_t*>(pages), n_pages, page_stride, head_stride, (int)page_size, bits};
    return cache_write({const_cast<void*>(K), k_ts, k_hs}, {const_cast<void*>(V), v_ts, v_hs}, dtype == GPTQ_DTYPE_F32, T,
                       (int)H, (int)D, slots, p, static_cast<hipStream_t>(stream)) == hipSuccess
               ? GPTQ_OK
               : GPTQ_ERR_HIP;
}

gptq_status_t gptq_cache_read(const void* pages, int64_t n_pages, int64_t page_stride, int64_t head_stride,
                              int64_t page_size, int bits, const int32_t* slots, int64_t T, int64_t H, int64_t D, void* K,
                              void* V, gptq_dtype_t dtype, int64_t k_ts, int64_t k_hs, int64_t v_ts, int64_t v_hs,
                              void* stream) {
    if (!dtype_ok(dtype) || T < 0 || T > kMaxTokens || !pages_ok(pages, n_pages, page_stride, head_stride, page_size, H, D, bits))
        return GPTQ_ERR_ARG;
    if (!apart(T, H, D, k_ts, k_hs) || !apart(T, H, D, v_ts, v_hs)) return GPTQ_ERR_ARG;
    if (T == 0) return GPTQ_OK;
    if (!K || !V || K == V || !slots) return GPTQ_ERR_ARG;
    TimerScope ts(static_cast<hipStream_t>(stream), GPTQ_TIMER_OTHER);
    const Pages p{static_cast<uint8_t*>(const_cast<void*>(pages)), n_pages, page_stride, head_stride, (int)page_size, bits};
    return cache_read(p, slots, T, (int)H, (int)D, {K, k_ts, k_hs}, {V, v_ts, v_hs}, dtype == GPTQ_DTYPE_F32,
                      static_cast<hipStream_t>(stream)) == hipSuccess
               ? GPTQ_OK
               : GPTQ_ERR_HIP;
}

size_t gptq_attention_workspace_bytes(int64_t R, int64_t Hq, int64_t H, int64_t D) {
    if (R < 1 || R > kMaxRequests || H < 1 || H > kMaxHeads || Hq < H || Hq > kMaxHeads || Hq % H != 0 || !head_ok(D)) return 0;
    return attention_workspace_bytes(R, Hq, H, D);
}

gptq_status_t gptq_cache_attention(const void* Q, gptq_dtype_t dtype, int64_t R, int64_t Hq, int64_t H, int64_t D,
                                   int64_t q_rs, int64_t q_hs, const void* pages, int64_t n_pages, int64_t page_stride,
                                   int64_t head_stride, int64_t page_size, int bits, const int32_t* table,
                                   int64_t ld_table, int64_t max_pages, const int32_t* lengths, float scale,
                                   int64_t window, void* out, int64_t o_rs, int64_t o_hs, float* lse, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dtype) || R < 0 || R > kMaxRequests || Hq < H || Hq > kMaxHeads || H < 1 || Hq % H != 0) return GPTQ_ERR_ARG;
    if (!pages_ok(pages, n_pages, page_stride, head_stride, page_size, H, D, bits)) return GPTQ_ERR_ARG;
    if (!stride_ok(q_rs) || !stride_ok(q_hs) || !apart(R, Hq, D, o_rs, o_hs)) return GPTQ_ERR_ARG;
    if (max_pages < 0 || max_pages > (((int64_t)1 << 31) - 1) / page_size || ld_table < 0 || ld_table > kMaxStride) return GPTQ_ERR_ARG;
    if (!attention_line_ok(R, Hq, H, max_pages * page_size)) return GPTQ_ERR_ARG;
    if (!std::isfinite(scale) || window < 0) return GPTQ_ERR_ARG;
    if (R == 0) return GPTQ_OK;
    if (!Q || !out || Q == out || !lengths || (max_pages > 0 && !table)) return GPTQ_ERR_ARG;
    const size_t need = attention_workspace_bytes(R, Hq, H, D);
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % kAlign != 0 || workspace_bytes < need) return GPTQ_ERR_WORKSPACE;
    AttentionArgs a{{const_cast<void*>(Q), q_rs, q_hs}, {out, o_rs, o_hs}, dtype == GPTQ_DTYPE_F32, (int)R, (int)Hq, (int)H, (int)D,
                    {static_cast<uint8_t*>(const_cast<void*>(pages)), n_pages, page_stride, head_stride, (int)page_size, bits},
                    table, ld_table, max_pages, lengths, scale, window, lse};
    TimerScope ts(static_cast<hipStream_t>(stream), GPTQ_TIMER_OTHER);
    return cache_attention(a, workspace, static_cast<hipStream_t>(stream)) == hipSuccess ? GPTQ_OK : GPTQ_ERR_HIP;
}

}  // extern "C"
