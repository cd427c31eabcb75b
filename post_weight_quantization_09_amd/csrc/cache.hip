// The paged cache of keys and values: rows quantised as they are written, and read back.
//
// A row of a token and head is kept on the symmetric grid of gptq_quantize_layer: s = absmax / (2^(b-1) - 1/2), codes
// round-half-even(x / s).  The rounding is exact, not that of a rounded quotient: x times the reciprocal is off by less than
// 2^-15, so q = rint(x * (1 / s)) is right or, next to a border, the other neighbour's.  The remainder x - q s is representable
// (q has at most 8 bits, |x - q s| is not above s / 2 by more than a few of x's last places): one fused multiply-add gives it,
// and comparing it with s / 2 moves q where the other is nearer, or even.  Borders are no rare case to branch on: a row's largest
// value lies on one, and bf16 values do often.
//
// Memory traffic is the bound.  A wave takes eight tokens of a head (two heads of 64): a lane holds two or four
// dimensions of each, so that rows are read and written in whole lines, their largest values found by maxima across the
// lanes (of eight rows together, so that every step halves the registers), and eight tokens of a lane's dimensions are what the values' layout stores side by side.  Where eight
// tokens fill eight slots from a multiple of eight on, in order, they are stored with 8 or 16 bytes a lane; the wave that
// holds the first of them takes all eight, so that runs of any beginning in the batch are written so.  Other tokens' values
// go byte by byte into the octets that they share with tokens of other calls.
//
// Measured on MI355X, 16384 tokens, 8 heads of 128, bf16 rows, 84 MB each way: 4 bits written in 27 us (3.1 TB/s; vector
// instructions take 63% of the cycles, 24 a value: 13 round it exactly, the others take it from its word, mask it and pack its
// code), read in 18 us (4.7 TB/s).  One row a workgroup, its values stored byte by byte: 116 and 61 us.  8 bits, 101 MB: 24.5 and
// 18.1; 16 bits, 134 MB: 24.3 and 21.8; 65536 tokens in 4, 8 and 16 bits 85 and 84, 95 and 90, 110 and 108 (4 to 4.9 TB/s).
// 64 tokens of a decode step: 5.3 and 4.7 us, latency.
#include "context.hpp"

namespace gptq {

namespace {

constexpr int kOctet = 8;

struct CacheArgs {
    const void* k;
    const void* v;
    int64_t k_ts, k_hs, v_ts, v_hs;
    const int32_t* slots;
    uint8_t* pages;
    int64_t page_stride, head_stride;
    uint32_t n_slots;
    int T, H, D, Dp, page_size;
    Divisor by_page;
};

constexpr float kRound = 12582912.0f;           // 1.5 2^23: added to a small value, the sum's last bits are that value rounded

// x / s rounded to nearest, ties to even, in the last bits of the result (kRound's added).
__device__ __forceinline__ int exact_round(float x, float s, float inv) {
    const float t = fmaf(x, inv, kRound), q = t - kRound, rem = fmaf(-q, s, x);
    // twice the remainder against s as whole numbers, an odd q's with one more: a tie is not above s where q is even
    const uint32_t twice = __float_as_uint(fabsf(rem) + fabsf(rem)) + (__float_as_uint(t) & 1u);
    const int toward = (__float_as_int(rem) >> 31) | 1;
    return __float_as_int(t) + (twice > __float_as_uint(s) ? toward : 0);
}

template <int BITS>
__device__ __forceinline__ float grid_scale(uint32_t absmax) {
    constexpr float kTop = (float)(1 << (BITS - 1)) - 0.5f;
    return absmax >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : fmaxf(__uint_as_float(absmax) / kTop, 0x1p-126f);
}

template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t x) {
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true));
}

__device__ __forceinline__ uint32_t max_of_sixteen(uint32_t x) {
    x = max_dpp<0xB1>(x);                       // quad_perm 1, 0, 3, 2
    x = max_dpp<0x4E>(x);                       // quad_perm 2, 3, 0, 1
    x = max_dpp<0x141>(x);                      // row_half_mirror
    return max_dpp<0x140>(x);                   // row_mirror
}

__device__ __forceinline__ uint32_t max_swap32(uint32_t x, uint32_t y) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    return max(r[0], r[1]);
}
__device__ __forceinline__ uint32_t max_swap16(uint32_t x, uint32_t y) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    return max(r[0], r[1]);
}

// The largest of eight rows' values over all lanes, or (TWO) over each half's 32: a lane's result is that of row row_of(lane),
// and row i's is in lane lane_of(i) (of each half).  A swap puts two rows where one was: each step has half the registers.
template <bool TWO>
__device__ __forceinline__ uint32_t max_of_rows(const uint32_t (&m)[kOctet], int lane) {
    if constexpr (TWO) {
        uint32_t c[4];
        for (int i = 0; i < 4; ++i) c[i] = max_of_sixteen(max_swap16(m[i], m[i + 4]));      // 16 lanes: i, the next 16: i + 4
        const uint32_t low = lane & 1 ? c[1] : c[0], high = lane & 1 ? c[3] : c[2];
        return lane & 2 ? high : low;
    } else {
        uint32_t a[4], b[2];
        for (int i = 0; i < 4; ++i) a[i] = max_swap32(m[i], m[i + 4]);                      // lower half: i, upper: i + 4
        for (int i = 0; i < 2; ++i) b[i] = max_of_sixteen(max_swap16(a[i], a[i + 2]));      // 16 lanes each: i, i + 2, i + 4, i + 6
        return lane & 1 ? b[1] : b[0];
    }
}
template <bool TWO>
__device__ __forceinline__ int lane_of(int i) { return TWO ? (i >> 2) * 16 + (i & 3) : (i >> 1) * 16 + (i & 1); }
template <bool TWO>
__device__ __forceinline__ int row_of(int lane) { return TWO ? (lane & 3) + 4 * (lane >> 4 & 1) : (lane & 1) + 2 * (lane >> 4); }

// N elements of any alignment that their type has, as they are stored; N stored from fp32.
template <typename E, int N>
struct Raw;
template <int N>
struct Raw<float, N> {
    typedef float __attribute__((ext_vector_type(N))) vec;
    typedef vec __attribute__((aligned(4))) any;
    vec v;
    __device__ void load(const float* p) { v = *reinterpret_cast<const any*>(p); }
    __device__ float get(int i) const { return v[i]; }
};
template <int N>
struct Raw<__bf16, N> {
    typedef uint32_t __attribute__((ext_vector_type(N / 2))) vec;
    typedef vec __attribute__((aligned(2))) any;
    vec v;
    __device__ void load(const __bf16* p) { v = *reinterpret_cast<const any*>(p); }
    __device__ float get(int i) const { return i % 2 ? bf16hi_to_f32(v[i / 2]) : bf16lo_to_f32(v[i / 2]); }
};

template <int N>
__device__ __forceinline__ void store_row(float* p, const float (&x)[N]) {
    typedef float __attribute__((ext_vector_type(N))) vec;
    typedef vec __attribute__((aligned(4))) any;
    vec v;
    for (int i = 0; i < N; ++i) v[i] = x[i];
    *reinterpret_cast<any*>(p) = v;
}
template <int N>
__device__ __forceinline__ void store_row(__bf16* p, const float (&x)[N]) {
    typedef uint32_t __attribute__((ext_vector_type(N / 2))) vec;
    typedef vec __attribute__((aligned(2))) any;
    vec v;
    for (int i = 0; i < N / 2; ++i) v[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<any*>(p) = v;
}

// Which of a wave's tokens are taken together.  Lane i looks at token t0 - 7 + i; bit j of the results is token t0 + j.
struct Tokens {
    int32_t slot[kOctet];                       // of the wave's own tokens; -1 outside the pages
    int octet;                                  // the first of eight tokens that fill eight slots, or -1
    int32_t octet_slot;
    uint32_t single;                            // tokens in no such eight
    int32_t row_slot;                           // slot of token row_of(lane)
};

template <bool TWO>
__device__ __forceinline__ Tokens tokens_of(const CacheArgs& a, int t0, int lane) {
    Tokens w;
    const int t = t0 - (kOctet - 1) + lane;
    const bool here = lane < 3 * kOctet - 2 && t >= 0 && t < a.T;
    int32_t slot = here ? a.slots[t] : -1;
    if ((uint32_t)slot >= a.n_slots) slot = -1;
    const int32_t next = __shfl_down(slot, 1);
    uint64_t full = __ballot(slot >= 0 && next == slot + 1);
    full &= full >> 1;
    full &= full >> 2;                          // four steps in order
    full = full & (full >> 3) & __ballot(slot >= 0 && slot % kOctet == 0);
    uint64_t covered = full | full << 1;
    covered |= covered << 2;
    covered |= covered << 4;
    const uint32_t own = (uint32_t)(full >> (kOctet - 1)) & 0xFFu;
    w.octet = own ? __ffs((int)own) - 1 : -1;
    w.octet_slot = __builtin_amdgcn_readlane(slot, own ? w.octet + kOctet - 1 : 0);
    for (int j = 0; j < kOctet; ++j) w.slot[j] = __builtin_amdgcn_readlane(slot, j + kOctet - 1);
    w.row_slot = __shfl(slot, row_of<TWO>(lane) + kOctet - 1);
    w.single = (uint32_t)(~covered >> (kOctet - 1)) & 0xFFu & ((1u << min(a.T - t0, kOctet)) - 1u);
    return w;
}

// A wave's rows: its lanes' head and dimensions.  TWO: each half has a head (of 64 dimensions).
template <int PD, bool TWO>
struct Lanes {
    int head, d, from;                          // from: where a lane reads; one that has no part of a row, its beginning
    bool on, inside;                            // has part of a block's row, of the elements
    __device__ Lanes(const CacheArgs& a, int lane) {
        head = TWO ? 2 * blockIdx.y + (lane >> 5) : blockIdx.y;
        d = (TWO ? lane & 31 : lane) * PD;
        on = d < a.Dp && head < a.H;
        inside = on && d < a.D;
        from = d < a.D ? d : 0;
    }
};

// The block and the place in it of a slot.
struct Place {
    uint32_t page, at;
    __device__ Place(const CacheArgs& a, int32_t slot) : page(a.by_page.quotient((uint32_t)slot)), at((uint32_t)slot - page * a.page_size) {}
};

// Rows first + i of a head for the bits i of `which` (one at least), whichever for the others.  No branch is taken on a row, so
// that all are under way before the first is waited for.
template <typename E, int PD>
struct Rows {
    Raw<E, PD> x[kOctet];
    __device__ void load(const E* from, int64_t ts, int first, uint32_t which) {
        const int some = __ffs((int)which) - 1;
        for (int i = 0; i < kOctet; ++i) x[i].load(from + (first + (which >> i & 1 ? i : some)) * ts);
    }
};

template <int BITS, int PD, bool TWO>
struct Codes {
    uint32_t code[kOctet][PD];
    float mine;                                 // scale of row row_of(lane)
    template <typename E>
    __device__ void of(const Rows<E, PD>& r, bool inside, int lane) {                       // not inside: zeros
        float x[kOctet][PD];
        for (int i = 0; i < kOctet; ++i)
            for (int j = 0; j < PD; ++j) x[i][j] = r.x[i].get(j);
        constexpr uint32_t kMask = (1u << BITS) - 1u;
        const uint32_t part = inside ? kMask : 0u;
        if constexpr (BITS == 16) {
            for (int i = 0; i < kOctet; ++i)
                for (int j = 0; j < PD; ++j) code[i][j] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[i][j]) & part;
        } else {
            uint32_t m[kOctet];
            for (int i = 0; i < kOctet; ++i) {
                m[i] = 0;
                for (int j = 0; j < PD; ++j) m[i] = max(m[i], __float_as_uint(x[i][j]) & 0x7FFFFFFFu);
            }
            mine = grid_scale<BITS>(max_of_rows<TWO>(m, lane));                             // a lane finds the scale of one row
            const int top = __float_as_int(kRound) + (int)(kMask >> 1);
            for (int i = 0; i < kOctet; ++i) {
                const int from = lane_of<TWO>(i);
                float scale = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), from));
                if (TWO) scale = lane < 32 ? scale : __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), from + 32));
                const float inv = __builtin_amdgcn_rcpf(scale);
                const uint32_t mask = scale == scale ? part : 0u;                           // rows that are not finite: zeros
                for (int j = 0; j < PD; ++j) code[i][j] = (uint32_t)min(exact_round(x[i][j], scale, inv), top) & mask;
            }
        }
    }
};

template <typename E, int BITS, int PD, bool TWO>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheArgs a) {
    const int lane = threadIdx.x & 63, t0 = (blockIdx.x * (blockDim.x >> 6) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kOctet;
    if (t0 >= a.T) return;
    const Lanes<PD, TWO> l(a, lane);
    const Tokens w = tokens_of<TWO>(a, t0, lane);
    uint32_t valid = 0;
    for (int i = 0; i < kOctet; ++i) valid |= (uint32_t)(w.slot[i] >= 0) << i;
    const uint32_t single = w.single & valid;
    if (!valid && w.octet < 0) return;
    const uint32_t part = (uint32_t)a.page_size * a.Dp * BITS / 8;
    uint8_t* head = a.pages + l.head * a.head_stride;
    const bool together = w.octet >= 0;
    const int source = min(l.head, a.H - 1);
    const E* k = static_cast<const E*>(a.k) + t0 * a.k_ts + source * a.k_hs + l.from;
    const E* v = static_cast<const E*>(a.v) + t0 * a.v_ts + source * a.v_hs + l.from;
    // the scales' lanes: eight in a head, with a row each
    const bool scaler = BITS < 16 && (lane & 15) < (TWO ? 4 : 2) && l.head < a.H;
    const int row = row_of<TWO>(lane);
    const auto write_scale = [&](float s, int32_t slot, bool values) {
        const Place p(a, slot);
        reinterpret_cast<float*>(head + (int64_t)p.page * a.page_stride + 2 * part)[(values ? a.page_size : 0) + p.at] = s;
    };

    Rows<E, PD> x, z;
    if (valid) x.load(k, a.k_ts, 0, valid);
    if (together || single) z.load(v, a.v_ts, together ? w.octet : 0, together ? 0xFFu : single);
    Codes<BITS, PD, TWO> c;

    // keys: a row per token
    c.of(x, l.inside, lane);
    if (scaler && (valid >> row & 1)) write_scale(c.mine, w.row_slot, false);
    for (int i = 0; i < kOctet; ++i) {
        if (!(valid >> i & 1) || !l.on) continue;
        const Place p(a, w.slot[i]);
        uint8_t* block = head + (int64_t)p.page * a.page_stride;
        uint8_t* to = block + (p.at * a.Dp + l.d) * BITS / 8;
        if constexpr (BITS == 16) {
            for (int j = 0; j < PD / 2; ++j) reinterpret_cast<uint32_t*>(to)[j] = c.code[i][2 * j] | c.code[i][2 * j + 1] << 16;
        } else {
            uint32_t y = 0;
            for (int j = 0; j < PD; ++j) y |= c.code[i][j] << BITS * j;
            if constexpr (BITS * PD == 8) *to = (uint8_t)y;
            else if constexpr (BITS * PD == 16) *reinterpret_cast<uint16_t*>(to) = (uint16_t)y;
            else *reinterpret_cast<uint32_t*>(to) = y;
        }
    }

    c.of(z, l.inside, lane);
    if (together) {
        if (scaler) write_scale(c.mine, w.octet_slot + row, true);
        const Place p(a, w.octet_slot);
        uint8_t* block = head + (int64_t)p.page * a.page_stride;
        if (l.on) {
            uint32_t y[BITS * PD / 4];              // a dimension's eight entries are BITS / 4 words
            if constexpr (BITS == 16) {
                for (int j = 0; j < PD; ++j)
                    for (int i = 0; i < 4; ++i) y[4 * j + i] = c.code[2 * i][j] | c.code[2 * i + 1][j] << 16;
            } else if constexpr (BITS == 8) {
                for (int j = 0; j < PD; ++j)
                    for (int i = 0; i < 2; ++i)
                        y[2 * j + i] = c.code[4 * i][j] | c.code[4 * i + 1][j] << 8 | c.code[4 * i + 2][j] << 16 | c.code[4 * i + 3][j] << 24;
            } else {
                for (int j = 0; j < PD / 2; ++j)
                    for (int i = 0; i < 2; ++i) {
                        y[2 * j + i] = 0;
                        for (int q = 0; q < 4; ++q) y[2 * j + i] |= (c.code[4 * i + q][2 * j] | c.code[4 * i + q][2 * j + 1] << 4) << 8 * q;
                    }
            }
            uint8_t* to = block + part + (p.at / kOctet * a.Dp + l.d) * BITS;
            if constexpr (BITS * PD / 4 == 2) {
                *reinterpret_cast<u32x2*>(to) = u32x2{y[0], y[1]};
            } else {
                for (int i = 0; i < BITS * PD / 16; ++i)
                    reinterpret_cast<u32x4*>(to)[i] = u32x4{y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]};
            }
        }
        if (!single) return;
        z.load(v, a.v_ts, 0, single);               // beside an octet, at the end of a run
        c.of(z, l.inside, lane);
    }
    if (scaler && (single >> row & 1)) write_scale(c.mine, w.row_slot, true);
    for (int i = 0; i < kOctet; ++i) {
        if (!(single >> i & 1) || !l.on) continue;
        const Place p(a, w.slot[i]);
        uint8_t* block = head + (int64_t)p.page * a.page_stride;
        uint8_t* to = block + part + (p.at / kOctet * a.Dp + l.d) * BITS + p.at % kOctet * (BITS == 16 ? 2 : 1);
        if constexpr (BITS == 16) {
            for (int j = 0; j < PD; ++j) *reinterpret_cast<uint16_t*>(to + 16 * j) = (uint16_t)c.code[i][j];
        } else if constexpr (BITS == 8) {
            for (int j = 0; j < PD; ++j) to[8 * j] = (uint8_t)c.code[i][j];
        } else {
            for (int j = 0; j < PD / 2; ++j) to[8 * j] = (uint8_t)(c.code[i][2 * j] | c.code[i][2 * j + 1] << 4);
        }
    }
}

// A code of BITS bits (in two's complement) from its place in a word.
template <int BITS>
__device__ __forceinline__ float code_at(uint32_t w, int place) {
    return (float)((int)(w << (32 - BITS - BITS * place)) >> (32 - BITS));
}

// Keys of eight tokens, or values of eight tokens one by one: a lane's dimensions of each as they are stored, a word for each
// piece that lies by itself.
template <int BITS, int PD>
struct Kept {
    uint32_t y[kOctet][PD];
    float scale[kOctet];
    // without a branch on a token: one outside the pages reads slot 0, and store() leaves it out
    __device__ void load(const CacheArgs& a, const Tokens& w, const uint8_t* head, uint32_t part, int d, bool values) {
        for (int i = 0; i < kOctet; ++i) {
            const Place p(a, max(w.slot[i], 0));
            const uint8_t* block = head + (int64_t)p.page * a.page_stride;
            if constexpr (BITS < 16) scale[i] = reinterpret_cast<const float*>(block + 2 * part)[(values ? a.page_size : 0) + p.at];
            if (values) {
                const uint8_t* from = block + part + (p.at / kOctet * a.Dp + d) * BITS + p.at % kOctet * (BITS == 16 ? 2 : 1);
                if constexpr (BITS == 16) {
                    for (int j = 0; j < PD; ++j) y[i][j] = *reinterpret_cast<const uint16_t*>(from + 16 * j);
                } else {
                    for (int j = 0; j < PD * BITS / 8; ++j) y[i][j] = from[8 * j];
                }
            } else {
                const uint8_t* from = block + (p.at * a.Dp + d) * BITS / 8;
                if constexpr (BITS == 16) {
                    for (int j = 0; j < PD / 2; ++j) y[i][j] = reinterpret_cast<const uint32_t*>(from)[j];
                } else if constexpr (BITS * PD == 8) {
                    y[i][0] = *from;
                } else if constexpr (BITS * PD == 16) {
                    y[i][0] = *reinterpret_cast<const uint16_t*>(from);
                } else {
                    y[i][0] = *reinterpret_cast<const uint32_t*>(from);
                }
            }
        }
    }
    template <typename E>
    __device__ void store(const Tokens& w, E* rows, int64_t ts, bool values, uint32_t which) const {
        constexpr int kEach = BITS == 4 ? 2 : 1;    // dimensions of a byte, where values lie byte by byte
        for (int i = 0; i < kOctet; ++i) {
            if (!(which >> i & 1)) continue;
            float x[PD];
            for (int j = 0; j < PD; ++j) {
                if constexpr (BITS == 16) x[j] = values ? bf16lo_to_f32(y[i][j]) : j % 2 ? bf16hi_to_f32(y[i][j / 2]) : bf16lo_to_f32(y[i][j / 2]);
                else x[j] = scale[i] * (values ? code_at<BITS>(y[i][j / kEach], j % kEach) : code_at<BITS>(y[i][0], j));
                if (w.slot[i] < 0) x[j] = 0.0f;
            }
            store_row<PD>(rows + i * ts, x);
        }
    }
};

template <typename E, int BITS, int PD, bool TWO>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheArgs a) {
    const int lane = threadIdx.x & 63, t0 = (blockIdx.x * (blockDim.x >> 6) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kOctet;
    if (t0 >= a.T) return;
    const Lanes<PD, TWO> l(a, lane);
    const Tokens w = tokens_of<TWO>(a, t0, lane);
    if (!l.inside) return;
    const uint32_t part = (uint32_t)a.page_size * a.Dp * BITS / 8, own = (1u << min(a.T - t0, kOctet)) - 1u;
    const uint8_t* head = a.pages + l.head * a.head_stride;
    E* k = (E*)a.k + t0 * a.k_ts + l.head * a.k_hs + l.d;
    E* v = (E*)a.v + t0 * a.v_ts + l.head * a.v_hs + l.d;

    Kept<BITS, PD> keys, values;
    keys.load(a, w, head, part, l.d, false);
    uint32_t y[BITS * PD / 4];                      // eight tokens' values of a lane's dimensions
    f32x4 scale[2];
    const bool together = w.octet >= 0;
    if (together) {
        const Place p(a, w.octet_slot);
        const uint8_t* block = head + (int64_t)p.page * a.page_stride;
        const uint8_t* from = block + part + (p.at / kOctet * a.Dp + l.d) * BITS;
        if constexpr (BITS * PD / 4 == 2) {
            const u32x2 q = *reinterpret_cast<const u32x2*>(from);
            y[0] = q[0], y[1] = q[1];
        } else {
            for (int i = 0; i < BITS * PD / 16; ++i) {
                const u32x4 q = reinterpret_cast<const u32x4*>(from)[i];
                for (int j = 0; j < 4; ++j) y[4 * i + j] = q[j];
            }
        }
        if constexpr (BITS < 16) {
            const f32x4* s = reinterpret_cast<const f32x4*>(block + 2 * part + 4 * (a.page_size + p.at));
            scale[0] = s[0], scale[1] = s[1];
        }
    }
    if (w.single) values.load(a, w, head, part, l.d, true);

    keys.store(w, k, a.k_ts, false, own);
    if (together) {
        for (int i = 0; i < kOctet; ++i) {
            float x[PD];
            for (int j = 0; j < PD; ++j) {
                if constexpr (BITS == 16) x[j] = i % 2 ? bf16hi_to_f32(y[4 * j + i / 2]) : bf16lo_to_f32(y[4 * j + i / 2]);
                else if constexpr (BITS == 8) x[j] = scale[i / 4][i % 4] * code_at<8>(y[2 * j + i / 4], i % 4);
                else x[j] = scale[i / 4][i % 4] * code_at<4>(y[2 * (j / 2) + i / 4], 2 * (i % 4) + j % 2);
            }
            store_row<PD>(v + (w.octet + i) * a.v_ts, x);
        }
    }
    if (w.single) values.store(w, v, a.v_ts, true, w.single);
}

CacheArgs cache_args(HeadRows k, HeadRows v, int64_t T, int H, int D, const int32_t* slots, const Pages& p) {
    return {k.p, v.p, k.ts, k.hs, v.ts, v.hs, slots, p.p, p.page_stride, p.head_stride, (uint32_t)(p.n * p.page_size),
            (int)T, H, D, stored_head_size(D), p.page_size, Divisor((uint32_t)p.page_size)};
}

// A wave per eight tokens; four waves a workgroup where that leaves one for every CU, else one.  With one and with four, 8 heads of
// 128 in 8 bits: 64 tokens written 4.8 and 5.4 us, read 4.1 and 4.9; 1024 tokens 6.0 and 5.8, 5.0 and 4.6; 4096 tokens 11.9 and
// 10.2, 8.8 and 7.5.
struct CacheGrid {
    dim3 grid;
    unsigned threads;
    explicit CacheGrid(const CacheArgs& a) {
        const int64_t octets = ceil_div(a.T, kOctet), heads = ceil_div(a.H, a.Dp == 64 ? 2 : 1);
        const int waves = octets * heads >= 1024 ? 4 : 1;
        threads = 64u * waves;
        grid = dim3((unsigned)ceil_div(octets, waves), (unsigned)heads);
    }
};

// launch(element, dimensions of a lane, whether a wave has two heads)
template <typename F>
void for_lanes(const CacheArgs& a, bool f32, const F& launch) {
    const auto with = [&](auto e) {
        if (a.Dp == 64) launch(e, std::integral_constant<int, 2>{}, std::true_type{});
        else if (a.Dp <= 128) launch(e, std::integral_constant<int, 2>{}, std::false_type{});
        else launch(e, std::integral_constant<int, 4>{}, std::false_type{});
    };
    if (f32) with(0.0f);
    else with((__bf16)0.0f);
}

}  // namespace

hipError_t cache_write(HeadRows k, HeadRows v, bool f32, int64_t T, int H, int D, const int32_t* slots, Pages pages,
                       hipStream_t stream) {
    const CacheArgs a = cache_args(k, v, T, H, D, slots, pages);
    const CacheGrid g(a);
    const auto launch = [&](auto e, auto pd, auto two) {
        using E = decltype(e);
        constexpr int PD = decltype(pd)::value;
        constexpr bool TWO = decltype(two)::value;
        if (pages.bits == 16) cache_write_kernel<E, 16, PD, TWO><<<g.grid, g.threads, 0, stream>>>(a);
        else if (pages.bits == 8) cache_write_kernel<E, 8, PD, TWO><<<g.grid, g.threads, 0, stream>>>(a);
        else cache_write_kernel<E, 4, PD, TWO><<<g.grid, g.threads, 0, stream>>>(a);
    };
    for_lanes(a, f32, launch);
    return hipGetLastError();
}

hipError_t cache_read(Pages pages, const int32_t* slots, int64_t T, int H, int D, HeadRows k, HeadRows v, bool f32,
                      hipStream_t stream) {
    const CacheArgs a = cache_args(k, v, T, H, D, slots, pages);
    const CacheGrid g(a);
    const auto launch = [&](auto e, auto pd, auto two) {
        using E = decltype(e);
        constexpr int PD = decltype(pd)::value;
        constexpr bool TWO = decltype(two)::value;
        if (pages.bits == 16) cache_read_kernel<E, 16, PD, TWO><<<g.grid, g.threads, 0, stream>>>(a);
        else if (pages.bits == 8) cache_read_kernel<E, 8, PD, TWO><<<g.grid, g.threads, 0, stream>>>(a);
        else cache_read_kernel<E, 4, PD, TWO><<<g.grid, g.threads, 0, stream>>>(a);
    };
    for_lanes(a, f32, launch);
    return hipGetLastError();
}

}  // namespace gptq
