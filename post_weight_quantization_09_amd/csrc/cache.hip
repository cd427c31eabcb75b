// The paged cache of keys and values: rows quantised as they are written, and read back.
//
// A row of a token and head is kept on the symmetric grid of gptq_quantize_layer: s = absmax / (2^(b-1) - 1/2), codes
// round-half-even(x / s).  The rounding is exact, not that of a rounded quotient: with q = rint(x * (1 / s)) the remainder
// x - q s is representable (q has at most 8 bits, |x - q s| is not above s / 2 by more than a few of x's last places), so
// one fused multiply-add gives it and comparing it with s / 2 moves q to the neighbour where that is nearer, or even.
//
// Memory traffic is the bound.  A wave takes eight tokens of a head (two heads of 64): a lane holds two or four
// dimensions of each, so that rows are read and written in whole lines, their largest values found by maxima across the
// lanes, and eight tokens of a lane's dimensions are what the values' layout stores side by side.  Where eight
// tokens fill eight slots from a multiple of eight on, in order, they are stored with 8 or 16 bytes a lane; the wave that
// holds the first of them takes all eight, so that runs of any beginning in the batch are written so.  Other tokens' values
// go byte by byte into the octets that they share with tokens of other calls.
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

__device__ __forceinline__ int exact_code(float x, float s, float inv, float low, float high) {
    float q = rintf(x * inv);
    const float rem = fmaf(-q, s, x), twice = 2.0f * fabsf(rem);
    const bool odd = ((int)q & 1) != 0;
    if (twice > s || (twice == s && odd)) q += copysignf(1.0f, rem);
    return (int)fminf(fmaxf(q, low), high);
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

// The largest of a row's lanes: all 64, or each half's 32.
__device__ __forceinline__ uint32_t max_of_lanes(uint32_t x, bool halves) {
    x = max_dpp<0xB1>(x);                       // quad_perm 1, 0, 3, 2
    x = max_dpp<0x4E>(x);                       // quad_perm 2, 3, 0, 1
    x = max_dpp<0x141>(x);                      // row_half_mirror
    x = max_dpp<0x140>(x);                      // row_mirror
    auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = max(r[0], r[1]);
    if (halves) return x;
    r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return max(r[0], r[1]);
}

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
    for (int i = 0; i < N / 2; ++i) v[i] = pack_bf16x2_rne(x[2 * i], x[2 * i + 1]);
    *reinterpret_cast<any*>(p) = v;
}

// Which of a wave's tokens are taken together.  Lane i looks at token t0 - 7 + i; bit j of the results is token t0 + j.
struct Tokens {
    int32_t slot[kOctet];                       // of the wave's own tokens; -1 outside the pages
    int octet;                                  // the first of eight tokens that fill eight slots, or -1
    int32_t octet_slot;
    uint32_t single;                            // tokens in no such eight
};

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
    w.single = (uint32_t)(~covered >> (kOctet - 1)) & 0xFFu & ((1u << min(a.T - t0, kOctet)) - 1u);
    return w;
}

// A wave's rows: its lanes' head and dimensions.
template <int PD>
struct Lanes {
    int head, d;
    bool on, halves;
    __device__ Lanes(const CacheArgs& a, int lane) {
        halves = a.Dp == 64;                    // PD 2: two heads
        const int in = halves ? lane & 31 : lane;
        head = blockIdx.y * (halves ? 2 : 1) + (halves ? lane >> 5 : 0);
        d = in * PD;
        on = d < a.Dp && head < a.H;
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

template <int BITS, int PD>
struct Codes {
    uint32_t code[kOctet][PD];
    float scale[kOctet];
    template <typename E>
    __device__ void of(const Rows<E, PD>& r, bool inside, bool halves) {        // not inside: zeros
        constexpr float kLow = -(float)(1 << (BITS < 16 ? BITS - 1 : 0)), kHigh = -kLow - 1.0f;
        for (int i = 0; i < kOctet; ++i) {
            float x[PD];
            for (int j = 0; j < PD; ++j) x[j] = inside ? r.x[i].get(j) : 0.0f;
            if constexpr (BITS == 16) {
                for (int j = 0; j < PD; ++j) code[i][j] = (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)x[j]);
            } else {
                uint32_t m = 0;
                for (int j = 0; j < PD; ++j) m = max(m, __float_as_uint(x[j]) & 0x7FFFFFFFu);
                const float s = grid_scale<BITS>(max_of_lanes(m, halves)), inv = __builtin_amdgcn_rcpf(s);
                scale[i] = s;
                const bool fine = s == s;
                for (int j = 0; j < PD; ++j)
                    code[i][j] = fine ? (uint32_t)exact_code(x[j], s, inv, kLow, kHigh) & ((1u << BITS) - 1u) : 0u;
            }
        }
    }
};

template <typename E, int BITS, int PD>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheArgs a) {
    const int lane = threadIdx.x & 63, t0 = (blockIdx.x * (blockDim.x >> 6) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kOctet;
    if (t0 >= a.T) return;
    const Lanes<PD> l(a, lane);
    const Tokens w = tokens_of(a, t0, lane);
    uint32_t valid = 0;
    for (int i = 0; i < kOctet; ++i) valid |= (uint32_t)(w.slot[i] >= 0) << i;
    const uint32_t single = w.single & valid;
    if (!valid && w.octet < 0) return;
    const uint32_t part = (uint32_t)a.page_size * a.Dp * BITS / 8;
    uint8_t* head = a.pages + l.head * a.head_stride;
    // lanes without an element of a row read the first of the first head
    const bool inside = l.on && l.d < a.D, together = w.octet >= 0;
    const E* k = static_cast<const E*>(a.k) + t0 * a.k_ts + (inside ? l.head * a.k_hs + l.d : 0);
    const E* v = static_cast<const E*>(a.v) + t0 * a.v_ts + (inside ? l.head * a.v_hs + l.d : 0);

    Rows<E, PD> x, z;
    if (valid) x.load(k, a.k_ts, 0, valid);
    if (together || single) z.load(v, a.v_ts, together ? w.octet : 0, together ? 0xFFu : single);
    Codes<BITS, PD> c;

    // keys: a row per token
    c.of(x, inside, l.halves);
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
            if (l.d == 0) reinterpret_cast<float*>(block + 2 * part)[p.at] = c.scale[i];
        }
    }

    c.of(z, inside, l.halves);
    if (together) {
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
            if constexpr (BITS < 16)
                if (l.d == 0) {
                    f32x4* s = reinterpret_cast<f32x4*>(block + 2 * part + 4 * (a.page_size + p.at));
                    s[0] = f32x4{c.scale[0], c.scale[1], c.scale[2], c.scale[3]};
                    s[1] = f32x4{c.scale[4], c.scale[5], c.scale[6], c.scale[7]};
                }
        }
        if (!single) return;
        z.load(v, a.v_ts, 0, single);               // beside an octet, at the end of a run
        c.of(z, inside, l.halves);
    }
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
        if constexpr (BITS < 16)
            if (l.d == 0) reinterpret_cast<float*>(block + 2 * part)[a.page_size + p.at] = c.scale[i];
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

template <typename E, int BITS, int PD>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheArgs a) {
    const int lane = threadIdx.x & 63, t0 = (blockIdx.x * (blockDim.x >> 6) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * kOctet;
    if (t0 >= a.T) return;
    const Lanes<PD> l(a, lane);
    const Tokens w = tokens_of(a, t0, lane);
    if (!l.on || l.d >= a.D) return;
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

// A wave per eight tokens; as many waves a workgroup as leave a workgroup for every CU.
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

}  // namespace

hipError_t cache_write(HeadRows k, HeadRows v, bool f32, int64_t T, int H, int D, const int32_t* slots, Pages pages,
                       hipStream_t stream) {
    const CacheArgs a = cache_args(k, v, T, H, D, slots, pages);
    const CacheGrid g(a);
    const auto pick = [&](auto e, auto pd) {
        using E = decltype(e);
        constexpr int PD = decltype(pd)::value;
        return pages.bits == 16 ? cache_write_kernel<E, 16, PD> : pages.bits == 8 ? cache_write_kernel<E, 8, PD> : cache_write_kernel<E, 4, PD>;
    };
    const auto two = std::integral_constant<int, 2>{};
    const auto four = std::integral_constant<int, 4>{};
    auto* kernel = a.Dp <= 128 ? (f32 ? pick(0.0f, two) : pick((__bf16)0.0f, two)) : (f32 ? pick(0.0f, four) : pick((__bf16)0.0f, four));
    kernel<<<g.grid, g.threads, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t cache_read(Pages pages, const int32_t* slots, int64_t T, int H, int D, HeadRows k, HeadRows v, bool f32,
                      hipStream_t stream) {
    const CacheArgs a = cache_args(k, v, T, H, D, slots, pages);
    const CacheGrid g(a);
    const auto pick = [&](auto e, auto pd) {
        using E = decltype(e);
        constexpr int PD = decltype(pd)::value;
        return pages.bits == 16 ? cache_read_kernel<E, 16, PD> : pages.bits == 8 ? cache_read_kernel<E, 8, PD> : cache_read_kernel<E, 4, PD>;
    };
    const auto two = std::integral_constant<int, 2>{};
    const auto four = std::integral_constant<int, 4>{};
    auto* kernel = a.Dp <= 128 ? (f32 ? pick(0.0f, two) : pick((__bf16)0.0f, two)) : (f32 ? pick(0.0f, four) : pick((__bf16)0.0f, four));
    kernel<<<g.grid, g.threads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace gptq
