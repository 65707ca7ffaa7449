// Append of new keys and values to pages of 8-bit codes, one scale for each
// page, head and side.
//
//     s' = max(s, 2^ceil(log2(max|x| / M)))     over the page's new rows x; s
//                                               counts where it holds rows
//     code = round(x / s'),  M = 448 (e4m3), 127 (int8)
// A page's scale only grows while it fills, and when it does, the codes held
// are divided by s'/s and rounded again.  Scales are powers of two, so that
// dividing by them is exact: a value is rounded once, and an e4m3 code keeps
// its digits when its page grows (but for those below the smallest normal
// code); an int8 code is off by less than one step of the final scale however
// often its page has grown.  For e4m3 a power of two costs nothing, as a code's
// digits are the same in every octave; for int8 it is half a bit on average.
//
// Prompts: each row is read once and its codes are written once: HBM-bound.  A
// prompt of 32,768 tokens (8 heads of 128, normed and turned, bf16) takes 48 us
// on pages of 16, 4.2 TB/s, where a copy of 2 GiB reaches 4.8 to 4.9, 51 on pages
// of 64, and 76 on pages of 128, whose rows are read and turned twice; without
// norm and rotation 45.  Single tokens: launch-bound (64 of them 4.0 to 4.6 us,
// 4.2 of kernel), and the page is touched only where its scale grows.
//
// Norm and rotation have the formula's roundings, x * r * w and two products and
// a sum to each element, none of them fused: a key that a rounding has moved may
// get the next code, and so keys get those of the same formula in other fp32 but
// where the sum of squares differs (128 chunks of 512 tokens, 8 heads of 128, int8:
// 0.24 of a million codes differ from PyTorch's, 0.82 with the rotation's products
// fused and r as the last factor, which takes 1 us less on pages of 64).
//
// Mapping: as in norm_rope.hip D/16 lanes hold a row of 16 elements each.
//   * Chunks: a workgroup takes one page of one request and up to 16 heads of one
//     side, so that the cosines of the page's tokens are made once for all its
//     heads (by way of LDS).  A wave holds two steps of rows (16 rows of head_dim
//     128) as they are turned, with the next head's on their way; one, two or
//     four waves share a head by the page's new rows, and their maxima go by way
//     of LDS.  Of more rows than that (128, 64 and 32 of head_dim 64,
//     128 and 256) the maximum is found first, and they are read and turned
//     again.  (Pages of 64 read twice took 58 us; eight steps held by one wave as
//     they were read took all registers, 86.)
//     Four waves on a SIMD leave 128 registers: int8 takes 126, e4m3 spills 4 (12
//     bytes of scratch a lane).
//   * Single tokens: a wave takes as many (head, side) pairs of a token as it
//     holds rows.
#include <algorithm>

#include "head_rows.h"

namespace engram {
namespace {

typedef uint16_t u16x2v __attribute__((ext_vector_type(2)));
constexpr uint32_t kMagnitude = 0x7FFFFFFFu, kInfinite = 0x7F800000u;

// The two kinds of codes.
struct CodeE4m3 {
    // |x| <= largest = 1.75 * 2^8
    static constexpr uint32_t kMantissa = 0x600000u, kExponent = 8u;
    static __device__ __forceinline__ uint32_t four(const float* x, float by) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * by, x[1] * by, 0, false);
        return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * by, x[3] * by, lo, true));
    }
    static __device__ __forceinline__ uint32_t again(const float* x, float ratio) { return four(x, ratio); }
    static __device__ __forceinline__ void values(uint32_t w, float* x) {
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
        const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
        x[0] = a[0];
        x[1] = a[1];
        x[2] = b[0];
        x[3] = b[1];
    }
};
struct CodeI8 {
    // |x| <= largest = (127 / 64) * 2^6
    static constexpr uint32_t kMantissa = 0x7E0000u, kExponent = 6u;
    // Codes held, times a ratio of -1 to 1; -128, which no append writes, is -127 where the sign changes.
    static __device__ __forceinline__ uint32_t again(const float* x, float ratio) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = ratio < 0.0f ? fmaxf(x[i], -127.0f) : x[i];
        return four(y, ratio);
    }
    static __device__ __forceinline__ uint32_t four(const float* x, float by) {
        // 1.5 * 2^23 leaves the whole number nearest to the product (ties to even) in the low bits: one rounding, as the
        // product is inside of the fused step
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(uint32_t, __builtin_fmaf(x[i], by, 12582912.0f));
        const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x0C0C0400u), b = __builtin_amdgcn_perm(w[3], w[2], 0x04000C0Cu);
        return a | b;
    }
    static __device__ __forceinline__ void values(uint32_t w, float* x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
    }
};

// The least power of two whose largest code holds a magnitude, given by its bits; a NaN or infinity has NaN.
template <class C>
__device__ __forceinline__ float scale_for(uint32_t bits) {
    if (bits >= kInfinite) return __builtin_nanf("");
    if (bits == 0u) return 0.0f;
    const int32_t e = static_cast<int32_t>((bits + (0x7FFFFFu - C::kMantissa)) >> 23) - static_cast<int32_t>(C::kExponent);
    return __builtin_bit_cast(float, static_cast<uint32_t>(max(e, 1)) << 23);
}

// A page's scale before and after: `old` counts where the page holds rows.
struct Scale {
    float now, by;  // by: 1 / now (0 for 0)
    float ratio;    // of the codes held, where they have to be rounded again; else 1
};
__device__ __forceinline__ Scale grown(float need, float old, bool held) {
    Scale s;
    const bool more = held && need > fabsf(old);  // (a scale from elsewhere may be negative, and stays so)
    // a NaN on either side stays
    s.now = more || !held || need != need ? need : old;
    s.by = s.now == 0.0f ? 0.0f : 1.0f / s.now;
    s.ratio = more ? old * s.by : 1.0f;
    return s;
}

template <class C>
__device__ __forceinline__ void encode16(uint8_t* row, const float* x, float by, const Blocks& b) {
    *reinterpret_cast<u32x2v*>(row + b.b0 * 8u) = u32x2v{C::four(x, by), C::four(x + 4, by)};
    *reinterpret_cast<u32x2v*>(row + b.b1 * 8u) = u32x2v{C::four(x + 8, by), C::four(x + 12, by)};
}

// 16 codes rounded again.
template <class C>
__device__ __forceinline__ u32x4v again(u32x4v w, float ratio) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x[4];
        C::values(w[i], x);
        w[i] = C::again(x, ratio);
    }
    return w;
}

__device__ __forceinline__ uint32_t largest16(const float* x) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = max(m, __builtin_bit_cast(uint32_t, x[e]) & kMagnitude);
    return m;
}

// The lanes' exchange within a row of LPH, and over the wave, without LDS.
template <int kControl>
__device__ __forceinline__ uint32_t moved(uint32_t x) {
    return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), kControl, 0xF, 0xF, true));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;  // of 16 lanes
template <int LPH>
__device__ __forceinline__ float row_sum(float x) {
    const auto add = [&](uint32_t y) { x += __builtin_bit_cast(float, y); };
    const auto bits = [&]() { return __builtin_bit_cast(uint32_t, x); };
    add(moved<kXor1>(bits()));
    add(moved<kXor2>(bits()));
    if constexpr (LPH >= 8) add(moved<kMirror8>(bits()));
    if constexpr (LPH >= 16) add(moved<kMirror16>(bits()));
    return x;
}
template <int LPH>
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
    x = max(x, moved<kXor1>(x));
    x = max(x, moved<kXor2>(x));
    if constexpr (LPH >= 8) x = max(x, moved<kMirror8>(x));
    if constexpr (LPH >= 16) x = max(x, moved<kMirror16>(x));
    return x;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    x = row_max<16>(x);
    const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = max(static_cast<uint32_t>(a[0]), static_cast<uint32_t>(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return max(static_cast<uint32_t>(b[0]), static_cast<uint32_t>(b[1]));
}

// 1 / sqrt(x) within an fp32 step; the instruction by itself knows no numbers below 2^-126.
__device__ __forceinline__ float inverse_root(float x) {
    const bool small = x < 0x1p-96f;
    return __builtin_amdgcn_rsqf(small ? x * 0x1p96f : x) * (small ? 0x1p48f : 1.0f);
}

// The rotation with each product and sum rounded by itself.
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
#pragma clang fp contract(off)
    const float ac = a * c, bs = b * s, as = a * s, bc = b * c;
    a = ac - bs;
    b = as + bc;
}
__device__ __forceinline__ void turn_apart(float* x, const Turn& t, bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn_pair(x[2 * e], x[2 * e + 1], t.c[e], t.s[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) turn_pair(x[e], x[8 + e], t.c[e], t.s[e]);
    }
}

// A request's new tokens and the keys that they are.  Lengths are bounded by what exists.
struct Fresh {
    uint32_t q0, q_len;
    int32_t kv_len, first;  // keys first .. kv_len - 1; those below 0 are left out
};
__device__ __forceinline__ Fresh fresh_of(const AppendPagesArgs& A, uint32_t b) {
    Fresh r;
    if (A.cu_q) {
        const int32_t n = static_cast<int32_t>(A.n_tok);
        const int32_t q0 = min(max(A.cu_q[b], 0), n), q1 = min(max(A.cu_q[b + 1], q0), n);
        r.q0 = static_cast<uint32_t>(q0);
        r.q_len = static_cast<uint32_t>(q1 - q0);
    } else {
        r.q0 = b * A.uniform_q;
        r.q_len = A.uniform_q;
    }
    const uint64_t room = static_cast<uint64_t>(A.table_width) << A.cache.page_shift;
    constexpr int32_t kMost = INT32_MAX - 4095;
    r.kv_len = min(max(A.kv_len[b], 0), room < static_cast<uint64_t>(kMost) ? static_cast<int32_t>(room) : kMost);
    r.first = r.kv_len - static_cast<int32_t>(r.q_len);
    return r;
}

// Where a request's pages begin among all, with room for each request's first and last: a run of n tokens touches at most
// floor((n + page - 2) / page) + 1 <= floor(n / page) + 2 pages, and floor(x + y) + 2 - floor(x) >= floor(y) + 2.
__device__ __forceinline__ uint32_t pages_before(const AppendPagesArgs& A, uint32_t b) {
    const int32_t n = static_cast<int32_t>(A.n_tok);
    return (static_cast<uint32_t>(min(max(A.cu_q[b], 0), n)) >> A.cache.page_shift) + 2u * b;
}

constexpr uint32_t kSteps = 8;   // of a wave's rows, whose cosines are held
constexpr uint32_t kHeads = 16;  // of a workgroup at most, their keys or their values (append_heads)

// One page of one request: rows row0 .. row0 + n_rows - 1 of it are new, tokens tok0 on.
template <class T, int D, class C>
struct Page {
    static constexpr int LPH = D / 16;
    static constexpr uint32_t RPW = 64 / LPH, kHold = kSteps * RPW;  // rows of a step, rows whose cosines are held
    const AppendPagesArgs& A;
    f32x2v* cs;  // LDS: cosines and sines of kHold rows
    int64_t page;
    uint32_t row0, n_rows, tok0, head0, n_heads;
    uint32_t wave, lane, j, of_step, rb;
    Blocks bl;
    float weight[16];

    // A head's keys or values.
    template <bool kKey>
    struct Pair {
        uint32_t head;
    };
    template <bool kKey>
    __device__ __forceinline__ float* scale_of(Pair<kKey> p) const {
        return (kKey ? A.cache.k_scale : A.cache.v_scale) + page * A.cache.n_kv_heads + p.head;
    }
    template <bool kKey>
    __device__ __forceinline__ uint8_t* codes_of(Pair<kKey> p) const {
        return (kKey ? A.cache.k + page * A.cache.k_page_stride : A.cache.v + page * A.cache.v_page_stride) +
               (static_cast<int64_t>(p.head) << A.cache.page_shift) * D;
    }
    // the page's scale, if it holds rows
    template <bool kKey>
    __device__ __forceinline__ float held_scale(Pair<kKey> p) const { return row0 ? *scale_of(p) : 0.0f; }

    // Row r (and of_step more) of the pair, as it was given; past the last row, that one again.
    struct Raw {
        u32x4v w[2];
    };
    template <bool kKey>
    __device__ __forceinline__ Raw load(Pair<kKey> p, uint32_t r) const {
        constexpr int kSide = kKey ? 0 : 1;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(A.src[kSide]) + p.head * A.src_head[kSide] +
                              (tok0 + min(r + of_step, n_rows - 1u)) * A.src_tok[kSide];
        return Raw{{*reinterpret_cast<const u32x4v*>(src + bl.b0 * 8u), *reinterpret_cast<const u32x4v*>(src + bl.b1 * 8u)}};
    }
    // Where pair q of row r's cosine and sine lie: 16-byte blocks of two pairs, turned within their 64 bytes by the lane that
    // reads them, so that 16 lanes of a read meet on no bank (all rows begin on the same one).
    __device__ __forceinline__ uint32_t turn_at(uint32_t r, uint32_t q) const {
        const uint32_t turn = (r * LPH + (q >> 3)) >> 2;
        return r * (8u * rb) + (q & ~7u) + ((q + 2u * turn) & 6u) + (q & 1u);
    }
    __device__ __forceinline__ Turn turn_for(uint32_t r) const {
        Turn t;
#pragma unroll
        for (uint32_t e = 0; e < 8; e += 2) {
            const uint32_t q = A.interleaved ? (e < 4 ? 4u * j + e : 4u * (j + rb) + (e - 4)) : 8u * j + e;
            const f32x4v x = *reinterpret_cast<const f32x4v*>(cs + turn_at(r, q));
            t.c[e] = x[0];
            t.s[e] = x[1];
            t.c[e + 1] = x[2];
            t.s[e + 1] = x[3];
        }
        return t;
    }
    // Cosines and sines of rows r0 .. r0 + kHold - 1, by the whole workgroup.
    __device__ __forceinline__ void make_turns(uint32_t r0) const {
        if (!rb) return;
        const uint32_t pairs = 8u * rb, n = min(n_rows - r0, kHold) * pairs;
        for (uint32_t i = threadIdx.x; i < n; i += 256u) {
            const uint32_t row = i / pairs;
            const uint32_t q = i - row * pairs;
            cs[turn_at(row, q)] = cos_sin(static_cast<double>(A.positions[tok0 + r0 + row]) * A.inv_freq[q]);
        }
    }
    // The row as it is to be stored; f: its norm's factor.
    template <bool kKey>
    __device__ __forceinline__ void turned(const Raw& h, Pair<kKey>, uint32_t r, uint32_t r0, float f, float* x) const {
        unpack8<T>(h.w[0], x);
        unpack8<T>(h.w[1], x + 8);
        if constexpr (kKey) {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = x[e] * f * weight[e];
            if (j < rb) turn_apart(x, turn_for(min(r + of_step, n_rows - 1u) - r0), A.interleaved != 0);
        }
    }
    template <bool kKey>
    __device__ __forceinline__ float factor(const Raw& h, Pair<kKey>) const {
        if constexpr (!kKey) return 1.0f;
        float x[16], ss = 0.0f;
        unpack8<T>(h.w[0], x);
        unpack8<T>(h.w[1], x + 8);
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = __builtin_fmaf(x[e], x[e], ss);
        const float f = inverse_root(row_sum<LPH>(ss) * (1.0f / D) + A.eps);
        return A.weight ? f : 1.0f;
    }
    // The largest magnitude of the row, by its bits.
    template <bool kKey>
    __device__ __forceinline__ uint32_t largest(const Raw& h, Pair<kKey> p, uint32_t r, uint32_t r0, float f) const {
        if constexpr (kKey) {
            float x[16];
            turned(h, p, r, r0, f, x);
            return largest16(x);
        } else {  // 16-bit magnitudes are in order as whole numbers
            u16x2v m = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2v, h.w[i / 4][i % 4] & 0x7FFF7FFFu));
            const uint32_t both = max(static_cast<uint32_t>(m[0]), static_cast<uint32_t>(m[1]));
            return __builtin_bit_cast(uint32_t, T::lo(both));
        }
    }
    // The page's scale, and the codes that it holds; the new rows' factor.
    // (kOf waves share the head.)
    template <uint32_t kOf, bool kKey>
    __device__ __forceinline__ float settle(Pair<kKey> p, uint32_t most, float old) const {
        const Scale s = grown(scale_for<C>(most), old, row0 > 0u);
        const uint32_t at = (wave & (kOf - 1u)) * 64u + lane;
        if (at == 0) *scale_of(p) = s.now;
        if (s.ratio != 1.0f) {
            uint8_t* const codes = codes_of(p);
            for (uint32_t i = at * 16u; i < row0 * D; i += kOf * 1024u) {
                u32x4v* const q = reinterpret_cast<u32x4v*>(codes + i);
                *q = again<C>(*q, s.ratio);
            }
        }
        return s.by;
    }
    template <bool kKey>
    __device__ __forceinline__ void store(const Raw& h, Pair<kKey> p, uint32_t r, uint32_t r0, float by) const {
        float x[16];
        turned(h, p, r, r0, factor(h, p), x);
        put(x, p, r, by);
    }
    template <bool kKey>
    __device__ __forceinline__ void put(const float* x, Pair<kKey> p, uint32_t r, float by) const {
        if (r + of_step < n_rows) encode16<C>(codes_of(p) + static_cast<uint64_t>(row0 + r + of_step) * D, x, by, bl);
    }

    // Up to two steps of rows to a wave: held as they are turned, the next head's on their way.  kOf waves share a head's rows,
    // and the waves' maxima go by way of LDS (most: two sets of 4 words, used in turn, so that one barrier a head is enough).
    template <uint32_t kOf, bool kKey>
    __device__ __forceinline__ void held_rows(uint32_t* most) const {
        constexpr uint32_t kAtOnce = 4u / kOf;
        const uint32_t r = (wave & (kOf - 1u)) * 2u * RPW, first = wave / kOf;
        const auto ask = [&](uint32_t k, Raw* raw) {
            const Pair<kKey> p = {head0 + min(k, n_heads - 1u)};
            raw[0] = load(p, r);
            raw[1] = load(p, r + RPW);
            return held_scale(p);
        };
        Raw next[2];
        float next_old = ask(first, next);
        if (kKey) {
            make_turns(0);
            __syncthreads();
        }
        const uint32_t rounds = (n_heads + kAtOnce - 1u) / kAtOnce;  // the same for all waves
        for (uint32_t i = 0; i < (kOf == 1 ? (n_heads - min(first, n_heads) + 3u) / 4u : rounds); ++i) {
            const uint32_t k = i * kAtOnce + first;
            const bool live = kOf == 1 || k < n_heads;
            const Pair<kKey> p = {head0 + min(k, n_heads - 1u)};
            float x[2][16];
            uint32_t m = 0;
#pragma unroll
            for (uint32_t z = 0; z < 2; ++z) {
                turned(next[z], p, r + z * RPW, 0, factor(next[z], p), x[z]);
                m = max(m, largest16(x[z]));
            }
            const float old = next_old;
            if (k + kAtOnce < n_heads) next_old = ask(k + kAtOnce, next);
            m = wave_max(m);
            if constexpr (kOf > 1) {
                uint32_t* const of_round = most + (i & 1u) * 4u;
                if (lane == 0) of_round[wave] = m;
                __syncthreads();
#pragma unroll
                for (uint32_t w = 0; w < kOf; ++w) m = max(m, of_round[(wave & ~(kOf - 1u)) + w]);
            }
            if (!live) continue;
            const float by = settle<kOf>(p, m, old);
            put(x[0], p, r, by);
            if (r + RPW < n_rows) put(x[1], p, r + RPW, by);
        }
    }

    // More, that are not turned: read twice, the second time from the caches.
    template <bool kKey>
    __device__ __forceinline__ void more_rows() const {
        for (uint32_t k = wave; k < n_heads; k += 4u) {
            const Pair<kKey> p = {head0 + k};
            const float old = held_scale(p);
            const float by = settle<1>(p, wave_max(largest_of(p, 0, n_rows)), old);
            store_all(p, 0, n_rows, by);
        }
    }
    template <bool kKey>
    __device__ __forceinline__ uint32_t largest_of(Pair<kKey> p, uint32_t r0, uint32_t r1) const {
        uint32_t m = 0;
        each(p, r0, r1, [&](const Raw& raw, uint32_t r) { m = max(m, largest(raw, p, r, r0, factor(raw, p))); });
        return m;
    }
    template <bool kKey>
    __device__ __forceinline__ void store_all(Pair<kKey> p, uint32_t r0, uint32_t r1, float by) const {
        each(p, r0, r1, [&](const Raw& raw, uint32_t r) { store(raw, p, r, r0, by); });
    }
    // A head's rows step by step, kAhead steps on their way.
    template <bool kKey, class F>
    __device__ __forceinline__ void each(Pair<kKey> p, uint32_t r0, uint32_t r1, F f) const {
        constexpr uint32_t kAhead = 2;
        Raw raw[kAhead];
#pragma unroll
        for (uint32_t i = 0; i < kAhead; ++i) raw[i] = load(p, r0 + i * RPW);
        for (uint32_t r = r0; r < r1; r += kAhead * RPW) {
#pragma unroll
            for (uint32_t i = 0; i < kAhead; ++i) {
                const Raw now = raw[i];
                raw[i] = load(p, r + (kAhead + i) * RPW);
                if (i == 0 || r + i * RPW < r1) f(now, r + i * RPW);
            }
        }
    }

    // More rows than a wave holds: read twice.  most: LDS of kHeads words.
    template <bool kKey>
    __device__ __forceinline__ void in_parts(uint32_t* most) const {
        if (threadIdx.x < kHeads) most[threadIdx.x] = 0;
        for (uint32_t pass = 0; pass < 2; ++pass) {
            for (uint32_t r0 = 0; r0 < n_rows; r0 += kHold) {
                __syncthreads();
                if (kKey) make_turns(r0);
                __syncthreads();
                for (uint32_t k = wave; k < n_heads; k += 4u) {
                    const Pair<kKey> p = {head0 + k};
                    const uint32_t r1 = min(r0 + kHold, n_rows);
                    if (pass == 0) {
                        const uint32_t m = wave_max(largest_of(p, r0, r1));
                        if (lane == 0) most[k] = max(most[k], m);  // the wave's own
                    } else {
                        store_all(p, r0, r1, __builtin_bit_cast(float, most[k]));
                    }
                }
            }
            if (pass == 0) {
                __syncthreads();
                for (uint32_t k = wave; k < n_heads; k += 4u) {
                    const Pair<kKey> p = {head0 + k};
                    const float by = settle<1>(p, most[k], held_scale(p));
                    if (lane == 0) most[k] = __builtin_bit_cast(uint32_t, by);
                }
            }
        }
    }

    template <bool kKey>
    __device__ __forceinline__ void append(uint32_t* most) const {
        if (n_rows <= 2 * RPW)
            held_rows<1, kKey>(most);
        else if (n_rows <= 4 * RPW)
            held_rows<2, kKey>(most);
        else if (n_rows <= kHold)
            held_rows<4, kKey>(most);
        else if (!kKey || !rb)
            more_rows<kKey>();
        else
            in_parts<kKey>(most);
    }
};

template <class T, int D, class C>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4))) void append_pages_kernel(const AppendPagesArgs A,
                                                                                                           uint32_t heads_each) {
    using P = Page<T, D, C>;
    __shared__ __attribute__((aligned(16))) f32x2v sm_cs[P::kHold * (D / 2)];
    __shared__ uint32_t sm_most[kHeads];
    const uint32_t lane = threadIdx.x & 63u;
    uint32_t b, at;  // request, and which of its pages
    if (A.pages_per) {
        b = blockIdx.x / A.pages_per;
        at = blockIdx.x - b * A.pages_per;
    } else {
        uint32_t lo = 0, n = A.n_seq;  // the last request that begins at or before this place, 64 candidates at a time
        while (n > 1u) {
            const uint32_t step = (n + 63u) / 64u, i = lo + lane * step;
            const bool before = i < lo + n && pages_before(A, i) <= blockIdx.x;
            const uint32_t k = static_cast<uint32_t>(__builtin_popcountll(__ballot(before)));
            const uint32_t first = k ? lo + (k - 1u) * step : lo;
            n = min(step, lo + n - first);
            lo = first;
        }
        b = lo;
        at = blockIdx.x - min(blockIdx.x, pages_before(A, lo));
    }
    const Fresh req = fresh_of(A, b);
    const uint32_t shift = A.cache.page_shift;
    const int32_t lo = max(req.first, 0);
    if (lo >= req.kv_len) return;
    const uint32_t in_table = (static_cast<uint32_t>(lo) >> shift) + at;
    if (in_table > static_cast<uint32_t>(req.kv_len - 1) >> shift) return;
    const int64_t page = A.table[b * A.table_stride + in_table];
    if (page < 0 || page >= A.cache.n_pages) return;
    const uint32_t key0 = in_table << shift;
    P p = {A, sm_cs};
    p.page = page;
    p.row0 = max(static_cast<uint32_t>(lo), key0) - key0;
    p.n_rows = min(static_cast<uint32_t>(req.kv_len) - key0, 1u << shift) - p.row0;
    p.tok0 = req.q0 + (key0 + p.row0 - static_cast<uint32_t>(req.first));
    const uint32_t of_side = gridDim.y / 2u, part = blockIdx.y % of_side;
    p.head0 = part * heads_each;
    p.n_heads = min(A.cache.n_kv_heads - p.head0, heads_each);
    p.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    p.lane = lane;
    p.j = lane & (P::LPH - 1u);
    p.of_step = lane / P::LPH;
    p.rb = A.rotary / 16u;
    p.bl = blocks_of(p.j, p.rb);
    if (blockIdx.y < of_side) {
#pragma unroll
        for (int e = 0; e < 16; ++e) p.weight[e] = 1.0f;
        if (A.weight) {
            const uint16_t* wp = reinterpret_cast<const uint16_t*>(A.weight);
            unpack8<T>(*reinterpret_cast<const u32x4v*>(wp + p.bl.b0 * 8u), p.weight);
            unpack8<T>(*reinterpret_cast<const u32x4v*>(wp + p.bl.b1 * 8u), p.weight + 8);
        }
        p.template append<true>(sm_most);
    } else {
        p.template append<false>(sm_most);
    }
}

// One token a request, its first (others are past max_q_len): a wave takes RPW (head, side) pairs of it.
template <class T, int D, class C>
__global__ __launch_bounds__(256) void append_token_kernel(const AppendPagesArgs A, uint32_t steps) {
    constexpr int LPH = D / 16;
    constexpr uint32_t RPW = 64 / LPH;
    __shared__ f32x2v sm_cs[4][D / 2];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u, j = lane & (LPH - 1u);
    const uint32_t item = blockIdx.x * 4u + wave, b = item / steps;
    if (b >= A.n_seq) return;
    const Fresh req = fresh_of(A, b);
    if (req.q_len == 0u || req.first < 0) return;
    const uint32_t tok = req.q0, heads = A.cache.n_kv_heads, shift = A.cache.page_shift;
    const uint32_t pair = (item - b * steps) * RPW + lane / LPH;
    const bool live = pair < 2u * heads;
    const uint32_t side = pair < heads ? 0u : 1u, head = live ? (side ? pair - heads : pair) : 0u;
    const uint32_t rb = A.rotary / 16u;
    const bool il = A.interleaved != 0;
    const Blocks bl = blocks_of(j, rb);
    u32x4v raw[2];
    {
        const uint16_t* src = reinterpret_cast<const uint16_t*>(side ? A.src[1] : A.src[0]) +
                              tok * (side ? A.src_tok[1] : A.src_tok[0]) + head * (side ? A.src_head[1] : A.src_head[0]);
        raw[0] = *reinterpret_cast<const u32x4v*>(src + bl.b0 * 8u);
        raw[1] = *reinterpret_cast<const u32x4v*>(src + bl.b1 * 8u);
    }
    const uint32_t key = static_cast<uint32_t>(req.first), place = key & ((1u << shift) - 1u);
    const int64_t page = A.table[b * A.table_stride + (key >> shift)];
    if (page < 0 || page >= A.cache.n_pages) return;
    float* const scale = (side ? A.cache.v_scale : A.cache.k_scale) + page * heads + head;
    const float old = place ? *scale : 0.0f;
    uint8_t* const codes = (side ? A.cache.v + page * A.cache.v_page_stride : A.cache.k + page * A.cache.k_page_stride) +
                           (static_cast<int64_t>(head) << shift) * D;
    if (rb) {
        const uint32_t pairs = 8u * rb;
#pragma unroll
        for (uint32_t i = 0; i < (D / 2 + 63) / 64; ++i) {
            const uint32_t at = i * 64u + lane;
            if (at < pairs) sm_cs[wave][at] = cos_sin(static_cast<double>(A.positions[tok]) * A.inv_freq[at]);
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
    float x[16];
    unpack8<T>(raw[0], x);
    unpack8<T>(raw[1], x + 8);
    if (side == 0) {  // the same for all lanes of a row
        if (A.weight) {
            float w[16], ss = 0.0f;
            const uint16_t* wp = reinterpret_cast<const uint16_t*>(A.weight);
            unpack8<T>(*reinterpret_cast<const u32x4v*>(wp + bl.b0 * 8u), w);
            unpack8<T>(*reinterpret_cast<const u32x4v*>(wp + bl.b1 * 8u), w + 8);
#pragma unroll
            for (int e = 0; e < 16; ++e) ss = __builtin_fmaf(x[e], x[e], ss);
            const float f = inverse_root(row_sum<LPH>(ss) * (1.0f / D) + A.eps);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = x[e] * f * w[e];
        }
        if (j < rb) turn_apart(x, turn_of(sm_cs[wave], j, rb, il), il);
    }
    const uint32_t m = row_max<LPH>(largest16(x));
    if (!live) return;
    const Scale s = grown(scale_for<C>(m), old, place > 0u);
    encode16<C>(codes + static_cast<uint64_t>(place) * D, x, s.by, bl);
    if (j == 0) *scale = s.now;
    if (s.ratio != 1.0f) {
#pragma unroll 4
        for (uint32_t r = 0; r < place; ++r) {
            u32x4v* const p = reinterpret_cast<u32x4v*>(codes + static_cast<uint64_t>(r) * D + j * 16u);
            *p = again<C>(*p, s.ratio);
        }
    }
}

template <class T, int D, class C>
hipError_t pages_one(const AppendPagesArgs& a, hipStream_t stream) {
    const uint32_t pairs = 2u * a.cache.n_kv_heads;
    if (a.most_q == 1u) {
        constexpr uint32_t kRows = 1024 / D;
        const uint32_t steps = (pairs + kRows - 1u) / kRows;
        hipLaunchKernelGGL((append_token_kernel<T, D, C>), dim3((a.n_seq * steps + 3u) / 4u), dim3(256), 0, stream, a, steps);
    } else {
        const uint32_t pages = a.pages_per ? a.n_seq * a.pages_per : (a.n_tok >> a.cache.page_shift) + 2u * a.n_seq;
        const uint32_t heads = a.cache.n_kv_heads;
        const uint32_t each = append_heads(pages, heads, a.rotary > 0);
        hipLaunchKernelGGL((append_pages_kernel<T, D, C>), dim3(pages, 2u * ((heads + each - 1u) / each)), dim3(256), 0, stream, a,
                           each);
    }
    return hipGetLastError();
}

template <class T, class C>
hipError_t pages_dim(const AppendPagesArgs& a, uint32_t dim, hipStream_t stream) {
    switch (dim) {
        case 64: return pages_one<T, 64, C>(a, stream);
        case 128: return pages_one<T, 128, C>(a, stream);
        default: return pages_one<T, 256, C>(a, stream);
    }
}

}  // namespace

hipError_t launch_append_pages(const AppendPagesArgs& a, uint32_t dim, uint32_t type, bool int8, hipStream_t stream) {
    if (type == ENGRAM_BF16)
        return int8 ? pages_dim<Bf16, CodeI8>(a, dim, stream) : pages_dim<Bf16, CodeE4m3>(a, dim, stream);
    return int8 ? pages_dim<F16, CodeI8>(a, dim, stream) : pages_dim<F16, CodeE4m3>(a, dim, stream);
}

}  // namespace engram
