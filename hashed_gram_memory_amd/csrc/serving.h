// Shared by the serving kernels (head norm + rotation, cache append, paged
// attention): element types, conversions, the cache's addressing.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "engram.h"

namespace engram {

typedef float f32x2v __attribute__((ext_vector_type(2)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef float f32x16v __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2v __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8v __attribute__((ext_vector_type(8)));

// What the two 16-bit element types share, by the bits of an exponent of all
// ones and those of the number 1.  A register pair of them is one uint32_t.
template <uint32_t kExp, uint32_t kUnit>
struct Halves {
    // all bits of each half that is an infinity or NaN: its exponent plus one carries into the sign's place
    static __device__ __forceinline__ uint32_t nonfinite(uint32_t w) {
        const uint32_t carry = ((w & (kExp * 0x10001u)) + kLow * 0x10001u) & 0x80008000u;
        return (carry >> 15) * 0xFFFFu;
    }
    // the number 1 in each half that is +infinity or NaN (-infinity or NaN), 0 in the others
    static __device__ __forceinline__ uint32_t not_below(uint32_t w) { return not_one(w, 0x8000u | kExp); }
    static __device__ __forceinline__ uint32_t not_above(uint32_t w) { return not_one(w, kExp); }
    // the number 1 or 0 in each half, by bits 0 and 1
    static __device__ __forceinline__ uint32_t ones(uint32_t bits) { return ((bits & 1u) | (bits & 2u) << 15) * kUnit; }

private:
    static constexpr uint32_t kLow = kExp & (~kExp + 1u);  // the exponent's last place
    static __device__ __forceinline__ uint32_t not_one(uint32_t w, uint32_t out) {
        const uint32_t x = w ^ (out * 0x10001u);  // 0 in the halves that do not count
        const uint32_t some = ((x & 0x7FFF7FFFu) + 0x7FFF7FFFu) | x;  // a half's sign: it is not 0
        return ((nonfinite(w) & some & 0x80008000u) >> 15) * kUnit;
    }
};

struct Bf16 : Halves<0x7F80u, 0x3F80u> {
    static __device__ __forceinline__ float lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
    static __device__ __forceinline__ float hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
    // round to nearest even
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const f32x2v x = {a, b};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2v));
    }
    static __device__ __forceinline__ f32x4v mfma16(u32x4v a, u32x4v b, f32x4v c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8v, a), __builtin_bit_cast(bf16x8v, b), c,
                                                       0, 0, 0);
    }
    static __device__ __forceinline__ f32x16v mfma32(u32x4v a, u32x4v b, f32x16v c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8v, a), __builtin_bit_cast(bf16x8v, b), c,
                                                       0, 0, 0);
    }
    // two e4m3 codes (bytes 0 and 1, or 2 and 3, of w): exact in this type
    template <bool kHigh>
    static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, kHigh));
    }
    // four int8 codes likewise: their floats have no digits below this type's.  (The compiler takes a byte out of its word
    // first, and 3.25 instructions to a code where these are 1.5.)
    static __device__ __forceinline__ u32x2v from_i8(uint32_t w) {
        float a, b, c, d;
        bytes(w, a, b, c, d);
        return u32x2v{halves(a, b), halves(c, d)};
    }
    static __device__ __forceinline__ void bytes(uint32_t w, float& a, float& b, float& c, float& d) {
        asm("v_cvt_f32_i32_sdwa %0, sext(%4) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0\n\t"
            "v_cvt_f32_i32_sdwa %1, sext(%4) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1\n\t"
            "v_cvt_f32_i32_sdwa %2, sext(%4) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2\n\t"
            "v_cvt_f32_i32_sdwa %3, sext(%4) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3"
            : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d)
            : "v"(w));
    }
    static __device__ __forceinline__ uint32_t halves(float a, float b) {
        return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u);
    }
    // Softmax terms are held as 2^kShift at their row's reference, and may pass
    // it by 2^kSlack before the reference moves.
    static constexpr float kShift = 0.0f, kSlack = 8.0f;
};

struct F16 : Halves<0x7C00u, 0x3C00u> {
    static __device__ __forceinline__ float lo(uint32_t w) {
        return static_cast<float>(__builtin_bit_cast(f16x2v, w)[0]);
    }
    static __device__ __forceinline__ float hi(uint32_t w) {
        return static_cast<float>(__builtin_bit_cast(f16x2v, w)[1]);
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const f32x2v x = {a, b};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, f16x2v));
    }
    static __device__ __forceinline__ f32x4v mfma16(u32x4v a, u32x4v b, f32x4v c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8v, a), __builtin_bit_cast(f16x8v, b), c, 0,
                                                      0, 0);
    }
    static __device__ __forceinline__ f32x16v mfma32(u32x4v a, u32x4v b, f32x16v c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8v, a), __builtin_bit_cast(f16x8v, b), c, 0,
                                                      0, 0);
    }
    template <bool kHigh>
    static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, kHigh));
    }
    // 1,024 + 128 + the code by its bits, less 1,152: both exact
    static __device__ __forceinline__ u32x2v from_i8(uint32_t w) {
        const f16x2v off = {static_cast<_Float16>(1152.0f), static_cast<_Float16>(1152.0f)};
        const uint32_t u = w ^ 0x80808080u;
        const f16x2v a = __builtin_bit_cast(f16x2v, __builtin_amdgcn_perm(u, 0x64646464u, 0x00050004u)) - off;
        const f16x2v b = __builtin_bit_cast(f16x2v, __builtin_amdgcn_perm(u, 0x64646464u, 0x00070006u)) - off;
        return u32x2v{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
    }
    // fp16 ends at 65,504 and has all its digits down to 2^-14: with a term of
    // 2^14 at most, one of 2^-21 of the reference is still a normal number.
    static constexpr float kShift = 7.0f, kSlack = 7.0f;
};

// What a cache holds: 16-bit numbers, or codes with a scale for each row (e4m3)
// or for each page and head (e4m3, int8).
enum Held : int { kHalves, kE4m3Rows, kE4m3Pages, kI8Pages };

// The four codes of w as numbers of type T, exactly.
template <class T, int kHeld>
__device__ __forceinline__ u32x2v from_codes(uint32_t w) {
    if constexpr (kHeld == kI8Pages)
        return T::from_i8(w);
    else
        return u32x2v{T::template from_e4m3<false>(w), T::template from_e4m3<true>(w)};
}

// Whether a scale is a power of two that keeps bf16's numbers clear of the type's ends: no sign, no digits, 2^-101 to 2^100.
__device__ __forceinline__ bool plain_scale(float scale) {
    const uint32_t bits = __builtin_bit_cast(uint32_t, scale);
    return (bits & 0x807FFFFFu) == 0u && bits - 0x0D000000u < 0x65000000u;
}
// The four codes of w times their page's scale as bf16: exact for a power of two, else rounded once.  kPlain: plain_scale
// holds, and the conversion of e4m3 scales by itself.
template <int kHeld, bool kPlain>
__device__ __forceinline__ u32x2v scaled_codes(uint32_t w, float scale) {
    if constexpr (kHeld == kI8Pages) {
        float a, b, c, d;
        Bf16::bytes(w, a, b, c, d);
        return u32x2v{Bf16::pack(a * scale, b * scale), Bf16::pack(c * scale, d * scale)};
    } else if constexpr (kPlain) {
        return u32x2v{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true))};
    } else {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
        return u32x2v{Bf16::pack(lo[0] * scale, lo[1] * scale), Bf16::pack(hi[0] * scale, hi[1] * scale)};
    }
}

// The four codes of w times a power of two of 2^-5 to 2^5 as fp16, exactly, or times 0 (kPlain: it is not).  int8: the factor
// comes as a pair of fp16, e4m3: as fp32.
template <int kHeld, bool kPlain>
__device__ __forceinline__ u32x2v shifted_codes(uint32_t w, uint32_t by) {
    if constexpr (kHeld == kI8Pages) {
        // 1,024 + 128 + the code by its bits, times the factor, less 1,152 of it: each exact
        const _Float16 off = static_cast<_Float16>(-1152.0f);
        const f16x2v f = __builtin_bit_cast(f16x2v, by), less = f * f16x2v{off, off};
        const uint32_t u = w ^ 0x80808080u;
        const f16x2v a = __builtin_bit_cast(f16x2v, __builtin_amdgcn_perm(u, 0x64646464u, 0x00050004u));
        const f16x2v b = __builtin_bit_cast(f16x2v, __builtin_amdgcn_perm(u, 0x64646464u, 0x00070006u));
        return u32x2v{__builtin_bit_cast(uint32_t, __builtin_elementwise_fma(a, f, less)),
                      __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(b, f, less))};
    }
    const float x = __builtin_bit_cast(float, by);
    if constexpr (kPlain)
        return u32x2v{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, x, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, x, true))};
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
    return u32x2v{F16::pack(lo[0] * x, lo[1] * x), F16::pack(hi[0] * x, hi[1] * x)};
}

// The larger, and the sum, of a lane's value and that of the lane 16 (32) away.
__device__ __forceinline__ f32x2v swap16(float x) {
    const uint32_t w = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return f32x2v{__builtin_bit_cast(float, static_cast<uint32_t>(r[0])), __builtin_bit_cast(float, static_cast<uint32_t>(r[1]))};
}
__device__ __forceinline__ f32x2v swap32(float x) {
    const uint32_t w = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return f32x2v{__builtin_bit_cast(float, static_cast<uint32_t>(r[0])), __builtin_bit_cast(float, static_cast<uint32_t>(r[1]))};
}
__device__ __forceinline__ float max16(float x) {
    const f32x2v r = swap16(x);
    return fmaxf(r[0], r[1]);
}
__device__ __forceinline__ float max32(float x) {
    const f32x2v r = swap32(x);
    return fmaxf(r[0], r[1]);
}
__device__ __forceinline__ float sum16(float x) {
    const f32x2v r = swap16(x);
    return r[0] + r[1];
}
__device__ __forceinline__ float sum32(float x) {
    const f32x2v r = swap32(x);
    return r[0] + r[1];
}

// The paged cache as the kernels see it: K and V each [n_pages][n_kv_heads]
// [page][dim], page p starting at p * page_stride elements; a cache of codes
// also has one fp32 scale for each (page, head, slot) or for each (page, head).
// page is 2^page_shift.
struct CacheView {
    uint8_t* k;
    uint8_t* v;
    float* k_scale;
    float* v_scale;
    int64_t k_page_stride;
    int64_t v_page_stride;
    int64_t n_pages;
    uint32_t n_kv_heads;
    uint32_t page_shift;
};

struct NormRopeArgs {
    const uint8_t* src[2];  // q and k
    uint8_t* dst[2];
    const uint8_t* weight[2];  // nullptr: no norm
    int64_t src_tok[2], src_head[2], dst_tok[2], dst_head[2];  // strides, elements
    uint32_t heads[2];
    const int32_t* positions;
    const double* inv_freq;
    uint32_t n_tok;
    uint32_t rotary;
    uint32_t interleaved;
    float eps;
};

struct AppendArgs {
    const uint8_t* src[2];  // k and v
    int64_t src_tok[2], src_head[2];
    const uint8_t* weight;
    const int32_t* positions;
    const double* inv_freq;
    const int64_t* slots;
    CacheView cache;
    uint32_t n_tok;
    uint32_t rotary;
    uint32_t interleaved;
    float eps;
};

// As AppendArgs, to pages with one scale each: the tokens of a request are the last of its kv_len keys.
struct AppendPagesArgs {
    const uint8_t* src[2];  // k and v
    int64_t src_tok[2], src_head[2];
    const uint8_t* weight;
    const int32_t* positions;
    const double* inv_freq;
    const int32_t* table;   // [n_seq][table_width], row stride table_stride
    const int32_t* kv_len;  // [n_seq]
    const int32_t* cu_q;    // [n_seq + 1], or nullptr: uniform_q tokens each
    CacheView cache;
    int64_t table_stride;
    uint32_t table_width;
    uint32_t n_seq, n_tok;
    uint32_t uniform_q;
    uint32_t most_q;        // tokens of a request at most; 0: not known
    uint32_t pages_per;     // pages set aside for each request; 0: as the lengths need
    uint32_t rotary;
    uint32_t interleaved;
    float eps;
};

// Heads of one side that a workgroup of chunks takes.  The cosines of a page's tokens are made once for up to 16 heads; where
// pages are few or nothing is turned, for 4, on more workgroups (8 heads of 128: a prompt of 32,768 tokens on pages of 16 48.0
// us with all heads together and 51.9 with 4, of 64 50.1 and 52.7, of 16 without rotation 47.1 and 44.8; 64 runs of 6 tokens
// 5.9 and 4.6).
inline uint32_t append_heads(uint64_t pages, uint32_t heads, bool turned) {
    return turned && pages * ((heads + 15u) / 16u) >= 512u ? 16u : 4u;
}
hipError_t launch_append_pages(const AppendPagesArgs& a, uint32_t dim, uint32_t type, bool int8, hipStream_t stream);
hipError_t launch_norm_rope(const NormRopeArgs& a, uint32_t dim, uint32_t type, hipStream_t stream);
hipError_t launch_append(const AppendArgs& a, uint32_t dim, uint32_t type, bool e4m3, hipStream_t stream);

}  // namespace engram
