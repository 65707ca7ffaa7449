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
    // fp16 ends at 65,504 and has all its digits down to 2^-14: with a term of
    // 2^14 at most, one of 2^-21 of the reference is still a normal number.
    static constexpr float kShift = 7.0f, kSlack = 7.0f;
};

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
// [page][dim], page p starting at p * page_stride elements; an e4m3 cache
// also has one fp32 scale for each (page, head, slot).  page is 2^page_shift.
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

hipError_t launch_norm_rope(const NormRopeArgs& a, uint32_t dim, uint32_t type, hipStream_t stream);
hipError_t launch_append(const AppendArgs& a, uint32_t dim, uint32_t type, bool e4m3, hipStream_t stream);

}  // namespace engram
