// Rows of heads in registers: a row's elements over its lanes, RMS norm and
// rotation (norm_rope.hip has the formulas and the mapping).
#pragma once

#include "serving.h"

namespace engram {
namespace {

// Cosine and sine of t, rounded once: t = k pi/2 + r with |r| <= pi/4 (pi/2 in two parts: its first 53 bits and the rest,
// so that k of 2^33 loses nothing), then the series of r, whose next terms are below 4e-13 and 9e-12 of the value.
__device__ __forceinline__ f32x2v cos_sin(double t) {
    const double k = __builtin_rint(t * 0.63661977236758134308);
    const double r = __builtin_fma(-k, 6.12323399573676588613e-17, __builtin_fma(-k, 1.57079632679489661923, t)), z = r * r;
    double c = 1.0 / 479001600, s = -1.0 / 39916800;
    c = __builtin_fma(c, z, -1.0 / 3628800);
    s = __builtin_fma(s, z, 1.0 / 362880);
    c = __builtin_fma(c, z, 1.0 / 40320);
    s = __builtin_fma(s, z, -1.0 / 5040);
    c = __builtin_fma(c, z, -1.0 / 720);
    s = __builtin_fma(s, z, 1.0 / 120);
    c = __builtin_fma(c, z, 1.0 / 24);
    s = __builtin_fma(s, z, -1.0 / 6);
    c = __builtin_fma(c, z, -0.5);
    c = __builtin_fma(c, z, 1.0);
    s = __builtin_fma(s * z, r, r);
    const float cf = static_cast<float>(c), sf = static_cast<float>(s);
    // k mod 4 quarter turns on
    const uint32_t quarter = static_cast<uint32_t>(static_cast<int32_t>(k - 4.0 * __builtin_floor(k * 0.25)));
    const float a = quarter & 1u ? sf : cf, b = quarter & 1u ? cf : sf;
    const uint32_t flip_a = ((quarter + 1u) & 2u) << 30, flip_b = (quarter & 2u) << 30;
    return f32x2v{__builtin_bit_cast(float, __builtin_bit_cast(uint32_t, a) ^ flip_a),
                  __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, b) ^ flip_b)};
}

struct Turn {
    float c[8], s[8];  // of block 0's pairs, then (interleaved) block 1's
};

// Those of lane j of a row, from its token's pairs.
__device__ __forceinline__ Turn turn_of(const f32x2v* cs, uint32_t j, uint32_t rb, bool interleaved) {
    Turn t;
    if (j < rb) {
#pragma unroll
        for (uint32_t e = 0; e < 8; ++e) {
            const f32x2v x = cs[interleaved ? (e < 4 ? 4u * j + e : 4u * (j + rb) + (e - 4)) : 8u * j + e];
            t.c[e] = x[0];
            t.s[e] = x[1];
        }
    }
    return t;
}

template <class T>
__device__ __forceinline__ void unpack8(u32x4v w, float* x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = T::lo(w[i]);
        x[2 * i + 1] = T::hi(w[i]);
    }
}

template <class T>
__device__ __forceinline__ u32x4v pack8(const float* x) {
    u32x4v w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = T::pack(x[2 * i], x[2 * i + 1]);
    return w;
}

// Norm over the row's LPH lanes; x: blocks 0 and 1 of this lane.
template <int LPH>
__device__ __forceinline__ void norm_row(float* x, const float* w, float eps) {
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = __builtin_fmaf(x[e], x[e], ss);
#pragma unroll
    for (int m = 1; m < LPH; m <<= 1) ss += __shfl_xor(ss, m);
    const float r = 1.0f / __builtin_sqrtf(ss * (1.0f / (16 * LPH)) + eps);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = x[e] * r * w[e];
}

__device__ __forceinline__ void turn_row(float* x, const Turn& t, bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = x[2 * e], b = x[2 * e + 1];
            x[2 * e] = a * t.c[e] - b * t.s[e];
            x[2 * e + 1] = a * t.s[e] + b * t.c[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = x[e], b = x[8 + e];
            x[e] = a * t.c[e] - b * t.s[e];
            x[8 + e] = a * t.s[e] + b * t.c[e];
        }
    }
}

// The two 8-element blocks of lane j of a row (rb = R/16 lanes rotate).
struct Blocks {
    uint32_t b0, b1;
};
__device__ __forceinline__ Blocks blocks_of(uint32_t j, uint32_t rb) {
    return j < rb ? Blocks{j, j + rb} : Blocks{2u * j, 2u * j + 1u};
}

}  // namespace
}  // namespace engram
