// Head norm, rotation by position, and the append into a paged cache.
//
// A head row x of dim D (one token, one head):
//     y_j = x_j * rsqrt(sum_j x_j^2 / D + eps) * w_j           (w given)
//     (y_a, y_b) -> (y_a cos t - y_b sin t, y_a sin t + y_b cos t)
// for the R/2 pairs (a, b) of the first R elements, t = position *
// inv_freq[pair]; pairs are (i, i + R/2), or (2i, 2i + 1) when interleaved.
// Everything is fp32 and rounded once at the store, but for the angle, its
// reduction to a quarter turn and the series of its cosine and sine, which are
// fp64: both are the fp32 numbers nearest to the true ones (but for 1e-10 of
// them) at any position.  In fp32 the product alone would be off by 0.03 rad at
// a position of a million, and the reduced angle by up to 9e-8 at any.
//
// The kernels read each row once and write it once: HBM-bound for prompts (32,768
// tokens of 32 + 8 heads of 128: 132 us, 5.1 TB/s, where a copy of 2 GiB reaches
// 4.8 to 4.9), launch-bound for single tokens (2.8 us of kernel).
//
// Mapping: D/16 lanes hold a row (16 elements each), so a wave holds 16 to 4
// rows of one token.  A rotating lane takes the 8-element blocks j and
// j + R/16: in the half form both elements of a pair are then in one lane and
// no lane exchanges anything but the norm's sum (2 to 4 cross-lane adds); in
// the interleaved form each block holds its own pairs.  Either way a lane
// needs 8 cosines and sines, computed once and used for every row that the
// wave takes of its token.
#include <algorithm>

#include "head_rows.h"

namespace engram {
namespace {

// The cosines and sines of a token's `pairs` pairs, one or two to a lane, by
// way of LDS to the lanes that use them (lane j of each row 8 of them): a wave
// computes each once, not once for each of its rows.  cs: this wave's.
template <int D>
__device__ __forceinline__ Turn load_turn(const double* __restrict__ inv_freq, int32_t pos, uint32_t j, uint32_t rb,
                                          bool interleaved, f32x2v* cs) {
    const uint32_t lane = threadIdx.x & 63u, pairs = 8u * rb;
#pragma unroll
    for (uint32_t i = 0; i < (D / 2 + 63) / 64; ++i) {
        const uint32_t at = i * 64u + lane;
        if (at < pairs) cs[at] = cos_sin(static_cast<double>(pos) * inv_freq[at]);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    return turn_of(cs, j, rb, interleaved);
}

template <class T, int D>
__global__ __launch_bounds__(256) void norm_rope_kernel(const NormRopeArgs A, uint32_t tok_base,
                                                        uint32_t tok_end, uint32_t chunks, uint32_t iters) {
    constexpr int LPH = D / 16, RPW = 64 / LPH;
    __shared__ f32x2v sm_cs[4][D / 2];
    const uint32_t item = blockIdx.x * 4u + (threadIdx.x >> 6);
    const uint32_t of_launch = item / chunks, chunk = item - of_launch * chunks;
    const uint32_t tok = tok_base + of_launch;
    if (tok >= tok_end) return;
    const uint32_t lane = threadIdx.x & 63u, j = lane & (LPH - 1u);
    const uint32_t rb = A.rotary / 16u;
    const bool il = A.interleaved != 0, turns = j < rb;
    const Blocks b = blocks_of(j, rb);
    const uint32_t total = A.heads[0] + A.heads[1];
    // a row is asked for before the cosines are made, or the row before it is done
    u32x4v next[2];
    const auto ask = [&](uint32_t it) {
        const uint32_t row = (chunk * iters + it) * RPW + lane / LPH;
        next[0] = next[1] = u32x4v{0u, 0u, 0u, 0u};
        if (row >= total) return;
        const uint32_t which = row < A.heads[0] ? 0u : 1u, head = which ? row - A.heads[0] : row;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(which ? A.src[1] : A.src[0]) +
                              tok * (which ? A.src_tok[1] : A.src_tok[0]) +
                              head * (which ? A.src_head[1] : A.src_head[0]);
        next[0] = *reinterpret_cast<const u32x4v*>(src + b.b0 * 8u);
        next[1] = *reinterpret_cast<const u32x4v*>(src + b.b1 * 8u);
    };
    ask(0);
    Turn t;
    if (rb) t = load_turn<D>(A.inv_freq, A.positions[tok], j, rb, il, sm_cs[threadIdx.x >> 6]);
    for (uint32_t it = 0; it < iters; ++it) {
        const uint32_t row = (chunk * iters + it) * RPW + lane / LPH;
        const bool live = row < total;
        const uint32_t which = row < A.heads[0] ? 0u : 1u;
        const uint32_t head = which ? row - A.heads[0] : row;
        float x[16];
        unpack8<T>(next[0], x);
        unpack8<T>(next[1], x + 8);
        if (it + 1 < iters) ask(it + 1);
        const uint16_t* wp = reinterpret_cast<const uint16_t*>(which ? A.weight[1] : A.weight[0]);
        if (wp) {  // the same for all lanes of a row
            float w[16];
            unpack8<T>(*reinterpret_cast<const u32x4v*>(wp + b.b0 * 8u), w);
            unpack8<T>(*reinterpret_cast<const u32x4v*>(wp + b.b1 * 8u), w + 8);
            norm_row<LPH>(x, w, A.eps);
        }
        if (turns) turn_row(x, t, il);
        if (live) {
            uint16_t* dst = reinterpret_cast<uint16_t*>(which ? A.dst[1] : A.dst[0]) +
                            tok * (which ? A.dst_tok[1] : A.dst_tok[0]) + head * (which ? A.dst_head[1] : A.dst_head[0]);
            *reinterpret_cast<u32x4v*>(dst + b.b0 * 8u) = pack8<T>(x);
            *reinterpret_cast<u32x4v*>(dst + b.b1 * 8u) = pack8<T>(x + 8);
        }
    }
}

// The divisor of a row's codes, and its reciprocal.
struct Divisor {
    float unit, d, r;
};
__device__ __forceinline__ Divisor divisor_of(float amax) {
    Divisor v;
    // keep x * 448 finite and the reciprocal too: a power of two taken from both changes nothing
    v.unit = amax >= 0x1p100f ? 0x1p-64f : amax < 0x1p-60f ? 0x1p64f : 1.0f;
    v.d = amax == 0.0f ? 1.0f : amax * v.unit;
    v.r = 1.0f / v.d;
    return v;
}

// Eight e4m3 codes of x * 448 / amax, nearest even.  x * 448 is exact where x
// is a 16-bit number (448 = 7 * 2^6): values, and what of a key is neither
// normed nor turned.  For other keys, fp32 numbers, it is one fp32 rounding
// more, which moves a code in 10^6 next to a tie, as those before it do.  A
// product with the reciprocal, put right by its remainder (exact in one fused
// step), is the quotient wherever that is an fp32 number, so that one half-way
// between two codes is seen as such.  A third of the instructions of 8
// divisions.
__device__ __forceinline__ u32x2v encode8(const float* x, const Divisor& v) {
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float y = (x[e] * v.unit) * 448.0f, a = y * v.r;
        q[e] = __builtin_fmaf(__builtin_fmaf(-a, v.d, y), v.r, a);
    }
    u32x2v w;
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    w[0] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true));
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
    w[1] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true));
    return w;
}

template <class T, int D, bool kE4m3>
__global__ __launch_bounds__(256) void append_kernel(const AppendArgs A, uint32_t tok_base,
                                                     uint32_t tok_end, uint32_t chunks, uint32_t iters) {
    constexpr int LPH = D / 16, RPW = 64 / LPH;
    __shared__ f32x2v sm_cs[4][D / 2];
    const uint32_t item = blockIdx.x * 4u + (threadIdx.x >> 6);
    const uint32_t of_launch = item / chunks, chunk = item - of_launch * chunks;
    const uint32_t tok = tok_base + of_launch;
    if (tok >= tok_end) return;
    const int64_t slot = A.slots[tok];
    const uint32_t lane = threadIdx.x & 63u, j = lane & (LPH - 1u);
    const uint32_t rb = A.rotary / 16u;
    const bool il = A.interleaved != 0, turns = j < rb;
    const Blocks b = blocks_of(j, rb);
    const uint32_t heads = A.cache.n_kv_heads, total = 2u * heads;
    u32x4v next[2];
    const auto ask = [&](uint32_t it) {
        const uint32_t row = (chunk * iters + it) * RPW + lane / LPH;
        next[0] = next[1] = u32x4v{0u, 0u, 0u, 0u};
        if (row >= total) return;
        const uint32_t which = row < heads ? 0u : 1u, head = which ? row - heads : row;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(which ? A.src[1] : A.src[0]) +
                              tok * (which ? A.src_tok[1] : A.src_tok[0]) +
                              head * (which ? A.src_head[1] : A.src_head[0]);
        next[0] = *reinterpret_cast<const u32x4v*>(src + b.b0 * 8u);
        next[1] = *reinterpret_cast<const u32x4v*>(src + b.b1 * 8u);
    };
    // A row is asked for before its token's place is known and the cosines are
    // made, or the row before it is done.  Codes take more registers: there a
    // row in flight costs a wave of each SIMD (9.4 us for 8.4 at 8,191 tokens
    // of 4 heads of 128 with it), so that it is asked for in its turn.
    if (!kE4m3) ask(0);
    // padding (negative) and slots past the pool are skipped
    if (slot < 0 || (slot >> A.cache.page_shift) >= A.cache.n_pages) return;
    const int64_t page = slot >> A.cache.page_shift;
    const uint32_t at = static_cast<uint32_t>(slot) & ((1u << A.cache.page_shift) - 1u);
    Turn t;
    if (rb) t = load_turn<D>(A.inv_freq, A.positions[tok], j, rb, il, sm_cs[threadIdx.x >> 6]);
    float w[16];
    if (A.weight) {
        const uint16_t* wp = reinterpret_cast<const uint16_t*>(A.weight);
        unpack8<T>(*reinterpret_cast<const u32x4v*>(wp + b.b0 * 8u), w);
        unpack8<T>(*reinterpret_cast<const u32x4v*>(wp + b.b1 * 8u), w + 8);
    }
    for (uint32_t it = 0; it < iters; ++it) {
        const uint32_t row = (chunk * iters + it) * RPW + lane / LPH;
        const bool live = row < total;
        const uint32_t which = row < heads ? 0u : 1u;
        const uint32_t head = which ? row - heads : row;
        if (kE4m3) ask(it);
        u32x4v r0 = next[0], r1 = next[1];
        if (!kE4m3 && it + 1 < iters) ask(it + 1);
        float x[16];
        unpack8<T>(r0, x);
        unpack8<T>(r1, x + 8);
        if (which == 0) {  // the same for all lanes of a row; a value row keeps its bits
            if (A.weight) norm_row<LPH>(x, w, A.eps);
            if (turns) turn_row(x, t, il);
            if (!kE4m3) {
                r0 = pack8<T>(x);
                r1 = pack8<T>(x + 8);
            }
        }
        const int64_t line = (static_cast<int64_t>(head) << A.cache.page_shift) + at;  // of the page's rows
        if (kE4m3) {
            // the largest magnitude by its bits, so that a NaN is the largest of all and reaches the scale
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) m = max(m, __builtin_bit_cast(uint32_t, x[e]) & 0x7FFFFFFFu);
#pragma unroll
            for (int k = 1; k < LPH; k <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), k)));
            const float amax = __builtin_bit_cast(float, m);
            const Divisor by = divisor_of(amax);
            if (live) {
                uint8_t* dst = (which ? A.cache.v + page * A.cache.v_page_stride : A.cache.k + page * A.cache.k_page_stride) +
                               line * D;
                *reinterpret_cast<u32x2v*>(dst + b.b0 * 8u) = encode8(x, by);
                *reinterpret_cast<u32x2v*>(dst + b.b1 * 8u) = encode8(x + 8, by);
                if (j == 0) {
                    float* sc = which ? A.cache.v_scale : A.cache.k_scale;
                    sc[((page * heads) << A.cache.page_shift) + line] = amax / 448.0f;
                }
            }
        } else if (live) {
            uint16_t* dst = reinterpret_cast<uint16_t*>(which ? A.cache.v : A.cache.k) +
                            page * (which ? A.cache.v_page_stride : A.cache.k_page_stride) + line * D;
            *reinterpret_cast<u32x4v*>(dst + b.b0 * 8u) = r0;
            *reinterpret_cast<u32x4v*>(dst + b.b1 * 8u) = r1;
        }
    }
}

// Tokens per launch from which a wave takes all rows of its token (the
// cosines are then computed once per token); below it each wave takes one step
// of rows, so that a few tokens still spread over the chip.
constexpr uint32_t kManyTokens = 2048;

// kernel(args, tok_base, tok_end, chunks, iters) over all tokens; a launch
// has at most 2^24 waves, so that its grid stays below 2^32 threads.
template <class Args>
hipError_t launch_rows(void (*kernel)(const Args, uint32_t, uint32_t, uint32_t, uint32_t), const Args& a, uint32_t rows,
                       uint32_t rows_per_wave, hipStream_t stream) {
    const uint32_t steps = (rows + rows_per_wave - 1u) / rows_per_wave;
    const uint32_t iters = a.n_tok >= kManyTokens ? steps : 1u;
    const uint32_t chunks = (steps + iters - 1u) / iters;
    const uint32_t most = std::max((1u << 24) / chunks, 1u);
    for (uint64_t base = 0; base < a.n_tok; base += most) {
        const uint32_t n = static_cast<uint32_t>(std::min<uint64_t>(most, a.n_tok - base));
        hipLaunchKernelGGL(kernel, dim3((n * chunks + 3u) / 4u), dim3(256), 0, stream, a, static_cast<uint32_t>(base),
                           static_cast<uint32_t>(base) + n, chunks, iters);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class T, int D>
hipError_t norm_rope_one(const NormRopeArgs& a, hipStream_t stream) {
    return launch_rows<NormRopeArgs>(norm_rope_kernel<T, D>, a, a.heads[0] + a.heads[1], 1024 / D, stream);
}

template <class T, int D, bool kE4m3>
hipError_t append_one(const AppendArgs& a, hipStream_t stream) {
    return launch_rows<AppendArgs>(append_kernel<T, D, kE4m3>, a, 2u * a.cache.n_kv_heads, 1024 / D, stream);
}

template <class T>
hipError_t norm_rope_dim(const NormRopeArgs& a, uint32_t dim, hipStream_t stream) {
    switch (dim) {
        case 64: return norm_rope_one<T, 64>(a, stream);
        case 128: return norm_rope_one<T, 128>(a, stream);
        default: return norm_rope_one<T, 256>(a, stream);
    }
}

template <class T, bool kE4m3>
hipError_t append_dim(const AppendArgs& a, uint32_t dim, hipStream_t stream) {
    switch (dim) {
        case 64: return append_one<T, 64, kE4m3>(a, stream);
        case 128: return append_one<T, 128, kE4m3>(a, stream);
        default: return append_one<T, 256, kE4m3>(a, stream);
    }
}

}  // namespace

hipError_t launch_norm_rope(const NormRopeArgs& a, uint32_t dim, uint32_t type, hipStream_t stream) {
    return type == ENGRAM_BF16 ? norm_rope_dim<Bf16>(a, dim, stream) : norm_rope_dim<F16>(a, dim, stream);
}

hipError_t launch_append(const AppendArgs& a, uint32_t dim, uint32_t type, bool e4m3, hipStream_t stream) {
    if (type == ENGRAM_BF16)
        return e4m3 ? append_dim<Bf16, true>(a, dim, stream) : append_dim<Bf16, false>(a, dim, stream);
    return e4m3 ? append_dim<F16, true>(a, dim, stream) : append_dim<F16, false>(a, dim, stream);
}

}  // namespace engram
