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
// Prompts: each row is read once and its codes are written once: HBM-bound.
// Single tokens: launch-bound, and the page is touched only where its scale
// grows.
//
// Mapping: as in norm_rope.hip D/16 lanes hold a row of 16 elements each.
//   * Chunks: a workgroup takes one page of one request and up to 16 (head,
//     side) pairs of it, a pair to a wave in turn, so that the cosines of the
//     page's tokens are made once for all its heads (by way of LDS).  A wave
//     holds 64 rows of head_dim 64 or 128 (32 of 256) as they were read, finds
//     their maximum, and turns and rounds them from the same registers; pages
//     with more new rows are read twice.
//   * Single tokens: a wave takes as many pairs of a token as it holds rows.
#include <algorithm>

#include "head_rows.h"

namespace engram {
namespace {

constexpr uint32_t kMagnitude = 0x7FFFFFFFu, kInfinite = 0x7F800000u;

// The two kinds of codes.
struct CodeE4m3 {
    // |x| <= largest = 1.75 * 2^8
    static constexpr uint32_t kMantissa = 0x600000u, kExponent = 8u;
    static __device__ __forceinline__ uint32_t four(const float* x, float by) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * by, x[1] * by, 0, false);
        return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(x[2] * by, x[3] * by, lo, true));
    }
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
    // a NaN on either side stays
    s.now = held ? (need > old || need != need ? need : old) : need;
    s.by = s.now == 0.0f ? 0.0f : 1.0f / s.now;
    s.ratio = held && s.now > old ? old * s.by : 1.0f;
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
        w[i] = C::four(x, ratio);
    }
    return w;
}

__device__ __forceinline__ uint32_t largest16(const float* x) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = max(m, __builtin_bit_cast(uint32_t, x[e]) & kMagnitude);
    return m;
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

template <class T, int D, class C>
__global__ __launch_bounds__(256) void append_pages_kernel(const AppendPagesArgs A) {
    constexpr int LPH = D / 16;
    constexpr uint32_t RPW = 64 / LPH, kSteps = D == 64 ? 4 : 8, kHold = kSteps * RPW;  // rows of a step, steps, rows held
    constexpr uint32_t kPairs = 16;  // (head, side) pairs of a workgroup
    __shared__ f32x2v sm_cs[kHold * (D / 2)];
    __shared__ uint32_t sm_most[kPairs];
    const uint32_t tid = threadIdx.x, lane = tid & 63u, j = lane & (LPH - 1u), of_step = lane / LPH;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
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
    // rows row0 .. row0 + n_rows - 1 of the page are new; in_table <= 2^31 / page, so that its keys are int32 but for the end
    const uint32_t key0 = in_table << shift;
    const uint32_t row0 = max(static_cast<uint32_t>(lo), key0) - key0;
    const uint32_t n_rows = min(static_cast<uint32_t>(req.kv_len) - key0, 1u << shift) - row0;
    const uint32_t tok0 = req.q0 + (key0 + row0 - static_cast<uint32_t>(req.first));

    const uint32_t rb = A.rotary / 16u, heads = A.cache.n_kv_heads;
    const uint32_t pair0 = blockIdx.y * kPairs, n_pairs = min(2u * heads - pair0, kPairs);
    const bool il = A.interleaved != 0, turns = j < rb, any_key = pair0 < heads;
    const Blocks bl = blocks_of(j, rb);
    float weight[16];
    if (A.weight && any_key) {
        const uint16_t* wp = reinterpret_cast<const uint16_t*>(A.weight);
        unpack8<T>(*reinterpret_cast<const u32x4v*>(wp + bl.b0 * 8u), weight);
        unpack8<T>(*reinterpret_cast<const u32x4v*>(wp + bl.b1 * 8u), weight + 8);
    }
    struct Held {
        u32x4v w[kSteps][2];
    };
    const auto load = [&](uint32_t pair, uint32_t r0) {
        Held h;
        const uint32_t side = pair < heads ? 0u : 1u, head = side ? pair - heads : pair;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(side ? A.src[1] : A.src[0]) +
                              head * (side ? A.src_head[1] : A.src_head[0]);
        const int64_t stride = side ? A.src_tok[1] : A.src_tok[0];
#pragma unroll
        for (uint32_t s = 0; s < kSteps; ++s) {
            if (r0 + s * RPW < n_rows) {  // the last row again, where a step is not full
                const uint16_t* p = src + (tok0 + min(r0 + s * RPW + of_step, n_rows - 1u)) * stride;
                h.w[s][0] = *reinterpret_cast<const u32x4v*>(p + bl.b0 * 8u);
                h.w[s][1] = *reinterpret_cast<const u32x4v*>(p + bl.b1 * 8u);
            }
        }
        return h;
    };
    // the row of step s as it is to be stored
    const auto row_of = [&](const Held& h, uint32_t pair, uint32_t s, uint32_t r0, float* x) __attribute__((always_inline)) {
        unpack8<T>(h.w[s][0], x);
        unpack8<T>(h.w[s][1], x + 8);
        if (pair < heads) {
            if (A.weight) norm_row<LPH>(x, weight, A.eps);
            const uint32_t row = min(s * RPW + of_step, n_rows - 1u - r0);  // as it was loaded
            if (turns) turn_row(x, turn_of(sm_cs + row * (8u * rb), j, rb, il), il);
        }
    };
    const auto make_turns = [&](uint32_t r0) {
        if (!rb || !any_key) return;
        const uint32_t pairs = 8u * rb, n = min(n_rows - r0, kHold) * pairs;
        for (uint32_t i = tid; i < n; i += 256u) {
            const uint32_t row = i / pairs;
            sm_cs[i] = cos_sin(static_cast<double>(A.positions[tok0 + r0 + row]) * A.inv_freq[i - row * pairs]);
        }
    };
    const auto largest = [&](const Held& h, uint32_t pair, uint32_t r0) {
        uint32_t m = 0;
#pragma unroll
        for (uint32_t s = 0; s < kSteps; ++s) {
            if (r0 + s * RPW < n_rows) {
                float x[16];
                row_of(h, pair, s, r0, x);
                m = max(m, largest16(x));
            }
        }
        return m;
    };
    const auto finish = [&](uint32_t m) {
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), k)));
        return m;
    };
    // the page's scale and the codes that it holds
    const auto settle = [&](uint32_t pair, uint32_t m, float old) {
        const uint32_t side = pair < heads ? 0u : 1u, head = side ? pair - heads : pair;
        const Scale s = grown(scale_for<C>(m), old, row0 > 0u);
        if (lane == 0) (side ? A.cache.v_scale : A.cache.k_scale)[page * heads + head] = s.now;
        if (s.ratio != 1.0f) {
            uint8_t* const codes = (side ? A.cache.v + page * A.cache.v_page_stride : A.cache.k + page * A.cache.k_page_stride) +
                                   (static_cast<int64_t>(head) << shift) * D;
            for (uint32_t i = lane * 16u; i < row0 * D; i += 1024u) {
                u32x4v* const p = reinterpret_cast<u32x4v*>(codes + i);
                *p = again<C>(*p, s.ratio);
            }
        }
        return s.by;
    };
    const auto old_scale = [&](uint32_t pair) {
        return row0 ? (pair < heads ? A.cache.k_scale : A.cache.v_scale)[page * heads + (pair < heads ? pair : pair - heads)] : 0.0f;
    };
    const auto store = [&](const Held& h, uint32_t pair, uint32_t r0, float by) {
        const uint32_t side = pair < heads ? 0u : 1u, head = side ? pair - heads : pair;
        uint8_t* const codes = (side ? A.cache.v + page * A.cache.v_page_stride : A.cache.k + page * A.cache.k_page_stride) +
                               ((static_cast<int64_t>(head) << shift) + row0) * D;
#pragma unroll
        for (uint32_t s = 0; s < kSteps; ++s) {
            const uint32_t r = r0 + s * RPW + of_step;
            if (r0 + s * RPW < n_rows) {
                float x[16];
                row_of(h, pair, s, r0, x);
                if (r < n_rows) encode16<C>(codes + static_cast<uint64_t>(r) * D, x, by, bl);
            }
        }
    };
    if (n_rows <= kHold) {
        make_turns(0);
        __syncthreads();
        for (uint32_t k = wave; k < n_pairs; k += 4u) {
            const uint32_t pair = pair0 + k;
            const float old = old_scale(pair);
            const Held h = load(pair, 0);
            store(h, pair, 0, settle(pair, finish(largest(h, pair, 0)), old));
        }
        return;
    }
    if (tid < kPairs) sm_most[tid] = 0;
    for (uint32_t r0 = 0; r0 < n_rows; r0 += kHold) {
        __syncthreads();
        make_turns(r0);
        __syncthreads();
        for (uint32_t k = wave; k < n_pairs; k += 4u) {
            const uint32_t m = finish(largest(load(pair0 + k, r0), pair0 + k, r0));
            if (lane == 0) sm_most[k] = max(sm_most[k], m);  // the wave's own
        }
    }
    __syncthreads();
    for (uint32_t k = wave; k < n_pairs; k += 4u) {
        const float by = settle(pair0 + k, sm_most[k], old_scale(pair0 + k));
        if (lane == 0) sm_most[k] = __builtin_bit_cast(uint32_t, by);
    }
    for (uint32_t r0 = 0; r0 < n_rows; r0 += kHold) {
        __syncthreads();
        make_turns(r0);
        __syncthreads();
        for (uint32_t k = wave; k < n_pairs; k += 4u)
            store(load(pair0 + k, r0), pair0 + k, r0, __builtin_bit_cast(float, sm_most[k]));
    }
}

// One token a request: a wave takes RPW (head, side) pairs of it.
template <class T, int D, class C>
__global__ __launch_bounds__(256) void append_token_kernel(const AppendPagesArgs A, uint32_t steps) {
    constexpr int LPH = D / 16;
    constexpr uint32_t RPW = 64 / LPH;
    __shared__ f32x2v sm_cs[4][D / 2];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u, j = lane & (LPH - 1u);
    const uint32_t item = blockIdx.x * 4u + wave, b = item / steps;
    if (b >= A.n_seq) return;
    const Fresh req = fresh_of(A, b);
    if (req.q_len != 1u || req.kv_len == 0) return;
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
    const uint32_t key = static_cast<uint32_t>(req.kv_len - 1), place = key & ((1u << shift) - 1u);
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
            float w[16];
            const uint16_t* wp = reinterpret_cast<const uint16_t*>(A.weight);
            unpack8<T>(*reinterpret_cast<const u32x4v*>(wp + bl.b0 * 8u), w);
            unpack8<T>(*reinterpret_cast<const u32x4v*>(wp + bl.b1 * 8u), w + 8);
            norm_row<LPH>(x, w, A.eps);
        }
        if (j < rb) turn_row(x, turn_of(sm_cs[wave], j, rb, il), il);
    }
    uint32_t m = largest16(x);
#pragma unroll
    for (int k = 1; k < LPH; k <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), k)));
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
        hipLaunchKernelGGL((append_pages_kernel<T, D, C>), dim3(pages, (pairs + 15u) / 16u), dim3(256), 0, stream, a);
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
