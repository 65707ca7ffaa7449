// Paged attention: the splits of a row joined, in their order.
//
//     M = max_s m_s,  l = sum_s 2^(m_s - M) l_s,  o = sum_s 2^(m_s - M) o_s / l
//
// Each part is read once.  kPer waves take a row: the maximum and sum first,
// with a split in each lane, then the parts, which wait for nothing but their
// weights, so that a wave has several in flight.
#include <algorithm>
#include <type_traits>

#include "paged_attention.h"

namespace engram {
namespace {

// kTile, kAlign: of the kernel that wrote the parts.
template <class T, int D, bool kE4m3, uint32_t kTile, int32_t kAlign, uint32_t kPer, uint32_t kWaves>
__global__ __launch_bounds__(kWaves * 64) void paged_join_kernel(const AttentionArgs A) {
    constexpr int E = D / 64;  // channels of a lane
    constexpr uint32_t kRowsOf = kWaves / kPer;
    using P = std::conditional_t<kE4m3, Bf16, T>;
    __shared__ float sm_o[kPer > 1 ? kWaves : 1][D];
    const uint32_t heads = A.cache.n_kv_heads;
    const uint32_t tile_at = blockIdx.x / heads, h = blockIdx.x - tile_at * heads;
    const Tile tile = find_tile<kTile>(A, tile_at);
    if (!tile.live) return;
    const Request req = request_of(A, tile.b);
    const uint32_t rows = req.q_len * A.group;
    if (tile.row0 >= rows || rows < A.min_rows || rows > A.max_rows) return;
    const uint32_t n_rows = min(kTile, rows - tile.row0);
    const Span span = span_of(A, req, tile.row0, n_rows);
    const int32_t base0 = span.lo & ~(kAlign - 1);
    if (span.hi <= base0 || static_cast<uint32_t>(span.hi - base0) <= A.split_tokens) return;  // written whole
    const uint32_t n_split = (static_cast<uint32_t>(span.hi - base0) + A.split_tokens - 1u) / A.split_tokens;

    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u;
    const uint32_t of_tile = blockIdx.y * kRowsOf + wave / kPer, part = wave % kPer;
    const bool live = of_tile < n_rows;
    const uint32_t row = tile.row0 + min(of_tile, n_rows - 1u);
    const uint32_t tok = req.q0 + row / A.group, head = h * A.group + row % A.group;
    const uint64_t flat = static_cast<uint64_t>(tok) * (heads * A.group) + head;
    const uint64_t first = part_index(A, 0, tile.b, h, row, flat), step = part_index(A, 1, tile.b, h, row, flat) - first;

    float top = -INFINITY;
    for (uint32_t s = lane; s < n_split; s += 64u) top = fmaxf(top, A.part_ml[(first + s * step) * 2]);
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) top = fmaxf(top, __shfl_xor(top, k));
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    for (uint32_t s = lane; s < n_split; s += 64u) {
        const f32x2v ml = *reinterpret_cast<const f32x2v*>(A.part_ml + (first + s * step) * 2);
        sum += __builtin_amdgcn_exp2f(ml[0] - ref) * ml[1];
    }
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) sum += __shfl_xor(sum, k);

    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll 4
    for (uint32_t s = part; s < n_split; s += kPer) {
        const uint64_t at = first + s * step;
        const float f = __builtin_amdgcn_exp2f(A.part_ml[at * 2] - ref);
        const float* src = A.part_o + at * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += f * src[e];
    }
    if constexpr (kPer > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) sm_o[wave][lane * E + e] = acc[e];
        __syncthreads();
        if (part != 0) return;
#pragma unroll
        for (uint32_t w = 1; w < kPer; ++w)
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] += sm_o[wave + w][lane * E + e];
    }
    if (!live) return;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t* dst = reinterpret_cast<uint16_t*>(A.out) + tok * A.out_tok + head * A.out_head + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = static_cast<uint16_t>(T::pack(acc[e] * inv, 0.0f));
    if (A.lse && lane == 0) A.lse[flat] = sum == 0.0f ? -INFINITY : (top + __log2f(sum) - P::kShift) * 0.69314718055994531f;
}

template <class T, int D, bool kE4m3, uint32_t kTile, int32_t kAlign, uint32_t kPer, uint32_t kWaves>
hipError_t join_one(const AttentionArgs& a, hipStream_t stream) {
    constexpr uint32_t kRowsOf = kWaves / kPer;
    uint32_t most = kTile;  // rows of a tile
    if (!a.cu_q) most = std::min(most, a.uniform_q * a.group);
    most = std::min(most, a.max_rows);
    const dim3 grid(tile_count<kTile>(a) * a.cache.n_kv_heads, (most + kRowsOf - 1u) / kRowsOf);
    hipLaunchKernelGGL((paged_join_kernel<T, D, kE4m3, kTile, kAlign, kPer, kWaves>), grid, dim3(kWaves * 64), 0, stream, a);
    return hipGetLastError();
}

template <class T, int D, bool kE4m3>
hipError_t join_dim(const AttentionArgs& a, bool many, hipStream_t stream) {
    if (many) return join_one<T, D, kE4m3, kTileRows, kTileAlign, 1, 4>(a, stream);
    if (a.n_split <= 32) return join_one<T, D, kE4m3, kRowsTile, kRowsAlign, 4, 4>(a, stream);
    return join_one<T, D, kE4m3, kRowsTile, kRowsAlign, 16, 16>(a, stream);
}

template <class T, bool kE4m3>
hipError_t join_type(const AttentionArgs& a, uint32_t dim, bool many, hipStream_t stream) {
    switch (dim) {
        case 64: return join_dim<T, 64, kE4m3>(a, many, stream);
        case 128: return join_dim<T, 128, kE4m3>(a, many, stream);
        default: return join_dim<T, 256, kE4m3>(a, many, stream);
    }
}

}  // namespace

hipError_t launch_paged_join(const AttentionArgs& a, uint32_t dim, uint32_t type, bool e4m3, bool many, hipStream_t stream) {
    if (type == ENGRAM_BF16)
        return e4m3 ? join_type<Bf16, true>(a, dim, many, stream) : join_type<Bf16, false>(a, dim, many, stream);
    return e4m3 ? join_type<F16, true>(a, dim, many, stream) : join_type<F16, false>(a, dim, many, stream);
}

}  // namespace engram
