// Paged attention: the splits of a row of paged_tile.hip joined, in their order.
//
//     R = max_s r_s,  l = sum_s 2^(r_s - R) l_s,  o = sum_s 2^(r_s - R) o_s / l
//
// A wave takes a row: the maximum and sum first, with a split in each lane,
// then the parts, which wait for nothing but their weights, so that the wave
// has several in flight.  Each part is read once: HBM-bound.
#include <algorithm>

#include "paged_attention.h"

namespace engram {
namespace {

constexpr uint32_t kWaves = 4;

template <class T, int D, uint32_t kRows>
__global__ __launch_bounds__(kWaves * 64) void paged_join_kernel(const AttentionArgs A) {
    constexpr int E = D / 64;  // channels of a lane
    const uint32_t heads = A.cache.n_kv_heads;
    const uint32_t tile_at = blockIdx.x / heads, h = blockIdx.x - tile_at * heads;
    const Tile tile = find_tile<kRows>(A, tile_at);
    if (!tile.live) return;
    const Request req = request_of(A, tile.b);
    const uint32_t rows = req.q_len * A.group;
    if (tile.row0 >= rows || rows < A.min_rows || rows > A.max_rows) return;
    const uint32_t n_rows = min(kRows, rows - tile.row0);
    const Span span = span_of(A, req, tile.row0, n_rows);
    const int32_t base0 = span.lo & ~(kTileAlign - 1);
    const uint32_t of_split = split_keys(A, req);
    if (span.hi <= base0 || static_cast<uint32_t>(span.hi - base0) <= of_split) return;  // written whole
    const uint32_t n_split = (static_cast<uint32_t>(span.hi - base0) + of_split - 1u) / of_split;

    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u;
    const uint32_t of_tile = blockIdx.y * kWaves + wave;
    if (of_tile >= n_rows) return;
    const uint32_t row = tile.row0 + of_tile;
    const uint32_t tok = req.q0 + row / A.group, head = h * A.group + row % A.group;
    const uint64_t flat = static_cast<uint64_t>(tok) * (heads * A.group) + head;
    const uint64_t step = static_cast<uint64_t>(A.n_tok) * (heads * A.group);

    const bool mine = lane < n_split;  // at most 32
    const f32x2v ml = *reinterpret_cast<const f32x2v*>(A.part_ml + (flat + (mine ? lane : 0u) * step) * 2);
    float top = mine ? ml[0] : -INFINITY;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) top = fmaxf(top, __shfl_xor(top, k));
    const float ref = top == -INFINITY ? 0.0f : top;
    const float f = mine ? __builtin_amdgcn_exp2f(ml[0] - ref) : 0.0f;
    float sum = mine ? f * ml[1] : 0.0f;
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) sum += __shfl_xor(sum, k);

    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll 4
    for (uint32_t s = 0; s < n_split; ++s) {
        const float fs = __shfl(f, static_cast<int>(s));
        const float* src = A.part_o + (flat + s * step) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += fs * src[e];
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t* dst = reinterpret_cast<uint16_t*>(A.out) + tok * A.out_tok + head * A.out_head + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = static_cast<uint16_t>(T::pack(acc[e] * inv, 0.0f));
    if (A.lse && lane == 0) A.lse[flat] = sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
}

template <class T, int D, uint32_t kRows>
hipError_t join_one(const AttentionArgs& a, hipStream_t stream) {
    uint32_t most = kRows;  // rows of a tile
    if (a.uniform_q) most = std::min(most, a.uniform_q * a.group);
    const dim3 grid(tile_count<kRows>(a) * a.cache.n_kv_heads, (most + kWaves - 1u) / kWaves);
    hipLaunchKernelGGL((paged_join_kernel<T, D, kRows>), grid, dim3(kWaves * 64), 0, stream, a);
    return hipGetLastError();
}

template <class T>
hipError_t join_dim(const AttentionArgs& a, uint32_t dim, hipStream_t stream) {
    switch (dim) {
        case 64: return join_one<T, 64, kHalfTile>(a, stream);
        case 128: return a.of_tile == kFullTile ? join_one<T, 128, kFullTile>(a, stream) : join_one<T, 128, kHalfTile>(a, stream);
        default: return join_one<T, 256, kHalfTile>(a, stream);
    }
}

}  // namespace

hipError_t launch_paged_join(const AttentionArgs& a, uint32_t dim, uint32_t type, hipStream_t stream) {
    return type == ENGRAM_BF16 ? join_dim<Bf16>(a, dim, stream) : join_dim<F16>(a, dim, stream);
}

}  // namespace engram
