// Shared by the paged attention kernels: arguments, the rows of a request,
// and how a launch finds them.
//
// The rows of a request and KV head are its (new token i, head g of the group)
// pairs, row r = i * G + g: the G query heads that share a KV head read the
// same keys, so a tile of rows reads each key once for all of them.  A row's
// token sits at position p = kv_len - q_len + i and sees the keys
// max(0, p - window + 1) .. p (window 0: all keys up to p).
#pragma once

#include "serving.h"

namespace engram {

struct AttentionArgs {
    const uint8_t* q;
    uint8_t* out;
    float* lse;              // nullptr: not wanted
    const int32_t* table;    // [n_seq][table_width], row stride table_stride
    const int32_t* kv_len;   // [n_seq]
    const int32_t* cu_q;     // [n_seq + 1], or nullptr: n_tok / n_seq tokens each
    CacheView cache;
    // Parts of divided rows, not yet divided by their sums: sums of values, and (reference r, sum of weights) in
    // units of 2^(x - r).  paged_tile.hip: [n_split][n_tok][n_q_heads][dim or 2]; paged_rows.hip: [n_work][2]
    // [min(max_rows, of_tile)][dim or 2], and what there is to join.
    float* part_o;
    float* part_ml;
    int4* part_job;          // [n_work]
    int64_t q_tok, q_head, out_tok, out_head;  // strides, elements
    int64_t table_stride;
    uint32_t table_width;
    uint32_t n_seq;
    uint32_t n_tok;
    uint32_t uniform_q;      // tokens of each request where cu_q is nullptr; a bound of them if there is only one; else 0
    uint32_t group;          // query heads per KV head
    uint32_t window;
    uint32_t split_tokens;   // paged_tile.hip: keys of a split at most (split_keys); 0: one split takes all
    uint32_t n_split;        // splits of a tile at most
    uint32_t n_work;         // paged_rows.hip: workgroups that share the keys evenly; 0: a workgroup takes a tile
    uint32_t min_rows, max_rows;  // requests of this launch: min_rows <= rows <= max_rows
    uint32_t of_tile;        // rows of a tile; paged_tile.hip: kFullTile or kHalfTile, paged_rows.hip: kRowsTile or twice that
    uint32_t tiles_per;      // tiles set aside for each request; 0: as the lengths need (find_tile)
    float scale_log2;        // scale * log2(e)
};

// A word that no kernel writes meanwhile, at an address that is the same for all lanes: by way of the scalar cache, so
// that waiting for it does not wait for the keys and values that were requested before it.
__device__ __forceinline__ int32_t load_scalar(const int32_t* p) {
    return *(const __attribute__((address_space(4))) int32_t*)(p);
}

__device__ __forceinline__ float load_scalar(const float* p) {
    return *(const __attribute__((address_space(4))) float*)(p);
}

// Keys of a request at most: the kernels ask for a few tiles past a request's last key, whose places are int32 too.
constexpr int32_t kMostKeys = INT32_MAX - 4095;

// One request as a launch sees it.  Lengths are bounded by what exists, so
// that no value of cu_q or kv_len leads outside of the buffers.
struct Request {
    uint32_t q0, q_len;
    int32_t kv_len;
};

__device__ __forceinline__ Request request_of(const AttentionArgs& A, uint32_t b) {
    Request r;
    if (A.cu_q) {
        const int32_t n = static_cast<int32_t>(A.n_tok);
        const int32_t q0 = min(max(A.cu_q[b], 0), n);
        const int32_t q1 = min(max(A.cu_q[b + 1], q0), n);
        r.q0 = static_cast<uint32_t>(q0);
        r.q_len = static_cast<uint32_t>(q1 - q0);
    } else {
        r.q0 = b * A.uniform_q;
        r.q_len = A.uniform_q;
    }
    const uint64_t room = static_cast<uint64_t>(A.table_width) << A.cache.page_shift;
    const int32_t most = room < static_cast<uint64_t>(kMostKeys) ? static_cast<int32_t>(room) : kMostKeys;
    r.kv_len = min(max(A.kv_len[b], 0), most);
    return r;
}

// Tiles of kRows rows over all requests.  With equal requests, or where a bound
// of their lengths is small, tile t is tile t % tiles_per of request
// t / tiles_per.  Else (cu_q) the tiles of request b start at
// floor(cu_q[b] * G / kRows) + b, which leaves room for each request's last,
// partly filled tile whatever the lengths are: floor(x + y) + 1 - floor(x)
// >= ceil(y).  The wave finds b 64 candidates at a time.
struct Tile {
    uint32_t b, row0;
    bool live;
};

template <uint32_t kRows>
__device__ __forceinline__ uint32_t tile_start(const AttentionArgs& A, uint32_t b) {
    const int32_t n = static_cast<int32_t>(A.n_tok);
    const uint64_t rows = static_cast<uint64_t>(min(max(A.cu_q[b], 0), n)) * A.group;
    return static_cast<uint32_t>(rows / kRows) + b;
}

template <uint32_t kRows>
__device__ __forceinline__ Tile find_tile(const AttentionArgs& A, uint32_t t) {
    Tile r;
    if (A.tiles_per) {
        r.b = t / A.tiles_per;
        r.row0 = (t - r.b * A.tiles_per) * kRows;
        r.live = r.b < A.n_seq;
        return r;
    }
    const uint32_t lane = threadIdx.x & 63u;
    uint32_t lo = 0, n = A.n_seq;  // the last request of [lo, lo + n) that starts at or before t
    while (n > 1u) {
        const uint32_t step = (n + 63u) / 64u;
        const uint32_t at = lo + lane * step;
        const bool before = at < lo + n && tile_start<kRows>(A, at) <= t;
        const uint32_t k = static_cast<uint32_t>(__builtin_popcountll(__ballot(before)));
        const uint32_t first = k ? lo + (k - 1u) * step : lo;  // lane 0 holds in every ordered cu_q
        n = min(step, lo + n - first);
        lo = first;
    }
    r.b = lo;
    r.row0 = (t - min(t, tile_start<kRows>(A, lo))) * kRows;
    r.live = true;
    return r;
}

template <uint32_t kRows>
inline uint32_t tile_count(const AttentionArgs& A) {
    if (A.tiles_per) return A.n_seq * A.tiles_per;
    return static_cast<uint32_t>(static_cast<uint64_t>(A.n_tok) * A.group / kRows) + A.n_seq;
}

// Keys that the rows [row0, row0 + n) of a request can see: [lo, hi).
struct Span {
    int32_t lo, hi;
};
__device__ __forceinline__ Span span_of(const AttentionArgs& A, const Request& r, uint32_t row0, uint32_t rows) {
    const int32_t back = r.kv_len - static_cast<int32_t>(r.q_len);
    const int32_t first = back + static_cast<int32_t>(row0 / A.group);
    const int32_t last = back + static_cast<int32_t>((row0 + rows - 1u) / A.group);
    Span s;
    s.hi = last + 1;
    s.lo = A.window && first >= static_cast<int32_t>(A.window) ? first - static_cast<int32_t>(A.window) + 1 : 0;
    return s;
}

constexpr uint32_t kLeastSplit = 256;  // keys of a split in paged_tile.hip at least

// Keys of a split in a divided launch of paged_tile.hip: of the longest of its requests, which the host does not know,
// n_split at most.  The host bounds them by the table's width, and a table is often as wide as the longest context that a
// server allows: 64 tokens over 4,096 keys (32 heads over 8 of 128, bf16) with a table for 131,072 took 127 us by that bound
// alone and take 27.2 now; with a table for 4,096 they took 26.9.  Looking at the lengths of several requests costs 1 us (24
// requests of up to 64 tokens over up to 8,192 keys 212.5 us against 211).  The same for all waves of the launch and the join.
__device__ __forceinline__ uint32_t split_keys(const AttentionArgs& A, const Request& req) {
    if (A.split_tokens == 0u) return 0u;
    int32_t longest = req.kv_len;
    if (A.n_seq > 1u) {
        for (uint32_t b = threadIdx.x & 63u; b < A.n_seq; b += 64u) {
            const Request r = request_of(A, b);
            const uint32_t rows = r.q_len * A.group;
            if (rows >= max(A.min_rows, 1u) && rows <= A.max_rows) longest = max(longest, r.kv_len);
        }
        for (uint32_t k = 1; k < min(A.n_seq, 64u); k <<= 1) longest = max(longest, __shfl_xor(longest, static_cast<int>(k)));
    }
    const uint32_t keys = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(longest));
    const uint32_t even = ((keys + A.n_split - 1u) / A.n_split + 63u) & ~63u;
    return min(A.split_tokens, max(even, kLeastSplit));
}

constexpr uint32_t kRowsTile = 16;   // rows of a tile in paged_rows.hip
constexpr uint32_t kFullTile = 256, kHalfTile = 128;  // and in paged_tile.hip; a full one for head_dim 128 only
constexpr int32_t kRowsBlock = 128;  // keys that a workgroup of paged_rows.hip takes at a time
constexpr int32_t kTileAlign = 64;   // a split's keys begin at a multiple of this many in paged_tile.hip

hipError_t launch_paged_rows(const AttentionArgs& a, uint32_t dim, uint32_t type, Held held, hipStream_t stream);
hipError_t launch_paged_tile(const AttentionArgs& a, uint32_t dim, uint32_t type, Held held, hipStream_t stream);
// Joins the parts of a divided launch of launch_paged_tile (launch_paged_rows joins its own).
hipError_t launch_paged_join(const AttentionArgs& a, uint32_t dim, uint32_t type, hipStream_t stream);

}  // namespace engram
