// Paged attention for few rows per request: single tokens and short runs.
//
//     o = sum_j p_j v_j / sum_j p_j,   p_j = exp2(s_j - max s),
//     s_j = scale * log2(e) * (q . k_j)
//
// One pass over the keys with a running maximum and sum.  The work is the
// reading of K and V, each byte once for every 16 rows of its KV head (once for
// a single token of up to 16 heads to a key, twice for 17 to 32 rows):
// HBM-bound.  64 requests of up to 8,192 keys (8 KV heads, head_dim 128, bf16)
// take 218 us, 5.6 TB/s, where a streaming read reaches 6.7 to 6.9, and over
// e4m3 131 us, 4.8 TB/s; with all of them full 360 us, 6.0 TB/s, and 192 us,
// 5.8 TB/s.
//
// Mapping (gfx950, wave64): a workgroup takes one tile of 16 rows of one KV
// head and a run of its keys; its 4 waves take 32 keys each in turn, straight
// from global memory into registers, and join through LDS at the end.
//   * S^T = K Q^T on 16x16x32 MFMA: A is K (lane m of a 16-lane group holds
//     key m, 8 channels), B is Q.  The result has a row in each lane of a
//     group and 4 consecutive keys in its registers, which is the B operand
//     of the second product as it stands: P never changes lanes.
//   * O^T = V^T P^T: a lane reads 8 keys of D/16 consecutive channels, 16
//     lanes together a whole V row, and turns the 8 x D/16 block inside its
//     own registers (one v_perm per pair of keys and channel): no LDS and no
//     transposed copy of V in memory.  The result has the row in the lane
//     again, so the rescaling by exp2(m_old - m_new) is lane-local, and D/4
//     consecutive channels, so rows are written whole.
//   * P is split into a 16-bit part and a 16-bit remainder and multiplied
//     twice: the matrix cores idle here, and the sum keeps about 16 bits of
//     every p instead of 8 (bf16), so that the output's own rounding is the
//     largest error.
// Keys that no row of the tile sees (past the end, before the window, on a
// page whose number is not one of the pool's) count as absent: their V is
// replaced by zero, as 0 * NaN of a page's old content would reach the sum.
// Keys that only some rows see keep their V.  Where the sums end with a NaN,
// the wave takes its keys again, and does the second product of steps that
// hold an infinity or NaN in V key by key, so that no row meets a value that
// its mask hides.  Looking at every V would be 130 instructions more in a step
// of 350.
#include <algorithm>
#include <type_traits>

#include "paged_attention.h"

namespace engram {
namespace {

constexpr uint32_t kRows = kRowsTile;
constexpr uint32_t kStep = 32;      // keys of a wave's step
constexpr uint32_t kWaves = 4;

// A kernel's only argument, read anew from where the hardware keeps it.
__device__ __forceinline__ AttentionArgs args_anew(const AttentionArgs& args) {
#ifdef __HIP_DEVICE_COMPILE__
    typedef const __attribute__((address_space(4))) AttentionArgs* At;
    At at = (At)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(at));
    return *at;
#else
    return args;  // the host's pass over the source
#endif
}

// kBytes of a row in a lane, held as one value: taken apart into words, it
// would be copied where paths join.
template <int kBytes>
struct Words {
    typedef uint32_t V __attribute__((ext_vector_type(kBytes / 4), aligned(kBytes < 16 ? kBytes : 16)));
    V w;
};
template <>
struct Words<4> {
    typedef uint32_t V __attribute__((ext_vector_type(1)));
    V w;
};
template <int kBytes>
__device__ __forceinline__ Words<kBytes> load_words(const uint8_t* p) {
    return Words<kBytes>{*reinterpret_cast<const typename Words<kBytes>::V*>(p)};
}

// Bits lo .. hi - 1 of 0 .. 31.
__device__ __forceinline__ uint32_t bits_of(int32_t lo, int32_t hi) {
    const uint32_t a = static_cast<uint32_t>(min(max(lo, 0), 32)), b = static_cast<uint32_t>(min(max(hi, 0), 32));
    return static_cast<uint32_t>((uint64_t(1) << b) - 1u) & ~static_cast<uint32_t>((uint64_t(1) << a) - 1u);
}

// How the keys of all tiles are shared out.  A request's keys, from the first
// that any of its rows sees, come in blocks of kRowsBlock; its tiles and KV
// heads (tile by tile, all heads of each) are laid end to end, and request
// after request, and each of n_work workgroups takes an equal run of blocks.
// So the lengths, which the host does not know, decide who does what, and all
// workgroups end together: 64 requests of up to 8,192 keys took 240 us with
// splits of one length for all.  A workgroup has at most two parts of divided
// tiles, its first and its last.
struct Load {
    Request req;
    int32_t lo;        // first key, a multiple of 32
    uint32_t blocks;   // of each tile and head, at least 1
    uint32_t weight;   // of the request: 0 if it has no rows here
};

__device__ __forceinline__ Load load_of(const AttentionArgs& A, uint32_t b) {
    Load l;
    l.req = request_of(A, b);
    const uint32_t rows = l.req.q_len * A.group;
    const Span s = span_of(A, l.req, 0, max(rows, 1u));
    l.lo = s.lo & ~31;
    const int32_t keys = max(s.hi - l.lo, 1);
    l.blocks = static_cast<uint32_t>(keys + (kRowsBlock - 1)) / kRowsBlock;
    const bool here = rows > 0 && rows >= A.min_rows && rows <= A.max_rows;
    l.weight = here ? (rows + kRows - 1u) / kRows * A.cache.n_kv_heads * l.blocks : 0u;
    return l;
}

struct Share {
    uint32_t r0, r1;      // blocks of all (the host sees to it that they are below 2^31)
    uint32_t b, off;      // the request in which it begins, and r0's place there
    uint32_t each, more;  // blocks of a share; the first `more` shares have one more
};

struct ShareLds {
    uint32_t wave_sum[kWaves];
    uint32_t b, off;
};

__device__ __forceinline__ uint32_t sum_up_to(uint32_t x) {  // over the lanes up to this one
    const uint32_t lane = threadIdx.x & 63u;
#pragma unroll
    for (uint32_t k = 1; k < 64; k <<= 1) {
        const uint32_t y = __shfl_up(x, k);
        x += lane >= k ? y : 0u;
    }
    return x;
}

__device__ __forceinline__ void cut_share(Share& s, uint32_t all, uint32_t n_work) {
    const uint32_t n = min(n_work, max(all, 1u)), w = blockIdx.x;
    s.each = all / n;
    s.more = all - s.each * n;
    s.r0 = w < n ? w * s.each + min(w, s.more) : all;
    s.r1 = w < n ? s.r0 + s.each + (w < s.more ? 1u : 0u) : all;
}

// This workgroup's share: a sum over the requests' loads, and the request in
// which it begins.  Up to 64 requests each wave does it by itself, a request in
// each lane, without LDS or a barrier.
__device__ __forceinline__ Share share_of(const AttentionArgs& A, ShareLds& sm) {
    Share s;
    const uint32_t tid = threadIdx.x, lane = tid & 63u;
    if (A.n_seq <= 64u) {
        const uint32_t mine = lane < A.n_seq ? load_of(A, lane).weight : 0u;
        const uint32_t upto = sum_up_to(mine);
        cut_share(s, __builtin_amdgcn_readlane(upto, 63), A.n_work);
        s.b = static_cast<uint32_t>(__builtin_popcountll(__ballot(upto <= s.r0))) & 63u;
        s.off = s.r0 - __builtin_amdgcn_readlane(upto - mine, s.b);
        return s;
    }
    constexpr uint32_t kThreads = kWaves * 64;
    const uint32_t per = (A.n_seq + kThreads - 1u) / kThreads;
    const uint32_t b0 = min(tid * per, A.n_seq), b1 = min(b0 + per, A.n_seq);
    uint32_t mine = 0;
#pragma unroll 4
    for (uint32_t b = b0; b < b1; ++b) mine += load_of(A, b).weight;
    uint32_t upto = sum_up_to(mine);
    if (lane == 63u) sm.wave_sum[tid >> 6] = upto;
    __syncthreads();
    uint32_t all = 0;
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) {
        upto += w < (tid >> 6) ? sm.wave_sum[w] : 0u;
        all += sm.wave_sum[w];
    }
    cut_share(s, all, A.n_work);
    s.b = s.off = 0;
    if (s.r0 >= s.r1) return s;  // the same for all threads
    if (s.r0 >= upto - mine && s.r0 < upto) {
        uint32_t at = upto - mine;
        for (uint32_t b = b0; b < b1; ++b) {
            const uint32_t weight = load_of(A, b).weight;
            if (s.r0 < at + weight) {
                sm.b = b;
                sm.off = s.r0 - at;
                break;
            }
            at += weight;
        }
    }
    __syncthreads();
    s.b = __builtin_amdgcn_readfirstlane(sm.b);
    s.off = __builtin_amdgcn_readfirstlane(sm.off);
    return s;
}

template <class T, int D, bool kE4m3>
__global__ __launch_bounds__(kWaves * 64)
    __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : D == 64 ? 3 : 2))) void paged_rows_kernel(const AttentionArgs args) {
    constexpr int EPL = D / 16;              // channels of V in a lane
    constexpr uint32_t CH = D / 32;          // MFMA steps of a score
    constexpr int ES = kE4m3 ? 1 : 2;        // bytes of an element
    constexpr int OP = D + 4;                // padded row of partial sums
    // P and V's type.  An e4m3 V is exact in bf16, whose range holds p * scale.
    using P = std::conditional_t<kE4m3, Bf16, T>;
    __shared__ ShareLds sm_share;
    __shared__ float sm_o[kWaves * kRows * OP];
    __shared__ float sm_m[kWaves][kRows], sm_l[kWaves][kRows];

    Share share;
    if (args.n_work) {
        share = share_of(args, sm_share);
        if (threadIdx.x == 0) args.part_job[blockIdx.x] = int4{0, 0, 0, 0};
        if (share.r0 >= share.r1) return;
    } else {
        const uint32_t tile_at = blockIdx.x / args.cache.n_kv_heads;
        const Tile tile = find_tile<kRows>(args, tile_at);
        if (!tile.live) return;
        share.b = tile.b;
        share.off = tile.row0 / kRows * args.cache.n_kv_heads + (blockIdx.x - tile_at * args.cache.n_kv_heads);
        share.r0 = 0;
        share.r1 = 1;
    }
    // one part of one tile after the other; a workgroup without a share has one tile, and takes all of it
    for (uint32_t r = share.r0; r < share.r1;) {
        // Arguments and lane anew for each part: kept across the parts, they and what follows from them take the registers
        // that the keys' loop needs (it spilled, and took twice the time).
        const AttentionArgs A = args_anew(args);
        uint32_t tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const uint32_t heads = A.cache.n_kv_heads;
        const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63u, n = lane & 15u, g = lane >> 4;
        const Load load = load_of(A, share.b);
        if (A.n_work && share.off >= load.weight) {  // the next request
            if (++share.b >= A.n_seq) return;
            share.off = 0;
            continue;
        }
        const Request req = load.req;
        const uint32_t rows = req.q_len * A.group;
        uint32_t unit, block0, blocks;
        if (A.n_work) {
            unit = share.off / load.blocks;
            block0 = share.off - unit * load.blocks;
            blocks = min(load.blocks - block0, share.r1 - r);
        } else {
            unit = share.off;
            block0 = 0;
            blocks = load.blocks;
        }
        const bool divided = blocks < load.blocks;
        r += A.n_work ? blocks : 1u;
        share.off += blocks;
        const uint32_t tile_row0 = unit / heads * kRows, h = unit % heads;
        if (tile_row0 >= rows || rows < A.min_rows || rows > A.max_rows) return;  // (without a share)
        const uint32_t n_rows = min(kRows, rows - tile_row0);
        const Span span = span_of(A, req, tile_row0, n_rows);
        const Span first_row = span_of(A, req, tile_row0, 1), last_row = span_of(A, req, tile_row0 + n_rows - 1u, 1);
        const int32_t c0 = load.lo + static_cast<int32_t>(block0) * kRowsBlock;
        const int32_t c1 = static_cast<int32_t>(min(static_cast<int64_t>(span.hi), c0 + static_cast<int64_t>(blocks) * kRowsBlock));

        // this lane's row (column n of the products)
        const uint32_t row = min(tile_row0 + n, rows - 1u);
        const uint32_t tok = req.q0 + row / A.group, head = h * A.group + row % A.group;
        const int32_t pos = req.kv_len - static_cast<int32_t>(req.q_len) + static_cast<int32_t>(row / A.group);
        const int32_t see_lo = A.window && pos >= static_cast<int32_t>(A.window) ? pos - static_cast<int32_t>(A.window) + 1 : 0;
        const uint32_t shift = A.cache.page_shift, in_page = (1u << shift) - 1u;
        const int32_t* __restrict__ table = A.table + (share.b) * A.table_stride;
        const int64_t of_head = static_cast<int64_t>(h) << shift;
        const uint8_t* const kh = A.cache.k + of_head * D * ES;
        const uint8_t* const vh = A.cache.v + of_head * D * ES;

        // The pages of a step's four runs of 8 keys (a page holds 8 at least); -1 where there is no such page.
        struct Pages {
            int32_t p[4];
        };
        auto ask_pages = [&](int32_t base) {
            Pages r;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int32_t p = load_scalar(table + (static_cast<uint32_t>(min(base + 8 * i, c1 - 1)) >> shift));
                r.p[i] = p >= 0 && p < A.cache.n_pages ? p : -1;
            }
            return r;
        };
        Words<16> kw[2][ES == 1 ? CH / 2 : CH];  // keys base + n and base + 16 + n
        Words<EPL * ES> vw[2][4];                // keys base + 4g + 0..3 and base + 16 + 4g + 0..3, which are also this lane's scores
        f32x4v ks[2], vs[2];
        auto ask_k = [&](int32_t base, const Pages& pg) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int64_t a = max(pg.p[2 * t], 0) * A.cache.k_page_stride, b = max(pg.p[2 * t + 1], 0) * A.cache.k_page_stride;
                const uint32_t key = (static_cast<uint32_t>(base) + 16 * t + n) & in_page;
                const uint8_t* p = kh + ((n >> 3 ? b : a) + static_cast<int64_t>(key * D)) * ES;
#pragma unroll
                for (uint32_t i = 0; i < (ES == 1 ? CH / 2 : CH); ++i)
                    kw[t][i] = load_words<16>(p + (ES == 1 ? 64 * i + 16 * g : (32 * i + 8 * g) * 2));
                if constexpr (kE4m3) {
                    const int64_t c = max(pg.p[2 * t], 0), d = max(pg.p[2 * t + 1], 0);
                    const uint32_t at = (static_cast<uint32_t>(base) + 16 * t + 4u * g) & in_page;
                    ks[t] = *reinterpret_cast<const f32x4v*>(A.cache.k_scale + ((((g >> 1 ? d : c) * heads) << shift) + of_head + at));
                }
            }
        };
        auto ask_v = [&](int32_t base, const Pages& pg) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int64_t a = max(pg.p[2 * t], 0) * A.cache.v_page_stride, b = max(pg.p[2 * t + 1], 0) * A.cache.v_page_stride;
                const uint32_t key = (static_cast<uint32_t>(base) + 16 * t + 4u * g) & in_page;
                const uint8_t* p = vh + ((g >> 1 ? b : a) + static_cast<int64_t>(key * D + n * EPL)) * ES;
#pragma unroll
                for (int i = 0; i < 4; ++i) vw[t][i] = load_words<EPL * ES>(p + i * D * ES);
                if constexpr (kE4m3) {
                    const int64_t c = max(pg.p[2 * t], 0), d = max(pg.p[2 * t + 1], 0);
                    vs[t] = *reinterpret_cast<const f32x4v*>(A.cache.v_scale + ((((g >> 1 ? d : c) * heads) << shift) + of_head + key));
                }
            }
        };

        u32x4v q[CH];
        {
            const uint8_t* qp = A.q + (tok * A.q_tok + head * A.q_head) * 2;
#pragma unroll
            for (uint32_t c = 0; c < CH; ++c) {
                // e4m3 keys come 16 channels a load, which orders the channels of a pair of steps
                const uint32_t d = kE4m3 ? 64 * (c / 2) + 16 * g + 8 * (c % 2) : 32 * c + 8 * g;
                q[c] = *reinterpret_cast<const u32x4v*>(qp + d * 2);
            }
        }
        float m, nb, l;  // the reference (a score in units of log2), kShift - m once there is one, the sum
        f32x4v o[EPL];
        for (bool careful = false;; careful = true) {
            m = -INFINITY;
            nb = l = 0.0f;
#pragma unroll
            for (int f = 0; f < EPL; ++f) o[f] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
            // The next step's keys are requested once this step's scores have used the registers, its values once the sums have.
            const int32_t first = c0 + static_cast<int32_t>(wave * kStep);
            Pages pages, ahead;
            if (first < c1) {
                pages = ask_pages(first);
                ask_k(first, pages);
                ask_v(first, pages);
                ahead = ask_pages(min(first + static_cast<int32_t>(kStep * kWaves), c1 - 1));
            }
            for (int32_t base = first; base < c1; base += kStep * kWaves) {
                const int32_t next = base + static_cast<int32_t>(kStep * kWaves);
                f32x4v s[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    s[t] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (uint32_t c = 0; c < CH; ++c) {
                        u32x4v a;
                        if constexpr (kE4m3) {
                            const uint32_t w0 = kw[t][c / 2].w[2 * (c % 2)], w1 = kw[t][c / 2].w[2 * (c % 2) + 1];
                            a = u32x4v{T::template from_e4m3<false>(w0), T::template from_e4m3<true>(w0),
                                       T::template from_e4m3<false>(w1), T::template from_e4m3<true>(w1)};
                        } else {
                            a = u32x4v{kw[t][c].w[0], kw[t][c].w[1], kw[t][c].w[2], kw[t][c].w[3]};
                        }
                        s[t] = T::mfma16(a, q[c], s[t]);
                    }
                }
                float x[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[t][i] = s[t][i] * A.scale_log2;
                        if constexpr (kE4m3) x[t][i] *= ks[t][i];
                    }
                if (next < c1) ask_k(next, ahead);

                // every row of the tile sees every key of a whole step; else each row's own keys
                const uint32_t there = ((g >> 1 ? pages.p[1] : pages.p[0]) >= 0 ? 0xFFFFu : 0u) |
                                       ((g >> 1 ? pages.p[3] : pages.p[2]) >= 0 ? 0xFFFF0000u : 0u);
                const bool whole = base >= last_row.lo && base + static_cast<int32_t>(kStep) <= min(first_row.hi, c1) &&
                                   (pages.p[0] | pages.p[1] | pages.p[2] | pages.p[3]) >= 0;
                uint32_t seen = ~0u;  // keys base + 4g + bit that this lane's row sees (bits 0 to 3 and 16 to 19 are used)
                if (!whole) {
                    const int32_t from = base + static_cast<int32_t>(4u * g);
                    seen = bits_of(see_lo - from, min(pos + 1, c1) - from) & there;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[t][i] = (seen >> (16 * t + i)) & 1u ? x[t][i] : -INFINITY;
                }
                float top = -INFINITY;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = fmaxf(top, x[t][i]);
                top = max32(max16(top));
                if (__any(top > m + P::kSlack)) {
                    const float m_new = fmaxf(m, top);
                    const float nb_new = m_new == -INFINITY ? 0.0f : P::kShift - m_new;
                    const float alpha = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(nb_new - nb);
                    l *= alpha;
#pragma unroll
                    for (int f = 0; f < EPL; ++f)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[f][i] *= alpha;
                    m = m_new;
                    nb = nb_new;
                }
                float p[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        p[t][i] = __builtin_amdgcn_exp2f(x[t][i] + nb);
                        l += p[t][i];
                        if constexpr (kE4m3) p[t][i] = (seen >> (16 * t + i)) & 1u ? p[t][i] * vs[t][i] : 0.0f;
                    }

                // V rows as 16-bit pairs of channels
                typedef Words<EPL * 2> Pairs;
                Pairs v[8];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (kE4m3) {
#pragma unroll
                            for (int e = 0; e < EPL / 2; ++e)
                                v[4 * t + i].w[e] = (e & 1) ? P::template from_e4m3<true>(vw[t][i].w[e / 2])
                                                            : P::template from_e4m3<false>(vw[t][i].w[e / 2]);
                        } else {
                            v[4 * t + i] = vw[t][i];
                        }
                    }
                if (!whole) {
                    const int32_t from = base + static_cast<int32_t>(4u * g);
                    const uint32_t any = bits_of(span.lo - from, c1 - from) & there;  // the others no row sees
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[k].w = (any >> (16 * (k / 4) + k % 4)) & 1u ? v[k].w : static_cast<typename Pairs::V>(0u);
                }
                uint32_t bad = 0;
                if (__builtin_expect(careful, 0)) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
#pragma unroll
                        for (int e = 0; e < EPL / 2; ++e) bad |= P::nonfinite(v[k].w[e]);
                }
                if (__builtin_expect(careful && __any(bad != 0), 0)) {
                    // Key by key, V by way of LDS (the waves' sums use it only later): lane (n, g) adds p * V[its channels] for
                    // the keys that row n sees.  A loop of few registers, after which the products go on with zeros.
                    uint32_t* const rows_v = reinterpret_cast<uint32_t*>(sm_o + wave * kRows * OP);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
#pragma unroll
                        for (int e = 0; e < EPL / 2; ++e) {
                            rows_v[(16 * (k / 4) + 4 * g + k % 4) * (D / 2) + n * (EPL / 2) + e] = v[k].w[e];
                            v[k].w[e] = 0u;
                        }
                    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll 1
                    for (uint32_t k = 0; k < kStep; ++k) {
                        const int from = static_cast<int>(((k & 15u) >> 2) * 16u + n);
                        const uint32_t at = (k >> 4) * 4u + (k & 3u);
                        float pk = p[0][0];
#pragma unroll
                        for (uint32_t z = 1; z < 8; ++z) pk = at == z ? p[z / 4][z % 4] : pk;
                        pk = __shfl(pk, from);
                        if ((static_cast<uint32_t>(__shfl(static_cast<int>(seen), from)) >> (16u * (k >> 4) + (k & 3u))) & 1u) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int e = 0; e < EPL / 2; ++e) {
                                    const uint32_t w = rows_v[k * (D / 2) + (4 * g + i) * (EPL / 2) + e];
                                    o[2 * e][i] = __builtin_fmaf(pk, P::lo(w), o[2 * e][i]);
                                    o[2 * e + 1][i] = __builtin_fmaf(pk, P::hi(w), o[2 * e + 1][i]);
                                }
                        }
                    }
                }
                u32x4v ph, pl;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float a = p[t][2 * i], b = p[t][2 * i + 1];
                        const uint32_t w = P::pack(a, b);
                        ph[2 * t + i] = w;
                        pl[2 * t + i] = P::pack(a - P::lo(w), b - P::hi(w));
                    }
#pragma unroll
                for (int f = 0; f < EPL; ++f) {
                    u32x4v a;
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        a[w] = __builtin_amdgcn_perm(v[2 * w + 1].w[f / 2], v[2 * w].w[f / 2], (f & 1) ? 0x07060302u : 0x05040100u);
                    o[f] = P::mfma16(a, ph, o[f]);
                    o[f] = P::mfma16(a, pl, o[f]);
                }
                if (next < c1) {
                    ask_v(next, ahead);
                    pages = ahead;
                    ahead = ask_pages(min(next + static_cast<int32_t>(kStep * kWaves), c1 - 1));
                }
            }
            // A NaN: it may be there by right, or come from 0 * infinity or 0 * NaN of a value that its row's mask hides, or from
            // an infinity times a remainder of P.  The keys again, with their values looked at.
            bool nan = false;
#pragma unroll
            for (int f = 0; f < EPL; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) nan |= o[f][i] != o[f][i];
            if (__builtin_expect(careful || !__any(nan), 1)) break;
        }

        // join the waves
        l = sum32(sum16(l));
        if (g == 0) {
            sm_m[wave][n] = m == -INFINITY ? m : -nb;
            sm_l[wave][n] = l;
        }
        float* mine = sm_o + (wave * kRows + n) * OP + g * (D / 4);
        if (n < n_rows) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int f = 0; f < EPL; f += 4)
                    *reinterpret_cast<f32x4v*>(mine + i * EPL + f) = f32x4v{o[f][i], o[f + 1][i], o[f + 2][i], o[f + 3][i]};
        }
        __syncthreads();

        const uint32_t at_row = tid >> 4, part = tid & 15u;  // row, EPL channels of it
        if (at_row < n_rows) {
            float top = -INFINITY;
#pragma unroll
            for (uint32_t w = 0; w < kWaves; ++w) top = fmaxf(top, sm_m[w][at_row]);
            const float ref = top == -INFINITY ? 0.0f : top;
            float sum = 0.0f, acc[EPL];
#pragma unroll
            for (int e = 0; e < EPL; ++e) acc[e] = 0.0f;
#pragma unroll
            for (uint32_t w = 0; w < kWaves; ++w) {
                const float f = __builtin_amdgcn_exp2f(sm_m[w][at_row] - ref);
                sum += f * sm_l[w][at_row];
                const float* src = sm_o + (w * kRows + at_row) * OP + part * EPL;
#pragma unroll
                for (int e = 0; e < EPL; ++e) acc[e] += f * src[e];
            }
            if (divided) {
                const uint32_t place = 2u * blockIdx.x + (block0 == 0 ? 1u : 0u);
                const uint64_t at = static_cast<uint64_t>(place) * min(A.max_rows, kRows) + at_row;
                float* dst = A.part_o + at * D + part * EPL;
#pragma unroll
                for (int e = 0; e < EPL; e += 4)
                    *reinterpret_cast<f32x4v*>(dst + e) = f32x4v{acc[e], acc[e + 1], acc[e + 2], acc[e + 3]};
                if (part == 0) *reinterpret_cast<f32x2v*>(A.part_ml + at * 2) = f32x2v{top, sum};
            } else {
                const uint32_t rr = tile_row0 + at_row;
                const uint32_t out_tok = req.q0 + rr / A.group, out_head = h * A.group + rr % A.group;
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                uint32_t w[EPL / 2];
#pragma unroll
                for (int e = 0; e < EPL / 2; ++e) w[e] = T::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
                uint32_t* dst = reinterpret_cast<uint32_t*>(A.out + (out_tok * A.out_tok + out_head * A.out_head + part * EPL) * 2);
#pragma unroll
                for (int e = 0; e < EPL / 2; ++e) dst[e] = w[e];
                if (A.lse && part == 0)
                    A.lse[static_cast<uint64_t>(out_tok) * (heads * A.group) + out_head] =
                        sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
            }
        }
        if (r < share.r1) {
            __syncthreads();  // LDS is read
        } else if (divided && block0 == 0 && tid == 0) {
            // the tile begins in this share and ends in a later one: {request, first row, head, shares} for the join
            const uint32_t x = share.r1 - 1u + (load.blocks - blocks), big = share.more * (share.each + 1u);
            const uint32_t to = x < big ? x / (share.each + 1u) : share.more + (x - big) / share.each;
            A.part_job[blockIdx.x] = int4{static_cast<int32_t>(share.b), static_cast<int32_t>(tile_row0), static_cast<int32_t>(h),
                                          static_cast<int32_t>(to - blockIdx.x + 1u)};
        }
    }
}

// The parts of a divided tile joined, in their order: the workgroup whose
// share a tile begins in has its first part, the next ones the others.  The
// references and sums first, then the values; 4 waves share a row's parts.
template <class T, int D>
__global__ __launch_bounds__(256) void rows_join_kernel(const AttentionArgs A) {
    constexpr int E = D / 64;  // channels of a lane
    __shared__ float sm_o[4][D];
    const int4 job = A.part_job[blockIdx.x];
    const uint32_t n_parts = static_cast<uint32_t>(job.w);
    if (n_parts < 2u) return;
    const Request req = request_of(A, static_cast<uint32_t>(job.x));
    const uint32_t rows = req.q_len * A.group, row = static_cast<uint32_t>(job.y) + blockIdx.y, h = static_cast<uint32_t>(job.z);
    if (row >= rows) return;
    const uint32_t heads = A.cache.n_kv_heads;
    const uint32_t tok = req.q0 + row / A.group, head = h * A.group + row % A.group;
    const uint32_t per = min(A.max_rows, kRows);
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63u;
    const auto place = [&](uint32_t s) {
        return static_cast<uint64_t>(2u * (blockIdx.x + s) + (s == 0 ? 1u : 0u)) * per + blockIdx.y;
    };
    float top = -INFINITY;
    for (uint32_t s = lane; s < n_parts; s += 64u) top = fmaxf(top, A.part_ml[place(s) * 2]);
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) top = fmaxf(top, __shfl_xor(top, k));
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    for (uint32_t s = lane; s < n_parts; s += 64u) {
        const f32x2v ml = *reinterpret_cast<const f32x2v*>(A.part_ml + place(s) * 2);
        sum += __builtin_amdgcn_exp2f(ml[0] - ref) * ml[1];
    }
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) sum += __shfl_xor(sum, k);
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll 8
    for (uint32_t s = wave; s < n_parts; s += 4u) {
        const uint64_t at = place(s);
        const float f = __builtin_amdgcn_exp2f(A.part_ml[at * 2] - ref);
        const float* src = A.part_o + at * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += f * src[e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[wave][lane * E + e] = acc[e];
    __syncthreads();
    if (wave != 0) return;
#pragma unroll
    for (uint32_t w = 1; w < 4; ++w)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += sm_o[w][lane * E + e];
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t* dst = reinterpret_cast<uint16_t*>(A.out) + tok * A.out_tok + head * A.out_head + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) dst[e] = static_cast<uint16_t>(T::pack(acc[e] * inv, 0.0f));
    if (A.lse && lane == 0)
        A.lse[static_cast<uint64_t>(tok) * (heads * A.group) + head] =
            sum == 0.0f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
}

template <class T, int D, bool kE4m3>
hipError_t rows_one(const AttentionArgs& a, hipStream_t stream) {
    const uint32_t groups = a.n_work ? a.n_work : tile_count<kRows>(a) * a.cache.n_kv_heads;
    hipLaunchKernelGGL((paged_rows_kernel<T, D, kE4m3>), dim3(groups), dim3(kWaves * 64), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.n_work) return e;
    hipLaunchKernelGGL((rows_join_kernel<T, D>), dim3(a.n_work, std::min(a.max_rows, kRows)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <class T, bool kE4m3>
hipError_t rows_dim(const AttentionArgs& a, uint32_t dim, hipStream_t stream) {
    switch (dim) {
        case 64: return rows_one<T, 64, kE4m3>(a, stream);
        case 128: return rows_one<T, 128, kE4m3>(a, stream);
        default: return rows_one<T, 256, kE4m3>(a, stream);
    }
}

}  // namespace

hipError_t launch_paged_rows(const AttentionArgs& a, uint32_t dim, uint32_t type, bool e4m3, hipStream_t stream) {
    if (type == ENGRAM_BF16) return e4m3 ? rows_dim<Bf16, true>(a, dim, stream) : rows_dim<Bf16, false>(a, dim, stream);
    return e4m3 ? rows_dim<F16, true>(a, dim, stream) : rows_dim<F16, false>(a, dim, stream);
}

}  // namespace engram
