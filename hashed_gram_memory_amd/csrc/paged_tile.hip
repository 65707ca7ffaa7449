// Paged attention for many rows per request: chunks of prompts.
//
//     o = sum_j p_j v_j / sum_j p_j,   p_j = exp2(c s_j + b),   s_j = q . k_j,
//     c = |scale| log2(e) (a negative scale flips q's signs)
//
// One pass over the keys; b = -c max s is held for each row and moves only
// when a score passes it by 2^kSlack, so that the sums are rescaled a few times
// at a row's first keys and hardly ever later.  The work is the two products:
// bound by the matrix pipes, and next to them by the exponentials.
//
// Mapping (gfx950, wave64): a workgroup takes a tile of 256 or 128 rows of one KV
// head and one split of their keys; each wave holds 32 rows' q, scores and sums
// in registers.  K and V go through LDS, a tile of KT keys at a time, in rings
// of four and five buffers.
//   * S^T = K Q^T on 32x32x16 MFMA: a lane holds a row and 16 of 32 keys, so
//     the maximum and sum of a row need one exchange between a wave's halves,
//     and the scores are the second product's B operand as they stand: P never
//     changes lanes.
//   * O^T = V^T P^T: V lies in LDS as it lies in memory; the transposing LDS
//     reads give four keys of a channel to a lane.
//   * 16-byte blocks of a key's row are swapped within its LDS row (K by the
//     key's low bits, V by two of them), so that neither kind of read has two
//     lanes on one bank.  A lane asks for the block that belongs to its place,
//     so the swap costs nothing.
//   * 16-bit tiles go from memory to LDS without a register between, three
//     turns before they are read; e4m3 codes by way of registers, where they
//     are widened (exactly).  Addresses come from the page table by scalar
//     loads, a turn early.
//   * The eight waves of a full tile are two on each SIMD, in two halves that
//     take turns: one does the products of a tile while the other does its
//     softmax and asks for tiles, so that the matrix pipe and the vector pipe of
//     a SIMD both work.  The four waves of a half tile leave room for another
//     workgroup on the CU, which the hardware mixes with it as it comes: better
//     where tiles differ or are not full.  For head_dim 64 all tiles are half
//     ones: a batch of 24 requests of 1 to 512 tokens with a window, fp16, took
//     66 us against 73 and a chunk of 2,048 over 32,768 keys of e4m3 1,001
//     against 1,109, for which the same chunk over 16 bits is 2% slower (678
//     against 663).  A head_dim of 256 leaves registers for one wave on a SIMD:
//     half tiles, one to a CU.  Over e4m3, whose tiles pass through registers,
//     full tiles spill 6 registers and head_dim 256 some 65.
//
// What it measured, for 2,048 tokens at the end of 32,768 keys, 32 heads over 8
// of head_dim 128, bf16: 1,314 us with two buffers, staged through registers,
// and no turns; 1,050 to 1,100 us as it stands, 1.01 PFLOP/s at the most, where
// a product of 8192^3 reached 1.25 to 1.37 on the same card.  A turn's products
// take 1,900 cycles of a wave for 1,190 that they take alone: LDS answers
// products and the other half's softmax issues between them.  Of the time,
// about a sixth is the card's power: zeros for q, K and V run that much faster.
//
// P is rounded once to the type of q and out (half a step of each p; their
// average over the keys adds to the output about what the output's own
// rounding does: 2.4e-3 of it in bf16 where 1.7e-3 are the output's, 2.9e-4 and
// 2.1e-4 in fp16).  Twice the digits, as in paged_rows.hip, are half as many
// products again, and here the products are what is waited for: with them the
// chunk took 1,450 us for 1,097, the batch of 24 requests 72.0 for 62.7, the
// chunk of head_dim 64 893 for 699.
//
// What a row does not see: scores of hidden keys become -inf before the
// maximum, and their p is 0.  A key that no row sees (past the end, before the
// window) is read from one that some row sees, and one on a page outside the
// pool as zeros, so nothing is read that is not the request's.  Keys that only
// some rows see can hold infinities or NaN in V, and 0 times them is NaN: where
// a workgroup's sums end with a NaN, it takes its keys again with zeros in the
// places of infinities and NaN, and counts those for the rows that see them by
// two more products, of ones (not below +inf, not above -inf).
#include <type_traits>

#include "paged_attention.h"

namespace engram {
namespace {

typedef short s16x4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4v lds_s16x4v;
typedef __attribute__((address_space(3))) const u32x4v lds_u32x4v;

// Block (16 bytes of 16-bit channels) of a key's LDS row where channel block c lies.
template <int D>
__device__ __forceinline__ uint32_t k_block(uint32_t key, uint32_t c) {
    return c ^ (D == 64 ? (key >> 1) & 7u : D == 128 ? key & 15u : key & 7u);
}
template <int D>
__device__ __forceinline__ uint32_t v_block(uint32_t key, uint32_t c) {
    return D == 64 ? c ^ (((key >> 1) & 1u) << 2) : c ^ ((key & 3u) << 2);
}

// The order of a turn's products: kScores of them with one LDS read each, kSums with two, the reads kAhead products
// early, which is what LDS takes to answer.  (Left to itself, the compiler reads one product early.)
template <int kScores, int kSums>
__device__ __forceinline__ void products_in_order() {
    constexpr int kMfma = 0x8, kRead = 0x100, kAhead = 6;
    static_assert(kScores >= kAhead && kSums >= kAhead, "");
    __builtin_amdgcn_sched_group_barrier(kRead, kAhead, 0);
#pragma unroll
    for (int i = 0; i < kScores - kAhead; ++i) {
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kRead, 1, 0);
    }
#pragma unroll
    for (int i = 0; i < kSums; ++i) {
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kRead, 2, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kMfma, kAhead, 0);
}

// What the rows of pages that are none are read from.
__device__ __attribute__((aligned(16))) const uint8_t g_zeros[4096] = {};

__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) void*)(p)));
}
// 16 bytes of each lane to LDS, lane after lane from an address that is the same for all.  The compiler knows of no such
// load: wait_loads is to stand between it and the barrier that its readers wait for.  M0 holds the LDS address.
__device__ __forceinline__ void to_lds(uint64_t base, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :
                 : "v"(offset), "s"(base), "s"(to)
                 : "m0", "memory");
}
// all but the last kMost loads have come
template <int kMost>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(kMost) : "memory");
}

// eight e4m3 codes as 16-bit numbers
template <class T>
__device__ __forceinline__ u32x4v widen(u32x2v w) {
    return u32x4v{T::template from_e4m3<false>(w[0]), T::template from_e4m3<true>(w[0]), T::template from_e4m3<false>(w[1]),
                  T::template from_e4m3<true>(w[1])};
}

template <class T, int D, bool kE4m3, int kWaves>
__global__ __launch_bounds__(kWaves * 64) __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : 2, D == 256 ? 1 : 2))) void paged_tile_kernel(
    const AttentionArgs A) {
    constexpr uint32_t kRows = kWaves * 32u, kThreads = kWaves * 64u;
    constexpr bool kTurns = kWaves == 8;            // two waves of a workgroup on a SIMD
    constexpr int KT = kTurns || D == 64 ? 64 : 32; // keys of a tile
    constexpr int TB = KT / 32;                     // blocks of 32 keys
    constexpr int CB = D / 8;                       // 16-byte blocks of a row
    constexpr int CH = D / 16;                      // MFMA steps of a score
    constexpr int FB = D / 32;                      // blocks of 32 channels
    constexpr int NL = KT * CB / int(kThreads);     // blocks of K (and of V) that a thread brings
    static_assert(NL >= 1 && NL * int(kThreads) == KT * CB, "every thread brings the same");
    using P = T;                                    // P and V's type; e4m3 codes are exact in both types
    constexpr uint32_t ES = kE4m3 ? 1 : 2;
    constexpr float kSlack = P::kSlack, kShift = P::kShift;
    // With codes P is p_j times V's scale, which fp16's range does not hold under a reference of the scores alone: there the
    // reference is that of c s_j + log2(scale), with the logarithm bounded so that the sum of the p_j stays in fp32's range.
    constexpr bool kScaled = kE4m3 && std::is_same_v<T, F16>;

    __shared__ __attribute__((aligned(1024))) uint16_t sm_k[4][KT * D];
    __shared__ __attribute__((aligned(1024))) uint16_t sm_v[5][KT * D];
    __shared__ __attribute__((aligned(16))) float sm_scale[8][kScaled ? 3 : 2][kE4m3 ? KT : 4];

    const uint32_t heads = A.cache.n_kv_heads;
    const uint32_t tile_at = blockIdx.x / heads, h = blockIdx.x - tile_at * heads;
    const Tile tile = find_tile<kRows>(A, tile_at);
    if (!tile.live) return;
    const Request req = request_of(A, tile.b);
    const uint32_t rows = req.q_len * A.group;
    if (tile.row0 >= rows || rows < A.min_rows || rows > A.max_rows) return;
    // a request's last rows have the most keys: first come, first served
    const uint32_t row0 = ((rows - 1u) / kRows) * kRows - tile.row0;
    const uint32_t n_rows = min(kRows, rows - row0);
    const Span span = span_of(A, req, row0, n_rows);

    // this split's keys [c0, c1)
    const int32_t base0 = span.lo & ~(kTileAlign - 1);
    const uint32_t split = blockIdx.y;
    const uint32_t of_split = split_keys(A, req);
    const bool divided = of_split != 0 && span.hi > base0 && static_cast<uint32_t>(span.hi - base0) > of_split;
    int32_t c0 = base0, c1 = max(span.hi, base0);
    if (divided) {
        const int64_t at = static_cast<int64_t>(base0) + static_cast<int64_t>(split) * of_split;
        if (at >= span.hi) return;
        c0 = static_cast<int32_t>(at);
        c1 = static_cast<int32_t>(min(at + of_split, static_cast<int64_t>(span.hi)));
    } else if (split != 0) {
        return;
    }
    const int32_t n_tiles = static_cast<int32_t>((static_cast<uint32_t>(c1 - c0) + KT - 1u) / KT);

    const uint32_t tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63u;
    const uint32_t n = lane & 31u, g = lane >> 5;

    // this lane's row (column n of the products), and what the wave's rows see
    const uint32_t wrow0 = row0 + wave * 32u;
    const bool alive = wrow0 < rows;
    const uint32_t row = min(wrow0 + n, rows - 1u);
    const uint32_t tok = req.q0 + row / A.group, head = h * A.group + row % A.group;
    const int32_t pos = req.kv_len - static_cast<int32_t>(req.q_len) + static_cast<int32_t>(row / A.group);
    const int32_t see_lo = A.window && pos >= static_cast<int32_t>(A.window) ? pos - static_cast<int32_t>(A.window) + 1 : 0;
    const uint32_t wlast = min(wrow0 + 31u, rows - 1u), wfirst = min(wrow0, rows - 1u);
    const Span wfirst_row = span_of(A, req, wfirst, 1), wlast_row = span_of(A, req, wlast, 1);
    const float c = A.scale_log2 == 0.0f ? 1e-45f : fabsf(A.scale_log2);  // never 0, for the sake of -inf * c

    u32x4v q[CH];
    {
        const uint8_t* qp = A.q + (tok * A.q_tok + head * A.q_head) * 2;
        const uint32_t flip = A.scale_log2 < 0.0f ? 0x80008000u : 0u;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            q[i] = *reinterpret_cast<const u32x4v*>(qp + (16 * i + 8 * g) * 2);
#pragma unroll
            for (int j = 0; j < 4; ++j) q[i][j] ^= flip;
        }
    }

    float m = -INFINITY;  // the reference: a score times c
    float nb = 0.0f;      // kShift - m, once there is one
    float l = 0.0f;
    f32x16v o[FB];
#pragma unroll
    for (int f = 0; f < FB; ++f)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[f][i] = 0.0f;

    const uint32_t shift = A.cache.page_shift, in_page = (1u << shift) - 1u;
    const int32_t* table = A.table + tile.b * A.table_stride;
    const uint8_t* const kh = A.cache.k + (static_cast<int64_t>(h) << shift) * D * ES;
    const uint8_t* const vh = A.cache.v + (static_cast<int64_t>(h) << shift) * D * ES;

    const auto base_of = [&](int32_t t) { return c0 + t * KT; };
    // A thread brings the blocks at the LDS places i * kThreads + tid of a tile.  A wave's blocks i are those of 64 / CB rows
    // within one run of 8 keys, and so on one page: their address is the same for all lanes but for a constant.
    constexpr uint32_t kStep = kThreads / CB;  // rows from one i to the next: blocks are swapped alike in them
    static_assert(kStep % (D == 256 ? 8 : 16) == 0, "");
    const uint32_t wave_row = wave * (64u / CB);
    const uint32_t k_col = k_block<D>(tid / CB, tid % CB) * 8u * ES, v_col = v_block<D>(tid / CB, tid % CB) * 8u * ES;
    struct Pages {
        int32_t of[NL];  // of the wave's blocks
    };
    // The first key of the wave's rows i, or where all of them lie outside of [span.lo, c1), of rows in the run next to them.
    const auto key_of = [&](int32_t t, int i) __attribute__((always_inline)) {
        const int64_t key = static_cast<int64_t>(base_of(t)) + wave_row + i * kStep;
        const int32_t low = (span.lo & ~7) + static_cast<int32_t>(wave_row & 7u);
        return static_cast<int32_t>(min(max(key, static_cast<int64_t>(low)), static_cast<int64_t>(c1 - 1)));
    };
    const auto ask_pages = [&](int32_t t) __attribute__((always_inline)) {
        Pages r;
#pragma unroll
        for (int i = 0; i < NL; ++i) r.of[i] = load_scalar(table + (static_cast<uint32_t>(key_of(t, i)) >> shift));
        return r;
    };
    // Where the wave's blocks come from: one address, and what each lane adds to it.  A key that no row sees takes the row of
    // one that some row sees: its weight is 0.
    struct Source {
        uint64_t k, v;
        uint32_t k_off, v_off;
    };
    struct Sources {
        Source of[NL];
    };
    const auto sources_of = [&](int32_t t, const Pages& pg) __attribute__((always_inline)) {
        Sources r;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int32_t key = key_of(t, i);
            const uint32_t in = static_cast<uint32_t>(key) & in_page;
            const int64_t p = pg.of[i];
            const bool ok = p >= 0 && p < A.cache.n_pages;
            const uint64_t none = reinterpret_cast<uint64_t>(g_zeros);
            r.of[i].k = ok ? reinterpret_cast<uint64_t>(kh + (p * A.cache.k_page_stride + in * D) * ES) : none;
            r.of[i].v = ok ? reinterpret_cast<uint64_t>(vh + (p * A.cache.v_page_stride + in * D) * ES) : none;
            const int32_t more = min(max(static_cast<int32_t>(lane / CB), span.lo - key), c1 - 1 - key);
            r.of[i].k_off = static_cast<uint32_t>(more) * (D * ES) + k_col;
            r.of[i].v_off = static_cast<uint32_t>(more) * (D * ES) + v_col;
        }
        return r;
    };
    // 16 bits: straight to LDS
    const auto fetch = [&](int32_t t, const Sources& from) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const uint32_t at = wave * 1024u + i * kThreads * 16u;
            to_lds(from.of[i].k, from.of[i].k_off, at + lds_address(&sm_k[t & 3][0]));
            to_lds(from.of[i].v, from.of[i].v_off, at + lds_address(&sm_v[static_cast<uint32_t>(t) % 5u][0]));
        }
    };
    // e4m3: by way of registers, to be widened
    struct Blocks {
        u32x2v k[NL], v[NL];
    };
    const auto ask = [&](const Sources& from) __attribute__((always_inline)) {
        Blocks r;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            r.k[i] = *reinterpret_cast<const u32x2v*>(from.of[i].k + from.of[i].k_off);
            r.v[i] = *reinterpret_cast<const u32x2v*>(from.of[i].v + from.of[i].v_off);
        }
        return r;
    };
    const auto put = [&](int32_t t, const Blocks& r) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const uint32_t at = (i * kThreads + tid) * 8u;
            *reinterpret_cast<u32x4v*>(&sm_k[t & 3][at]) = widen<T>(r.k[i]);
            *reinterpret_cast<u32x4v*>(&sm_v[static_cast<uint32_t>(t) % 5u][at]) = widen<P>(r.v[i]);
        }
    };
    // the scale of key tid % KT: of K (tid < KT), of V
    const auto ask_scale_page = [&](int32_t t) __attribute__((always_inline)) {
        const int64_t key = min(static_cast<int64_t>(base_of(t)) + tid % KT, static_cast<int64_t>(c1) - 1);
        return tid < 2u * KT ? table[static_cast<uint32_t>(key) >> shift] : -1;
    };
    const auto ask_scale = [&](int32_t t, int32_t page) __attribute__((always_inline)) {
        const uint32_t in = (static_cast<uint32_t>(base_of(t)) + tid % KT) & in_page;
        const float* from = tid < KT ? A.cache.k_scale : A.cache.v_scale;
        const bool ok = page >= 0 && page < A.cache.n_pages;
        return ok ? from[((static_cast<int64_t>(page) * heads + h) << shift) + in] : 0.0f;
    };
    const auto put_scale = [&](int32_t t, float x) __attribute__((always_inline)) {
        if (tid < 2u * KT) sm_scale[t & 7][tid / KT][tid % KT] = x;
        if constexpr (kScaled)
            if (tid >= KT && tid < 2u * KT) sm_scale[t & 7][2][tid % KT] = fminf(fmaxf(__log2f(fabsf(x)), -60.0f), 60.0f);
    };

    bool all_there = true;  // all pages: else every tile is looked at as one that a mask cuts
    f32x16v s[TB];       // scores, then softmax terms
    u32x4v pw[KT / 16];  // P in 16 bits
    // LDS places that a lane reads, in a tile's buffer: constant, so that a buffer's turn costs one addition for each
    uint32_t k_at[CH], v_at[FB];
#pragma unroll
    for (int i = 0; i < CH; ++i) k_at[i] = (n * D + k_block<D>(n, 2 * i + g) * 8u) * 2u;
    {
        const uint32_t z = lane & 15u;  // of 16 lanes that read 4 keys of 16 channels
        const uint32_t row_at = 4u * g + (z >> 2), col = 2u * ((lane >> 4) & 1u) + ((z & 3u) >> 1);
#pragma unroll
        for (int f = 0; f < FB; ++f) v_at[f] = (row_at * D + v_block<D>(row_at, 4 * f + col) * 8u + 4u * (z & 1u)) * 2u;
    }
    // S^T = K Q^T
    const auto scores = [&](int32_t t) __attribute__((always_inline)) {
        const uint32_t from = lds_address(&sm_k[t & 3][0]);
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[b][i] = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const uint32_t at = from + k_at[i];
#pragma unroll
            for (int b = 0; b < TB; ++b)
                s[b] = T::mfma32(*reinterpret_cast<lds_u32x4v*>(at + 32u * b * D * 2u), q[i], s[b]);
        }
    };
    // V's channels 32 f + n at the keys 16 st + 4g + 0..3 and 8 more; v_block takes the key's bits 0 and 1 only
    const auto values = [&](uint32_t at, int st) __attribute__((always_inline)) {
        const s16x4v x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4v*>(at + 16u * st * D * 2u));
        const s16x4v x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4v*>(at + (16u * st + 8u) * D * 2u));
        const u32x2v w0 = __builtin_bit_cast(u32x2v, x0), w1 = __builtin_bit_cast(u32x2v, x1);
        return u32x4v{w0[0], w0[1], w1[0], w1[1]};
    };
    // O^T += V^T P^T
    const auto sums = [&](int32_t t) __attribute__((always_inline)) {
        const uint32_t from = lds_address(&sm_v[static_cast<uint32_t>(t) % 5u][0]);
        uint32_t at[FB];
#pragma unroll
        for (int f = 0; f < FB; ++f) at[f] = from + v_at[f];
#pragma unroll
        for (int st = 0; st < KT / 16; ++st)
#pragma unroll
            for (int f = 0; f < FB; ++f) o[f] = P::mfma32(values(at[f], st), pw[st], o[f]);
    };
    const auto seen_of = [&](int32_t t) __attribute__((always_inline)) {  // the tile's keys that this lane's row sees
        const int32_t base = base_of(t);
        const int32_t lo = min(max(see_lo - base, 0), KT), hi = min(max(min(pos + 1, c1) - base, 0), KT);
        const uint64_t below = lo >= 64 ? 0u : ~uint64_t(0) << lo, above = hi >= 64 ? 0u : ~uint64_t(0) << hi;
        uint64_t seen = below & ~above;
        if (!all_there) {
#pragma unroll
            for (int i = 0; i < KT / 8; ++i) {
                const uint32_t key = min(static_cast<uint32_t>(base) + 8u * i, static_cast<uint32_t>(c1) - 1u);
                const int32_t p = load_scalar(table + (key >> shift));
                if (p < 0 || p >= A.cache.n_pages) seen &= ~(uint64_t(0xFF) << (8 * i));
            }
        }
        return seen;
    };
    // scores to P; the sums follow the reference
    const auto softmax = [&](int32_t t) __attribute__((always_inline)) {
        if constexpr (kE4m3) {
#pragma unroll
            for (int b = 0; b < TB; ++b)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const f32x4v ks = *reinterpret_cast<const f32x4v*>(&sm_scale[t & 7][0][32 * b + 8 * y + 4 * g]);
#pragma unroll
                    for (int z = 0; z < 4; ++z) s[b][4 * y + z] *= ks[z];
                }
        }
        const int32_t base = base_of(t);
        // tiles end where a split's keys do, or a row's
        const bool whole = base >= wlast_row.lo && base + KT <= wfirst_row.hi && all_there;
        uint64_t seen = ~uint64_t(0);
        if (!whole) {
            seen = seen_of(t);
#pragma unroll
            for (int b = 0; b < TB; ++b) {
                const uint32_t bits = static_cast<uint32_t>(seen >> (32 * b)) >> (4u * g);
#pragma unroll
                for (int i = 0; i < 16; ++i) s[b][i] = (bits >> (8 * (i / 4) + i % 4)) & 1u ? s[b][i] : -INFINITY;
            }
        }
        float top = -INFINITY;
        if constexpr (kScaled) {
#pragma unroll
            for (int b = 0; b < TB; ++b)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const f32x4v by = *reinterpret_cast<const f32x4v*>(&sm_scale[t & 7][2][32 * b + 8 * y + 4 * g]);
#pragma unroll
                    for (int z = 0; z < 4; ++z) top = fmaxf(top, __builtin_fmaf(s[b][4 * y + z], c, by[z]));
                }
            top = max32(top);
        } else {
#pragma unroll
            for (int b = 0; b < TB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
            top = max32(top) * c;
        }
        if (__any(top > m + kSlack)) {
            const float m_new = fmaxf(m, top);
            const float nb_new = m_new == -INFINITY ? 0.0f : kShift - m_new;
            const float alpha = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(nb_new - nb);
            l *= alpha;
#pragma unroll
            for (int f = 0; f < FB; ++f)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[f][i] *= alpha;
            m = m_new;
            nb = nb_new;
        }
        float part[2] = {0.0f, 0.0f};
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                s[b][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[b][i], c, nb));
                part[i & 1] += s[b][i];
            }
        l += part[0] + part[1];
        if constexpr (kE4m3) {
#pragma unroll
            for (int b = 0; b < TB; ++b)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const f32x4v vs = *reinterpret_cast<const f32x4v*>(&sm_scale[t & 7][1][32 * b + 8 * y + 4 * g]);
#pragma unroll
                    for (int z = 0; z < 4; ++z) s[b][4 * y + z] *= vs[z];
                }
            if (!whole) {  // 0 * NaN
#pragma unroll
                for (int b = 0; b < TB; ++b) {
                    const uint32_t bits = static_cast<uint32_t>(seen >> (32 * b)) >> (4u * g);
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[b][i] = (bits >> (8 * (i / 4) + i % 4)) & 1u ? s[b][i] : 0.0f;
                }
            }
        }
#pragma unroll
        for (int st = 0; st < KT / 16; ++st)
#pragma unroll
            for (int j = 0; j < 4; ++j) pw[st][j] = P::pack(s[st / 2][8 * (st % 2) + 2 * j], s[st / 2][8 * (st % 2) + 2 * j + 1]);
    };
    // the end of a phase: what it wrote to LDS is there, and nothing moves across
    const auto phase = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
        __builtin_amdgcn_sched_barrier(0);
    };

    // Two halves of the workgroup, a wave of each on every SIMD, take turns: while one does the products of its turn t
    // (the scores of tile t + 1, the sums of tile t), the other does the softmax of its own and brings tiles.  A tile that is
    // asked for in turn t is first read in turn t + 3.
    if (n_tiles > 0) {
        // e4m3 has a tile in registers between, and scales a turn behind for each step
        constexpr int kLead = kE4m3 ? 1 : 0;
        Blocks blocks;
        float scale = 0.0f;
        int32_t scale_page = -1;
        const Sources f0 = sources_of(0, ask_pages(0)), f1 = sources_of(1, ask_pages(1)), f2 = sources_of(2, ask_pages(2));
        if constexpr (kE4m3) {
            const Blocks b0 = ask(f0), b1 = ask(f1), b2 = ask(f2);
            blocks = ask(sources_of(3, ask_pages(3)));
            put_scale(0, ask_scale(0, ask_scale_page(0)));
            scale = ask_scale(1, ask_scale_page(1));
            scale_page = ask_scale_page(2);
            put(0, b0);
            put(1, b1);
            put(2, b2);
        } else {
            fetch(0, f0);
            fetch(1, f1);
            fetch(2, f2);
        }
        // of the pages that some row sees: those behind a window may have been freed (2,048 tokens with a window of 1,001, 32
        // heads over 8 of 64, pages of 16: 32.1 us, and 42.1 where a page before the first seen key counted as missing)
        bool bad = false;
        for (uint32_t i = (static_cast<uint32_t>(max(c0, span.lo)) >> shift) + tid; i <= static_cast<uint32_t>(c1 - 1) >> shift; i += kThreads) {
            const int32_t p = table[i];
            bad |= p < 0 || p >= A.cache.n_pages;
        }
        all_there = !__syncthreads_or(bad);
        if constexpr (!kE4m3) wait_loads<0>();
        Pages pages = ask_pages(3 + kLead);
        phase();
        // softmax of tile t, and tile b brought; its pages were asked for a turn before, and its addresses made among the
        // products, where a wave has instructions to spare.  Tiles past the last are brought too, and not read.
        const auto softmax_and_bring = [&](int32_t t, int32_t b, const Sources& from) __attribute__((always_inline)) {
            pages = ask_pages(b + 1 + kLead);
            softmax(t);
            if constexpr (kE4m3) {
                put_scale(b - 2, scale);
                scale = ask_scale(b - 1, scale_page);
                scale_page = ask_scale_page(b);
                put(b, blocks);
                blocks = ask(from);
            } else {
                fetch(b, from);
            }
        };
        if (kTurns && wave >= kWaves / 2) phase();
        Sources from = sources_of(3 + kLead, pages);
        scores(0);
        phase();
        softmax_and_bring(0, 3, from);
        phase();
        // The loop's place in the 32 bytes that an instruction fetch takes: of the eight this is as good as any where an
        // edit before it moves the loop by 4 bytes (0.3 to 2% between them; 2,048 tokens with a window of 4,090 145.4 us
        // here and 148.3 two places on).
        asm volatile(".p2align 5\n\t.rept 6\n\ts_nop 0\n\t.endr");
        for (int32_t t = 0; t + 1 < n_tiles; ++t) {
            __builtin_amdgcn_s_setprio(1);  // products first: they leave the other half enough of the issue slots
            from = sources_of(t + 4 + kLead, pages);
            scores(t + 1);
            sums(t);
            products_in_order<CH * TB, KT / 16 * FB>();
            if constexpr (!kE4m3) {  // tile t + 2 is there when both halves are past this; of tile t + 3 nothing is needed yet
                __builtin_amdgcn_sched_barrier(0);
                wait_loads<2 * NL>();
            }
            __builtin_amdgcn_s_setprio(0);
            phase();
            softmax_and_bring(t + 1, t + 4, from);
            phase();
        }
        sums(n_tiles - 1);
        if constexpr (!kE4m3) wait_loads<0>();
        if (kTurns && wave < kWaves / 2) phase();
    }

    // A NaN in the sums may be there by right, or come from 0 * infinity or 0 * NaN of a value that its row's mask hides:
    // the keys again, tile by tile, with infinities and NaN counted for the rows that see them and zeros in their places.
    bool nan = false;
#pragma unroll
    for (int f = 0; f < FB; ++f)
#pragma unroll
        for (int i = 0; i < 16; ++i) nan |= o[f][i] != o[f][i];
    if (__builtin_expect(__syncthreads_or(nan), 0)) {
        m = -INFINITY;
        nb = l = 0.0f;
#pragma unroll
        for (int f = 0; f < FB; ++f)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[f][i] = 0.0f;
#pragma unroll 1
        for (int32_t t = 0; t < n_tiles; ++t) {
            const Sources from = sources_of(t, ask_pages(t));
            if constexpr (kE4m3) {
                put(t, ask(from));
                put_scale(t, ask_scale(t, ask_scale_page(t)));
            } else {
                fetch(t, from);
                wait_loads<0>();
            }
            phase();
            {
                scores(t);
                softmax(t);
                const uint64_t seen = seen_of(t);
                const uint32_t at_v = lds_address(&sm_v[static_cast<uint32_t>(t) % 5u][0]);
#pragma unroll
                for (int st = 0; st < KT / 16; ++st) {
                    const uint32_t bits = static_cast<uint32_t>(seen >> (16 * st + 4u * g));  // keys 0..3 and 8..11 of these
                    u32x4v one;
#pragma unroll
                    for (int w = 0; w < 4; ++w) one[w] = P::ones((bits >> (8 * (w / 2) + 2 * (w % 2))) & 3u);
#pragma unroll
                    for (int f = 0; f < FB; ++f) {
                        u32x4v a = values(at_v + v_at[f], st), up, down;
                        f32x16v zero;
#pragma unroll
                        for (int i = 0; i < 16; ++i) zero[i] = 0.0f;
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            up[w] = P::not_below(a[w]);
                            down[w] = P::not_above(a[w]);
                            a[w] &= ~P::nonfinite(a[w]);
                        }
                        const f32x16v n_up = P::mfma32(up, one, zero);
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[f][i] += n_up[i] > 0.0f ? INFINITY : 0.0f;
                        const f32x16v n_down = P::mfma32(down, one, zero);
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[f][i] += n_down[i] > 0.0f ? -INFINITY : 0.0f;
                        o[f] = P::mfma32(a, pw[st], o[f]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
            phase();
        }
    }

    l = sum32(l);
    if (!alive || wrow0 + n >= rows) return;
    const uint32_t q_heads = heads * A.group;
    const uint64_t flat = static_cast<uint64_t>(tok) * q_heads + head;
    if (divided) {
        const uint64_t at = static_cast<uint64_t>(split) * A.n_tok * q_heads + flat;
        float* dst = A.part_o + at * D + 4 * g;
#pragma unroll
        for (int f = 0; f < FB; ++f)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                *reinterpret_cast<f32x4v*>(dst + 32 * f + 8 * y) =
                    f32x4v{o[f][4 * y], o[f][4 * y + 1], o[f][4 * y + 2], o[f][4 * y + 3]};
        if (g == 0) *reinterpret_cast<f32x2v*>(A.part_ml + at * 2) = f32x2v{m == -INFINITY ? m : -nb, l};
        return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint8_t* dst = A.out + (tok * A.out_tok + head * A.out_head + 4 * g) * 2;
#pragma unroll
    for (int f = 0; f < FB; ++f)
#pragma unroll
        for (int y = 0; y < 4; ++y)
            *reinterpret_cast<u32x2v*>(dst + (32 * f + 8 * y) * 2) =
                u32x2v{T::pack(o[f][4 * y] * inv, o[f][4 * y + 1] * inv), T::pack(o[f][4 * y + 2] * inv, o[f][4 * y + 3] * inv)};
    if (A.lse && g == 0) A.lse[flat] = l == 0.0f ? -INFINITY : (__log2f(l) - nb) * 0.69314718055994531f;
}

template <class T, int D, bool kE4m3, uint32_t kRows>
hipError_t tile_one(const AttentionArgs& a, hipStream_t stream) {
    constexpr int kWaves = kRows / 32;
    const dim3 grid(tile_count<kRows>(a) * a.cache.n_kv_heads, a.n_split);
    hipLaunchKernelGGL((paged_tile_kernel<T, D, kE4m3, kWaves>), grid, dim3(kWaves * 64), 0, stream, a);
    return hipGetLastError();
}

template <class T, bool kE4m3>
hipError_t tile_dim(const AttentionArgs& a, uint32_t dim, hipStream_t stream) {
    switch (dim) {
        case 64: return tile_one<T, 64, kE4m3, kHalfTile>(a, stream);
        case 128: 
            return a.of_tile == kFullTile ? tile_one<T, 128, kE4m3, kFullTile>(a, stream)
                                          : tile_one<T, 128, kE4m3, kHalfTile>(a, stream);
        default: return tile_one<T, 256, kE4m3, kHalfTile>(a, stream);
    }
}

}  // namespace

hipError_t launch_paged_tile(const AttentionArgs& a, uint32_t dim, uint32_t type, bool e4m3, hipStream_t stream) {
    if (type == ENGRAM_BF16) return e4m3 ? tile_dim<Bf16, true>(a, dim, stream) : tile_dim<Bf16, false>(a, dim, stream);
    return e4m3 ? tile_dim<F16, true>(a, dim, stream) : tile_dim<F16, false>(a, dim, stream);
}

}  // namespace engram
