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
// Mapping (gfx950, wave64): a workgroup takes kWaves * 32 rows of one KV head,
// and one split of their keys; each wave holds 32 rows' q, scores and sums in
// registers.  K and V go through LDS, a tile of KT keys at a time, in two
// buffers: the next tile is requested into registers before the products of
// this one and written to LDS after them, one barrier a tile.  Registers in
// between let the rows of absent keys be zeroed and e4m3 codes be decoded on
// the way.
//   * S^T = K Q^T on 32x32x16 MFMA: a lane holds a row and 16 of 32 keys, so
//     the maximum and sum of a row need one exchange between a wave's halves,
//     and the scores are the second product's B operand as they stand: P never
//     changes lanes.
//   * O^T = V^T P^T: V lies in LDS as it lies in memory; the transposing LDS
//     reads give four keys of a channel to a lane.
//   * 16-byte blocks of a key's row are swapped within its LDS row (K by the
//     key's low bits, V by two of them), so that neither kind of read has two
//     lanes on one bank.
// P is rounded once to 16 bits (bf16: half a step is 2^-9 of each p; its
// average over the keys adds to the output about what the output's own
// rounding does).  Twice the digits, as in paged_rows.hip, would cost half as
// many products again, and here the products are what is waited for.
//
// What a row does not see: scores of hidden keys become -inf before the
// maximum; keys that no row sees (past the end, before the window, on a page
// outside the pool) have zeros for V.  Where a tile that only some rows see
// in full holds infinities or NaN in V, they are replaced by zeros too, and
// counted for the rows that see them by two more products, of ones (not below
// +inf, not above -inf), so that no row meets a value that its mask hides.
#include <type_traits>

#include "paged_attention.h"

namespace engram {
namespace {

typedef short s16x4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4v lds_s16x4v;

// Block (16 bytes of 16-bit channels) of a key's LDS row where channel block c lies.
template <int D>
__device__ __forceinline__ uint32_t k_block(uint32_t key, uint32_t c) {
    return D == 64 ? c ^ ((key >> 1) & 7u) : c ^ (key & 15u);
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

// eight e4m3 codes as 16-bit numbers
template <class T>
__device__ __forceinline__ u32x4v widen(u32x2v w) {
    return u32x4v{T::template from_e4m3<false>(w[0]), T::template from_e4m3<true>(w[0]), T::template from_e4m3<false>(w[1]),
                  T::template from_e4m3<true>(w[1])};
}

template <class T, int D, bool kE4m3, int kWaves>
__global__ __launch_bounds__(kWaves * 64) __attribute__((amdgpu_waves_per_eu(2, 2))) void paged_tile_kernel(
    const AttentionArgs A) {
    constexpr uint32_t kRows = kWaves * 32u, kThreads = kWaves * 64u;
    constexpr int KT = D == 256 ? 32 : 64;          // keys of a tile
    constexpr int TB = KT / 32;                     // blocks of 32 keys
    constexpr int CB = D / 8;                       // 16-byte blocks of a row
    constexpr int CH = D / 16;                      // MFMA steps of a score
    constexpr int FB = D / 32;                      // blocks of 32 channels
    constexpr int NL = KT * CB / int(kThreads);     // blocks of K (and of V) that a thread brings
    static_assert(NL >= 1 && NL * int(kThreads) == KT * CB, "every thread brings the same");
    using P = std::conditional_t<kE4m3, Bf16, T>;   // P and V's type; e4m3 codes are exact in both types
    using Raw = std::conditional_t<kE4m3, u32x2v, u32x4v>;
    constexpr uint32_t ES = kE4m3 ? 1 : 2;
    constexpr float kSlack = P::kSlack, kShift = P::kShift;

    __shared__ __attribute__((aligned(1024))) uint16_t sm_k[3][KT * D];
    __shared__ __attribute__((aligned(1024))) uint16_t sm_v[4][KT * D];
    __shared__ __attribute__((aligned(16))) float sm_scale[4][2][kE4m3 ? KT : 4];
    __shared__ int32_t sm_page[8][KT];       // page of each key, -1: absent
    __shared__ uint64_t sm_there[8];         // keys that are there, by bit

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
    const Span first_row = span_of(A, req, row0, 1), last_row = span_of(A, req, row0 + n_rows - 1u, 1);

    // this split's keys [c0, c1)
    const int32_t base0 = span.lo & ~(kTileAlign - 1);
    const uint32_t split = blockIdx.y;
    const bool divided = A.split_tokens != 0 && span.hi > base0 && static_cast<uint32_t>(span.hi - base0) > A.split_tokens;
    int32_t c0 = base0, c1 = max(span.hi, base0);
    if (divided) {
        const int64_t at = static_cast<int64_t>(base0) + static_cast<int64_t>(split) * A.split_tokens;
        if (at >= span.hi) return;
        c0 = static_cast<int32_t>(at);
        c1 = static_cast<int32_t>(min(at + A.split_tokens, static_cast<int64_t>(span.hi)));
    } else if (split != 0) {
        return;
    }
    const int32_t n_tiles = (c1 - c0 + KT - 1) / KT;

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
    // Pages (wave 0): the table's entry for the tile's key `lane`, and, when it has come, what to make of it (-1 where no row
    // sees the key or there is no such page).
    const auto key_in = [&](int32_t t) {
        const int64_t key = static_cast<int64_t>(c0) + static_cast<int64_t>(t) * KT + lane;
        return key < c1 && key >= span.lo && lane < KT;
    };
    const auto ask_page = [&](int32_t t) {
        return key_in(t) ? table[static_cast<uint32_t>(c0 + t * KT + static_cast<int32_t>(lane)) >> shift] : -1;
    };
    const auto tell_page = [&](int32_t t, int32_t page) {
        const bool ok = key_in(t) && page >= 0 && page < A.cache.n_pages;
        if (lane < KT) sm_page[t & 7][lane] = ok ? page : -1;
        const uint64_t there = __ballot(ok);
        if (lane == 0) sm_there[t & 7] = there;
    };

    struct Pages {
        int32_t of[NL];  // of the thread's blocks
        int32_t scale;
    };
    const auto pages_of = [&](int32_t t) {
        Pages r;
#pragma unroll
        for (int i = 0; i < NL; ++i) r.of[i] = sm_page[t & 7][(i * kThreads + tid) / CB];
        r.scale = kE4m3 ? sm_page[t & 7][tid % KT] : 0;
        return r;
    };
    struct Blocks {
        Raw k[NL], v[NL];
        float scale;
        uint32_t absent;  // bit i: block i belongs to an absent key
    };
    const auto ask = [&](int32_t t, const Pages& pg) {
        Blocks r;
        r.absent = 0;
        r.scale = 0.0f;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const uint32_t at = i * kThreads + tid, row_at = at / CB, cb = at % CB;
            const int32_t page = pg.of[i];
            if (page < 0) r.absent |= 1u << i;
            const uint32_t in = ((static_cast<uint32_t>(base_of(t)) + row_at) & in_page) * D + cb * 8u;
            const int64_t p0 = max(page, 0);
            r.k[i] = *reinterpret_cast<const Raw*>(kh + (p0 * A.cache.k_page_stride + in) * ES);
            r.v[i] = *reinterpret_cast<const Raw*>(vh + (p0 * A.cache.v_page_stride + in) * ES);
        }
        if constexpr (kE4m3) {
            if (tid < 2u * KT) {
                const uint32_t row_at = tid % KT;
                const int32_t page = pg.scale;
                const uint32_t in = (static_cast<uint32_t>(base_of(t)) + row_at) & in_page;
                const float* from = tid < KT ? A.cache.k_scale : A.cache.v_scale;
                r.scale = from[((static_cast<int64_t>(max(page, 0)) * heads + h) << shift) + in];
                if (page < 0) r.scale = 0.0f;
            }
        }
        return r;
    };
    const auto put = [&](int32_t t, const Blocks& r) {
        const uint32_t kt = static_cast<uint32_t>(t) % 3u;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const uint32_t at = i * kThreads + tid, row_at = at / CB, cb = at % CB;
            u32x4v kw, vw;
            if constexpr (kE4m3) {
                kw = widen<T>(r.k[i]);
                vw = widen<P>(r.v[i]);
            } else {
                kw = r.k[i];
                vw = r.v[i];
            }
            if ((r.absent >> i) & 1u) vw = u32x4v{0u, 0u, 0u, 0u};
            *reinterpret_cast<u32x4v*>(&sm_k[kt][row_at * D + k_block<D>(row_at, cb) * 8u]) = kw;
            *reinterpret_cast<u32x4v*>(&sm_v[t & 3][row_at * D + v_block<D>(row_at, cb) * 8u]) = vw;
        }
        if constexpr (kE4m3) {
            if (tid < 2u * KT) sm_scale[t & 3][tid / KT][tid % KT] = r.scale;
        }
    };

    f32x16v s[TB];       // scores, then softmax terms
    u32x4v pw[KT / 16];  // P in 16 bits
    // S^T = K Q^T
    const auto scores = [&](int32_t t) {
        const uint16_t* kb = sm_k[static_cast<uint32_t>(t) % 3u];
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[b][i] = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int b = 0; b < TB; ++b) {
                const u32x4v a = *reinterpret_cast<const u32x4v*>(&kb[(32 * b + n) * D + k_block<D>(n, 2 * i + g) * 8u]);
                s[b] = T::mfma32(a, q[i], s[b]);
            }
    };
    // V's channels 32 f + n at the keys 16 st + 4g + 0..3 and 8 more; v_block takes the key's bits 0 and 1 only
    const auto values = [&](int32_t t, int st, int f) {
        const uint16_t* vb = sm_v[t & 3];
        const uint32_t z = lane & 15u;  // of 16 lanes that read 4 keys of 16 channels
        const uint32_t vrow = 4u * g + (z >> 2), vcol = 2u * ((lane >> 4) & 1u) + ((z & 3u) >> 1);
        const uint32_t at = (16 * st + vrow) * D + v_block<D>(vrow, 4 * f + vcol) * 8u + 4u * (z & 1u);
        const s16x4v x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4v*)&vb[at]);
        const s16x4v x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4v*)&vb[at + 8 * D]);
        const u32x2v w0 = __builtin_bit_cast(u32x2v, x0), w1 = __builtin_bit_cast(u32x2v, x1);
        return u32x4v{w0[0], w0[1], w1[0], w1[1]};
    };
    // O^T += V^T P^T
    const auto sums = [&](int32_t t) {
#pragma unroll
        for (int st = 0; st < KT / 16; ++st)
#pragma unroll
            for (int f = 0; f < FB; ++f) o[f] = P::mfma32(values(t, st, f), pw[st], o[f]);
    };
    constexpr uint64_t kAll = KT == 64 ? ~uint64_t(0) : (uint64_t(1) << (KT & 63)) - 1u;
    const auto seen_of = [&](int32_t t, uint64_t there) {  // the tile's keys that this lane's row sees
        const int32_t base = base_of(t);
        const int32_t lo = min(max(see_lo - base, 0), KT), hi = min(max(pos + 1 - base, 0), KT);
        const uint64_t below = lo >= 64 ? 0u : ~uint64_t(0) << lo, above = hi >= 64 ? 0u : ~uint64_t(0) << hi;
        return there & below & ~above;
    };
    // scores to P; the sums follow the reference
    const auto softmax = [&](int32_t t, uint64_t there) {
        if constexpr (kE4m3) {
#pragma unroll
            for (int b = 0; b < TB; ++b)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const f32x4v ks = *reinterpret_cast<const f32x4v*>(&sm_scale[t & 3][0][32 * b + 8 * y + 4 * g]);
#pragma unroll
                    for (int z = 0; z < 4; ++z) s[b][4 * y + z] *= ks[z];
                }
        }
        const int32_t base = base_of(t);
        const bool whole = base >= wlast_row.lo && base + KT <= wfirst_row.hi && there == kAll;
        uint64_t seen = kAll;
        if (!whole) {
            seen = seen_of(t, there);
#pragma unroll
            for (int b = 0; b < TB; ++b) {
                const uint32_t bits = static_cast<uint32_t>(seen >> (32 * b)) >> (4u * g);
#pragma unroll
                for (int i = 0; i < 16; ++i) s[b][i] = (bits >> (8 * (i / 4) + i % 4)) & 1u ? s[b][i] : -INFINITY;
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < TB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
        top = max32(top) * c;
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
                    const f32x4v vs = *reinterpret_cast<const f32x4v*>(&sm_scale[t & 3][1][32 * b + 8 * y + 4 * g]);
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
    const auto there_of = [&](int32_t t) { return sm_there[t & 7]; };
    const auto same = [](uint64_t x) {  // for all lanes
        const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x));
        const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x >> 32));
        return static_cast<uint64_t>(hi) << 32 | lo;
    };
    // the end of a phase: what it wrote to LDS is there, and nothing moves across
    const auto phase = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
        __builtin_amdgcn_sched_barrier(0);
    };

    // Two halves of the workgroup, a wave of each on every SIMD, take turns: while one does the products of its turn t
    // (the scores of tile t + 1, the sums of tile t), the other does the softmax of its own and brings tiles.  A tile that is
    // put in turn t is first read in turn t + 2, by when both halves have put their blocks.
    if (n_tiles > 0) {
        Blocks blocks;
        Pages pages;
        int32_t entry = -1;  // of a tile whose pages are not yet told
        if (wave == 0) {
            int32_t e[5];
#pragma unroll
            for (int t = 0; t < 5; ++t) e[t] = ask_page(t);
            entry = ask_page(5);
#pragma unroll
            for (int t = 0; t < 5; ++t) tell_page(t, e[t]);
        }
        phase();
        {
            const Blocks b0 = ask(0, pages_of(0)), b1 = ask(1, pages_of(1));
            blocks = ask(2, pages_of(2));
            pages = pages_of(3);
            put(0, b0);
            put(1, b1);
        }
        uint64_t there = there_of(0);  // each of these is read a turn before it is used
        phase();
        const auto bring = [&](int32_t t) {  // tile t into LDS, the next into registers
            if (t >= n_tiles) return;
            put(t, blocks);
            if (t + 1 < n_tiles) {
                blocks = ask(t + 1, pages);
                pages = pages_of(t + 2);
            }
            if (wave == 0) {
                tell_page(t + 3, entry);
                entry = ask_page(t + 4);
            }
        };
        if (wave >= kWaves / 2) phase();
        scores(0);
        phase();
        uint64_t now = same(there);
        there = there_of(1);
        softmax(0, now);
        bring(2);
        phase();
        for (int32_t t = 0; t + 1 < n_tiles; ++t) {
            scores(t + 1);
            sums(t);
            products_in_order<CH * TB, KT / 16 * FB>();
            phase();
            now = same(there);
            there = there_of(t + 2);
            softmax(t + 1, now);
            bring(t + 3);
            phase();
        }
        sums(n_tiles - 1);
        if (wave < kWaves / 2) phase();
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
            if (wave == 0) tell_page(t, ask_page(t));
            phase();
            put(t, ask(t, pages_of(t)));
            phase();
            {
                scores(t);
                const uint64_t there = same(there_of(t));
                softmax(t, there);
                const uint64_t seen = seen_of(t, there);
#pragma unroll
                for (int st = 0; st < KT / 16; ++st) {
                    const uint32_t bits = static_cast<uint32_t>(seen >> (16 * st + 4u * g));  // keys 0..3 and 8..11 of these
                    u32x4v one;
#pragma unroll
                    for (int w = 0; w < 4; ++w) one[w] = P::ones((bits >> (8 * (w / 2) + 2 * (w % 2))) & 3u);
#pragma unroll
                    for (int f = 0; f < FB; ++f) {
                        u32x4v a = values(t, st, f), up, down;
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

template <class T, int D, bool kE4m3>
hipError_t tile_one(const AttentionArgs& a, hipStream_t stream) {
    constexpr int kWaves = kTileRows / 32;
    const dim3 grid(tile_count<kTileRows>(a) * a.cache.n_kv_heads, a.n_split);
    hipLaunchKernelGGL((paged_tile_kernel<T, D, kE4m3, kWaves>), grid, dim3(kWaves * 64), 0, stream, a);
    return hipGetLastError();
}

template <class T, bool kE4m3>
hipError_t tile_dim(const AttentionArgs& a, uint32_t dim, hipStream_t stream) {
    switch (dim) {
        case 64: return tile_one<T, 64, kE4m3>(a, stream);
        case 128: return tile_one<T, 128, kE4m3>(a, stream);
        default: return tile_one<T, 256, kE4m3>(a, stream);
    }
}

}  // namespace

hipError_t launch_paged_tile(const AttentionArgs& a, uint32_t dim, uint32_t type, bool e4m3, hipStream_t stream) {
    if (type == ENGRAM_BF16) return e4m3 ? tile_dim<Bf16, true>(a, dim, stream) : tile_dim<Bf16, false>(a, dim, stream);
    return e4m3 ? tile_dim<F16, true>(a, dim, stream) : tile_dim<F16, false>(a, dim, stream);
}

}  // namespace engram
