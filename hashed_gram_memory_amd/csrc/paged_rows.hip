// Paged attention for few rows per request: single tokens and short runs.
//
//     o = sum_j p_j v_j / sum_j p_j,   p_j = exp2(s_j - max s),
//     s_j = scale * log2(e) * (q . k_j)
//
// One pass over the keys with a running maximum and sum.  The work is the
// reading of K and V, each byte once per KV head: HBM-bound.
//
// Mapping (gfx950, wave64): a workgroup takes one tile of 16 rows of one KV
// head and one split of its keys; its 4 waves take 32 keys each in turn,
// straight from global memory into registers, and join through LDS at the end.
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
// Keys that only some rows see keep their V; where such a step holds an
// infinity or NaN the product is done row by row, so that no row sees a
// value that its mask hides.
#include <type_traits>

#include "paged_attention.h"

namespace engram {
namespace {

constexpr uint32_t kRows = kRowsTile;
constexpr uint32_t kStep = 32;      // keys of a wave's step
constexpr uint32_t kWaves = 4;
constexpr uint32_t kPages = 1024;   // page numbers held in LDS at a time

template <int kBytes>
struct Words {
    uint32_t w[kBytes / 4];
};
template <int kBytes>
__device__ __forceinline__ Words<kBytes> load_words(const uint8_t* p) {
    Words<kBytes> r;
    if constexpr (kBytes == 4) {
        r.w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kBytes == 8) {
        const u32x2v x = *reinterpret_cast<const u32x2v*>(p);
        r.w[0] = x[0];
        r.w[1] = x[1];
    } else {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) {
            const u32x4v x = *reinterpret_cast<const u32x4v*>(p + 16 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) r.w[4 * i + j] = x[j];
        }
    }
    return r;
}

template <class T, int D, bool kE4m3>
__global__ __launch_bounds__(256) void paged_rows_kernel(const AttentionArgs A) {
    constexpr int EPL = D / 16;              // channels of V in a lane
    constexpr int CH = D / 32;               // MFMA steps of a score
    constexpr int ES = kE4m3 ? 1 : 2;        // bytes of an element
    constexpr int OP = D + 4;                // padded row of partial sums
    // P and V's type.  An e4m3 V is exact in bf16, whose range holds p * scale.
    using P = std::conditional_t<kE4m3, Bf16, T>;
    __shared__ int32_t sm_page[kPages];
    __shared__ float sm_o[kWaves * kRows * OP];
    __shared__ float sm_m[kWaves][kRows], sm_l[kWaves][kRows];

    const uint32_t heads = A.cache.n_kv_heads;
    const uint32_t tile_at = blockIdx.x / heads, h = blockIdx.x - tile_at * heads;
    const Tile tile = find_tile<kRows>(A, tile_at);
    if (!tile.live) return;
    const Request req = request_of(A, tile.b);
    const uint32_t rows = req.q_len * A.group;
    if (tile.row0 >= rows || rows < A.min_rows || rows > A.max_rows) return;
    const uint32_t n_rows = min(kRows, rows - tile.row0);
    const Span span = span_of(A, req, tile.row0, n_rows);
    const Span first_row = span_of(A, req, tile.row0, 1), last_row = span_of(A, req, tile.row0 + n_rows - 1u, 1);

    // this split's keys [c0, c1)
    const int32_t base0 = span.lo & ~(kRowsAlign - 1);
    const uint32_t split = blockIdx.y;
    const bool divided = A.split_tokens != 0 && span.hi > base0 &&
                         static_cast<uint32_t>(span.hi - base0) > A.split_tokens;
    int32_t c0 = base0, c1 = max(span.hi, base0);
    if (divided) {
        const int64_t at = static_cast<int64_t>(base0) + static_cast<int64_t>(split) * A.split_tokens;
        if (at >= span.hi) return;
        c0 = static_cast<int32_t>(at);
        c1 = static_cast<int32_t>(min(at + A.split_tokens, static_cast<int64_t>(span.hi)));
    } else if (split != 0) {
        return;
    }

    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t lane = threadIdx.x & 63u, n = lane & 15u, g = lane >> 4;

    // this lane's row (column n of the products)
    const uint32_t row = min(tile.row0 + n, rows - 1u);
    const uint32_t tok = req.q0 + row / A.group, head = h * A.group + row % A.group;
    const int32_t pos = req.kv_len - static_cast<int32_t>(req.q_len) + static_cast<int32_t>(row / A.group);
    const int32_t see_lo = A.window && pos >= static_cast<int32_t>(A.window) ? pos - static_cast<int32_t>(A.window) + 1 : 0;
    u32x4v q[CH];
    {
        const uint8_t* qp = A.q + (tok * A.q_tok + head * A.q_head) * 2;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            // e4m3 keys come 16 channels a load, which orders the channels of a pair of steps
            const int d = kE4m3 ? 64 * (c / 2) + 16 * g + 8 * (c % 2) : 32 * c + 8 * g;
            q[c] = *reinterpret_cast<const u32x4v*>(qp + d * 2);
        }
    }

    float m = -INFINITY, l = 0.0f;
    f32x4v o[EPL];
#pragma unroll
    for (int f = 0; f < EPL; ++f) o[f] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};

    const uint32_t shift = A.cache.page_shift, in_page = (1u << shift) - 1u;
    const int32_t* table = A.table + tile.b * A.table_stride;
    for (int32_t seg = c0; seg < c1;) {
        // page numbers of the next keys into LDS; -1 where there is no such page
        const uint32_t page0 = static_cast<uint32_t>(seg) >> shift;
        const int64_t room = (static_cast<int64_t>(page0) + kPages) << shift;
        const int32_t seg_end = room < c1 ? static_cast<int32_t>(room) : c1;
        const uint32_t n_pages = ((static_cast<uint32_t>(seg_end) - 1u) >> shift) - page0 + 1u;
        if (seg != c0) __syncthreads();
        for (uint32_t i = threadIdx.x; i < n_pages; i += 256u) {
            const int32_t p = table[page0 + i];
            sm_page[i] = p >= 0 && p < A.cache.n_pages ? p : -1;
        }
        __syncthreads();

        for (int32_t base = seg + static_cast<int32_t>(wave * kStep); base < seg_end; base += kStep * kWaves) {
            // K: keys base + n and base + 16 + n
            Words<16> kw[2][ES == 1 ? CH / 2 : CH];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int32_t key = min(base + 16 * t + static_cast<int32_t>(n), seg_end - 1);
                const int32_t page = max(sm_page[(static_cast<uint32_t>(key) >> shift) - page0], 0);
                const uint8_t* p = A.cache.k + (page * A.cache.k_page_stride +
                                                ((static_cast<int64_t>(h) << shift) + (key & in_page)) * D) * ES;
#pragma unroll
                for (int c = 0; c < (ES == 1 ? CH / 2 : CH); ++c)
                    kw[t][c] = load_words<16>(p + (ES == 1 ? 64 * c + 16 * g : (32 * c + 8 * g) * 2));
            }
            // V: keys base + 4g + 0..3 and base + 16 + 4g + 0..3, which are also this lane's scores
            Words<EPL * ES> vw[2][4];
            float ks[2][4], vs[2][4];
            bool there[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int32_t key = base + 16 * t + static_cast<int32_t>(4u * g);
                const int32_t in = min(key, (seg_end - 1) & ~3);
                const int32_t page = sm_page[(static_cast<uint32_t>(in) >> shift) - page0];
                there[t] = page >= 0;
                const int64_t line = (static_cast<int64_t>(h) << shift) + (in & in_page);
                const uint8_t* p = A.cache.v + (max(page, 0) * A.cache.v_page_stride + line * D + n * EPL) * ES;
#pragma unroll
                for (int i = 0; i < 4; ++i) vw[t][i] = load_words<EPL * ES>(p + i * D * ES);
                if constexpr (kE4m3) {
                    const int64_t at = ((static_cast<int64_t>(max(page, 0)) * heads) << shift) + line;
                    const f32x4v a = *reinterpret_cast<const f32x4v*>(A.cache.k_scale + at);
                    const f32x4v b = *reinterpret_cast<const f32x4v*>(A.cache.v_scale + at);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        ks[t][i] = a[i];
                        vs[t][i] = b[i];
                    }
                }
            }

            f32x4v s[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                s[t] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < CH; ++c) {
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

            // every row of the tile sees every key of a whole step; else each row's own keys
            const bool whole = base >= last_row.lo && base + static_cast<int32_t>(kStep) <= min(first_row.hi, c1) &&
                               !__any(!there[0] || !there[1]);
            uint32_t seen = 0xFFu;  // bit 4t + i
            float x[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[t][i] = s[t][i] * A.scale_log2;
                    if constexpr (kE4m3) x[t][i] *= ks[t][i];
                }
            if (!whole) {
                seen = 0;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int32_t key = base + 16 * t + static_cast<int32_t>(4u * g) + i;
                        const bool ok = there[t] && key >= see_lo && key <= pos && key < c1;
                        if (ok) seen |= 1u << (4 * t + i);
                        x[t][i] = ok ? x[t][i] : -INFINITY;
                    }
            }
            float top = -INFINITY;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = fmaxf(top, x[t][i]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m_new = fmaxf(m, top);
            const float ref = m_new == -INFINITY ? 0.0f : m_new;
            if (__any(m_new > m)) {
                const float alpha = __builtin_amdgcn_exp2f(m - ref);
                l *= alpha;
#pragma unroll
                for (int f = 0; f < EPL; ++f)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[f][i] *= alpha;
                m = m_new;
            }
            float p[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[t][i] = __builtin_amdgcn_exp2f((x[t][i] - ref) + P::kShift);
                    l += p[t][i];
                    if constexpr (kE4m3) p[t][i] = (seen >> (4 * t + i)) & 1u ? p[t][i] * vs[t][i] : 0.0f;
                }

            // V rows as 16-bit pairs of channels
            uint32_t v[8][EPL / 2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < EPL / 2; ++e) {
                        if constexpr (kE4m3)
                            v[4 * t + i][e] = (e & 1) ? P::template from_e4m3<true>(vw[t][i].w[e / 2])
                                                      : P::template from_e4m3<false>(vw[t][i].w[e / 2]);
                        else
                            v[4 * t + i][e] = vw[t][i].w[e];
                    }
            bool by_row = false;
            if (!whole) {
                bool odd = false;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    // keys that no row sees
                    const int32_t key = base + 16 * (k / 4) + static_cast<int32_t>(4u * g) + (k % 4);
                    const bool any = there[k / 4] && key >= span.lo && key < c1;
#pragma unroll
                    for (int e = 0; e < EPL / 2; ++e) {
                        v[k][e] = any ? v[k][e] : 0u;
                        odd |= (v[k][e] & P::kExponent) == P::kExponent ||
                               ((v[k][e] >> 16) & P::kExponent) == P::kExponent;
                    }
                }
                by_row = __any(odd);
            }
            if (!by_row) {
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
                        a[w] = __builtin_amdgcn_perm(v[2 * w + 1][f / 2], v[2 * w][f / 2],
                                                     (f & 1) ? 0x07060302u : 0x05040100u);
                    o[f] = P::mfma16(a, ph, o[f]);
                    o[f] = P::mfma16(a, pl, o[f]);
                }
            } else {
                // Row by row: lane (n, g) adds p[key] * V[key][its channels] for the keys that row n sees.
                for (uint32_t k = 0; k < kStep; ++k) {
                    const uint32_t from = ((k & 15u) >> 2) * 16u;
                    const uint32_t at = (k >> 4) * 4u + (k & 3u);
                    float pk = 0.0f;
#pragma unroll
                    for (uint32_t e = 0; e < 8; ++e) {
                        const float other = __shfl(p[e / 4][e % 4], from + n);
                        pk = at == e ? other : pk;
                    }
                    const uint32_t other_seen = static_cast<uint32_t>(__shfl(static_cast<int>(seen), from + n));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < EPL / 2; ++e) {
                            // V[key][D/4 * g + EPL * i + 2e ..]: held by lane 4g + i of the key's group
                            uint32_t w = 0;
#pragma unroll
                            for (uint32_t z = 0; z < 8; ++z) {
                                const uint32_t y = static_cast<uint32_t>(__shfl(static_cast<int>(v[z][e]), from + 4u * g + i));
                                w = at == z ? y : w;
                            }
                            if ((other_seen >> at) & 1u) {
                                o[2 * e][i] = __builtin_fmaf(pk, P::lo(w), o[2 * e][i]);
                                o[2 * e + 1][i] = __builtin_fmaf(pk, P::hi(w), o[2 * e + 1][i]);
                            }
                        }
                }
            }
        }
        seg = seg_end;
    }

    // join the waves
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g == 0) {
        sm_m[wave][n] = m;
        sm_l[wave][n] = l;
    }
    float* mine = sm_o + (wave * kRows + n) * OP + g * (D / 4);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int f = 0; f < EPL; f += 4)
            *reinterpret_cast<f32x4v*>(mine + i * EPL + f) = f32x4v{o[f][i], o[f + 1][i], o[f + 2][i], o[f + 3][i]};
    __syncthreads();

    const uint32_t r = threadIdx.x >> 4, part = threadIdx.x & 15u;  // row, EPL channels of it
    if (r >= n_rows) return;
    float top = -INFINITY;
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) top = fmaxf(top, sm_m[w][r]);
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, acc[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = 0.0f;
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(sm_m[w][r] - ref);
        sum += f * sm_l[w][r];
        const float* src = sm_o + (w * kRows + r) * OP + part * EPL;
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[e] += f * src[e];
    }
    const uint32_t rr = tile.row0 + r;
    const uint32_t out_tok = req.q0 + rr / A.group, out_head = h * A.group + rr % A.group;
    const uint64_t flat = static_cast<uint64_t>(out_tok) * (heads * A.group) + out_head;
    if (divided) {
        const uint64_t at = part_index(A, split, tile.b, h, rr, flat);
        float* dst = A.part_o + at * D + part * EPL;
#pragma unroll
        for (int e = 0; e < EPL; e += 4)
            *reinterpret_cast<f32x4v*>(dst + e) = f32x4v{acc[e], acc[e + 1], acc[e + 2], acc[e + 3]};
        if (part == 0) *reinterpret_cast<f32x2v*>(A.part_ml + at * 2) = f32x2v{top, sum};
        return;
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint32_t w[EPL / 2];
#pragma unroll
    for (int e = 0; e < EPL / 2; ++e) w[e] = T::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    uint32_t* dst = reinterpret_cast<uint32_t*>(A.out + (out_tok * A.out_tok + out_head * A.out_head + part * EPL) * 2);
#pragma unroll
    for (int e = 0; e < EPL / 2; ++e) dst[e] = w[e];
    if (A.lse && part == 0) A.lse[flat] = sum == 0.0f ? -INFINITY : (top + __log2f(sum) - P::kShift) * 0.69314718055994531f;
}

template <class T, int D, bool kE4m3>
hipError_t rows_one(const AttentionArgs& a, hipStream_t stream) {
    const dim3 grid(tile_count<kRows>(a) * a.cache.n_kv_heads, a.n_split);
    hipLaunchKernelGGL((paged_rows_kernel<T, D, kE4m3>), grid, dim3(256), 0, stream, a);
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
