// Host side of the serving calls (head norm + rotation, cache appends, paged
// attention): validation, the split of the keys, launches.  As in
// engram_api.cpp, every argument is checked before anything is launched and
// nothing here synchronises or allocates device memory.
#include <algorithm>
#include <math.h>

#include "engram_internal.h"
#include "paged_attention.h"

using namespace engram;

namespace {

bool good_dim(uint32_t d) { return d == 64 || d == 128 || d == 256; }
bool good_type(uint32_t t) { return t == ENGRAM_BF16 || t == ENGRAM_F16; }
bool of_pages(uint32_t t) { return t == ENGRAM_E4M3_PAGE || t == ENGRAM_I8_PAGE; }  // codes with a scale for each page

// Strides of a [tokens][heads][dim] tensor: whole 16-byte blocks, not negative.
bool good_strides(int64_t tok, int64_t head) {
    constexpr int64_t kMost = int64_t(1) << 40;
    return tok >= 0 && head >= 0 && tok < kMost && head < kMost && tok % 8 == 0 && head % 8 == 0;
}

int check_rotation(uint32_t rotary, uint32_t dim, int64_t n_tok, const int32_t* positions, const double* inv_freq,
                   uint32_t interleaved, float eps) {
    if (rotary % 16 != 0 || rotary > dim || interleaved > 1) return ENGRAM_EINVAL;
    if (!(eps >= 0.0f) || isinf(eps)) return ENGRAM_EINVAL;
    if (rotary && n_tok > 0 && (!positions || !inv_freq || !aligned(positions, 4) || !aligned(inv_freq, 8)))
        return ENGRAM_EINVAL;
    return ENGRAM_OK;
}

int view_of(const engram_kv_cache* c, CacheView* out) {
    if (!c) return ENGRAM_EINVAL;
    const bool coded = c->type == ENGRAM_E4M3 || of_pages(c->type);
    if (!good_type(c->type) && !coded) return ENGRAM_EUNSUPPORTED;
    if (!good_dim(c->head_dim)) return ENGRAM_EUNSUPPORTED;
    const uint32_t p = c->page_size;
    if (p < 8 || p > 1024 || (p & (p - 1)) != 0) return ENGRAM_EUNSUPPORTED;
    if (c->n_kv_heads == 0 || c->n_kv_heads > 65535 || c->n_pages <= 0 || c->n_pages > INT32_MAX) return ENGRAM_ERANGE;
    if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return ENGRAM_EINVAL;
    const int64_t inner = int64_t(c->n_kv_heads) * p * c->head_dim;
    const int64_t most = INT64_MAX / 2 / c->n_pages;
    for (int64_t s : {c->k_page_stride, c->v_page_stride})
        if (s < inner || s % 16 != 0 || s > most) return ENGRAM_EINVAL;
    if (coded && (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16)))
        return ENGRAM_EINVAL;
    out->k = static_cast<uint8_t*>(c->k);
    out->v = static_cast<uint8_t*>(c->v);
    out->k_scale = c->k_scale;
    out->v_scale = c->v_scale;
    out->k_page_stride = c->k_page_stride;
    out->v_page_stride = c->v_page_stride;
    out->n_pages = c->n_pages;
    out->n_kv_heads = c->n_kv_heads;
    out->page_shift = static_cast<uint32_t>(__builtin_ctz(p));
    return ENGRAM_OK;
}

// How one launch divides its keys.
struct Split {
    uint32_t tokens, n;  // keys of a split (0: all), splits; at most
    double us;           // what it is expected to take
};

// Many rows (paged_tile.hip).  A CU holds one workgroup of a full tile, two of
// half tiles (head_dim 256: one), so a launch takes groups * n / at_once rounds
// of a split's keys (of equal workgroups, one to a CU: the last is a whole one), and joining writes and reads n fp32 rows for each
// row; of up to 32 splits the one with the least of both.  A round took, for
// each key, 0.021, 0.036 and 0.036 us in half tiles of head_dim 64, 128 and 256
// and 0.032 us in full tiles of 128 (2,048 tokens over 32,768 keys, bf16), and
// about 5 us to begin and end.
Split split_tiles(double groups, bool equal, int64_t most_keys, uint64_t rows, uint32_t dim, uint32_t of_tile) {
    const double key_us = of_tile == kFullTile ? 0.032 : dim == 64 ? 0.021 : 0.036, join_us = rows * dim * 8.0 / 4e6;
    const double at_once = of_tile == kFullTile || dim == 256 ? 256 : 512;
    Split s = {0u, 1u, 0.0};
    most_keys = std::max<int64_t>(most_keys, 1);  // a table of no pages
    for (uint32_t n = 1; n <= 32; ++n) {
        const int64_t tokens = ((most_keys + n - 1) / n + 63) / 64 * 64;
        if (n > 1 && tokens < kLeastSplit) break;
        const double of_all = groups * n / at_once;
        const double rounds = equal && at_once == 256 ? ceil(of_all) : std::max(of_all, 1.0);
        const double us = rounds * (tokens * key_us + 5) + (n > 1 ? 6 + n * join_us : 0);
        if (n == 1 || us < s.us)
            s = {n > 1 ? static_cast<uint32_t>(tokens) : 0u, static_cast<uint32_t>((most_keys + tokens - 1) / tokens), us};
    }
    if (s.n <= 1) s.tokens = 0, s.n = 1;
    return s;
}

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Rows of a request and KV head up to which paged_rows.hip takes it, which
// reads the keys once for every 16 rows: 8 requests over 8,192 keys (8 KV heads,
// head_dim 128, bf16) take 59 us there with 32 rows each and 131 with 40, and 94
// in paged_tile.hip with 64.
constexpr uint32_t kFewRows = 32;

// A call's launches: the requests of few rows, those of many, or both.
struct Launches {
    AttentionArgs few, many;
    bool any_few, any_many;
    size_t few_o, few_ml, few_job, many_o, many_ml;  // bytes of their parts
};

// Checks a description and fills the kernels' arguments (without the workspace).
int attention_args(const engram_attention_desc* d, Launches* out, size_t* ws_bytes) {
    AttentionArgs* const a = &out->few;
    if (!d) return ENGRAM_EINVAL;
    CacheView view;
    const int st = view_of(d->cache, &view);
    if (st != ENGRAM_OK) return st;
    if (!good_type(d->type)) return ENGRAM_EUNSUPPORTED;
    if (good_type(d->cache->type) && d->cache->type != d->type) return ENGRAM_EUNSUPPORTED;
    if (d->n_seq < 0 || d->n_tok < 0 || d->table_width < 0 || d->max_q_len < 0 || d->window < 0) return ENGRAM_EINVAL;
    if (d->n_q_heads == 0 || d->n_q_heads > 65535 || d->n_q_heads % d->cache->n_kv_heads != 0) return ENGRAM_EINVAL;
    if (d->reserved0 != 0) return ENGRAM_EINVAL;
    if (d->n_tok > INT32_MAX / int64_t(d->n_q_heads) || d->n_seq > (1 << 24) || d->window > INT32_MAX ||
        d->table_width > INT32_MAX)
        return ENGRAM_ERANGE;
    *ws_bytes = 0;
    if (d->n_tok == 0) return ENGRAM_OK;
    if (d->n_seq == 0) return ENGRAM_EINVAL;
    if (!d->cu_q && d->n_tok % d->n_seq != 0) return ENGRAM_EINVAL;
    if (!isfinite(d->scale)) return ENGRAM_EINVAL;
    if (!d->q || !d->out || !d->kv_len || !aligned(d->q, 16) || !aligned(d->out, 16) || !aligned(d->kv_len, 4) ||
        !aligned(d->cu_q, 4) || !aligned(d->lse, 4))
        return ENGRAM_EINVAL;
    if (d->table_width > 0 && (!d->block_table || !aligned(d->block_table, 4) || d->table_stride < d->table_width))
        return ENGRAM_EINVAL;
    if (d->table_stride < 0 || d->table_stride > (int64_t(1) << 40)) return ENGRAM_EINVAL;
    if (!good_strides(d->q_token_stride, d->q_head_stride) || !good_strides(d->out_token_stride, d->out_head_stride))
        return ENGRAM_EINVAL;

    a->q = static_cast<const uint8_t*>(d->q);
    a->out = static_cast<uint8_t*>(d->out);
    a->lse = d->lse;
    a->table = d->block_table;
    a->kv_len = d->kv_len;
    a->cu_q = d->cu_q;
    a->cache = view;
    a->part_o = nullptr;
    a->part_ml = nullptr;
    a->q_tok = d->q_token_stride;
    a->q_head = d->q_head_stride;
    a->out_tok = d->out_token_stride;
    a->out_head = d->out_head_stride;
    a->table_stride = d->table_stride;
    a->table_width = static_cast<uint32_t>(d->table_width);
    a->n_seq = static_cast<uint32_t>(d->n_seq);
    a->n_tok = static_cast<uint32_t>(d->n_tok);
    const bool alike = !d->cu_q || d->n_seq == 1;  // requests that the host knows the bound of: equal ones, or the only one
    a->uniform_q = alike ? static_cast<uint32_t>(d->n_tok / d->n_seq) : 0u;
    a->group = d->n_q_heads / view.n_kv_heads;
    a->window = static_cast<uint32_t>(d->window);
    a->scale_log2 = d->scale * 1.4426950408889634f;
    a->min_rows = 0;
    a->max_rows = UINT32_MAX;
    a->tiles_per = 0;
    a->split_tokens = 0;
    a->n_split = 1;
    a->n_work = 0;
    a->part_job = nullptr;
    const uint64_t heads = view.n_kv_heads, group = a->group;
    const uint64_t bound = alike ? a->uniform_q
                                 : (d->max_q_len ? std::min<uint64_t>(d->max_q_len, a->n_tok) : a->n_tok);
    const uint64_t most_rows = bound * group;
    const int64_t all_keys = std::min<int64_t>(d->table_width << view.page_shift, kMostKeys);
    out->many = *a;
    out->any_few = !alike || most_rows <= kFewRows;
    out->any_many = most_rows > kFewRows;
    out->few_o = out->few_ml = out->few_job = out->many_o = out->many_ml = 0;
    // a window bounds the keys of a tile: its own, those of its other tokens, and the step it begins in
    const auto keys_of = [&](uint64_t rows, int64_t step) {
        return d->window ? std::min<int64_t>(all_keys, d->window + int64_t((rows + group - 1) / group) + step) : all_keys;
    };
    if (out->any_few) {
        AttentionArgs& f = out->few;
        f.max_rows = static_cast<uint32_t>(std::min<uint64_t>(most_rows, kFewRows));
        const bool sets = f.max_rows > kRowsTile && of_pages(d->cache->type);
        f.of_tile = sets ? 2 * kRowsTile : kRowsTile;
        f.tiles_per = (f.max_rows + f.of_tile - 1) / f.of_tile;
        // without a bound the tiles as the lengths need them may be fewer
        if (!alike && uint64_t(f.n_tok) * group / f.of_tile + f.n_seq < uint64_t(f.tiles_per) * f.n_seq) f.tiles_per = 0;
        const uint64_t groups = (sets ? tile_count<2 * kRowsTile>(f) : tile_count<kRowsTile>(f)) * heads;
        if (groups > (uint64_t(1) << 23)) return ENGRAM_ERANGE;
        // Few keys: a workgroup takes a tile by itself, without the second launch that joins the parts (bf16, 8 KV heads,
        // head_dim 128: one request of 512 keys 8.2 us against 9.4 divided, of 1,024 12.5 against 9.5; where there are
        // tiles for every CU, 64 requests of 1,024 keys 40.8 against 43.5).  Else 512 workgroups share all keys: two on
        // each CU keep HBM as busy as three or four do (64 requests of up to 8,192 keys 216 us against 224 and 224), and
        // leave fewer parts to join.  Where a few tiles have all the keys, one on each CU leaves half of the parts (one
        // request of 131,072 keys 99 us against 104, of 32,768 27.6 against 31.3, head_dim 256 98.6 against 106; from 16
        // requests on two are better, 115 against 108).  A wave of e4m3 rows has half the bytes in flight, and two of its
        // workgroups are better throughout (52 us against 56), but for head_dim 256 (57 against 48).
        const int64_t keys = keys_of(f.max_rows, 32);
        const int64_t blocks = (keys + kRowsBlock - 1) / kRowsBlock;
        const bool whole = blocks * d->cache->head_dim <= 512 || (groups >= 512 && blocks <= 8) || groups * blocks >> 31;
        const bool two = groups > 64 || (!good_type(d->cache->type) && d->cache->head_dim < 256);
        // Pages of codes with one scale, head_dim 64: there are registers for three workgroups on a CU (64 requests of up to
        // 8,192 keys 77.7 us against 92.3; a third one does not help head_dim 128, 135 against 135, nor 256).
        const bool three = two && of_pages(d->cache->type) && d->cache->head_dim == 64;
        f.n_work = whole ? 0u : static_cast<uint32_t>(std::min<uint64_t>(groups * blocks, three ? 768 : two ? 512 : 256));
        if (f.n_work) {
            const size_t rows = size_t(f.n_work) * 2 * std::min(f.max_rows, f.of_tile);
            out->few_o = up256(rows * d->cache->head_dim * 4);
            out->few_ml = up256(rows * 8);
            out->few_job = up256(f.n_work * sizeof(int4));
        }
    }
    if (out->any_many) {
        AttentionArgs& m = out->many;
        m.min_rows = out->any_few ? kFewRows + 1 : 0;
        const uint32_t dim = d->cache->head_dim;
        const uint64_t all_rows = uint64_t(m.n_tok) * d->n_q_heads;
        const auto divide = [&](uint32_t of_tile) {
            m.of_tile = of_tile;
            if (alike) m.tiles_per = static_cast<uint32_t>((most_rows + of_tile - 1) / of_tile);
            const uint64_t groups = (of_tile == kFullTile ? tile_count<kFullTile>(m) : tile_count<kHalfTile>(m)) * heads;
            if (groups >> 23) return Split{0u, 0u, 0.0};  // 512 threads each, and a grid has less than 2^32
            // of the tiles that requests begin, half are expected to be there
            const double likely = double(groups) - (m.tiles_per ? 0.0 : 0.5 * double(m.n_seq * heads));
            return split_tiles(likely, alike || d->window, keys_of(of_tile, kTileAlign), all_rows, dim, of_tile);
        };
        // head_dim 128: full tiles share each key among more rows and take turns (2,048 tokens over 32,768 keys 1,060 us
        // against 1,190 in half tiles); half tiles leave fewer rows empty and CUs idle (8 requests of 17 tokens, 4 heads
        // to a key, over 8,192 keys 61 us against 79; 16 of up to 512 with a window of 1,024 126 against 147).
        Split s = divide(kHalfTile);
        if (dim == 128) {
            const Split full = divide(kFullTile);
            if (full.n && (!s.n || full.us <= s.us)) s = full;
            else s = divide(kHalfTile);
        }
        if (!s.n) return ENGRAM_ERANGE;
        m.split_tokens = s.tokens;
        m.n_split = s.n;
        if (s.n > 1) {
            out->many_o = up256(s.n * all_rows * dim * 4);
            out->many_ml = up256(s.n * all_rows * 8);
        }
    }
    *ws_bytes = out->few_o + out->few_ml + out->few_job + out->many_o + out->many_ml;
    return ENGRAM_OK;
}

}  // namespace

extern "C" {

int engram_qk_norm_rope(const engram_norm_rope_desc* d, void* stream) {
    if (!d) return ENGRAM_EINVAL;
    if (!good_type(d->type) || !good_dim(d->head_dim)) return ENGRAM_EUNSUPPORTED;
    if (d->n_tok < 0 || d->reserved0 != 0) return ENGRAM_EINVAL;
    if (d->n_tok > kMaxTokens || d->n_q_heads > 65535 || d->n_k_heads > 65535) return ENGRAM_ERANGE;
    int st = check_rotation(d->rotary_dim, d->head_dim, d->n_tok, d->positions, d->inv_freq, d->interleaved, d->eps);
    if (st != ENGRAM_OK) return st;
    NormRopeArgs a;
    const struct {
        const void *src, *dst, *weight;
        uint32_t heads;
        int64_t st, sh, dt, dh;
    } side[2] = {{d->q, d->q_out, d->q_weight, d->n_q_heads, d->q_token_stride, d->q_head_stride, d->q_out_token_stride,
                  d->q_out_head_stride},
                 {d->k, d->k_out, d->k_weight, d->n_k_heads, d->k_token_stride, d->k_head_stride, d->k_out_token_stride,
                  d->k_out_head_stride}};
    for (int i = 0; i < 2; ++i) {
        const auto& s = side[i];
        if (s.heads && d->n_tok) {
            if (!s.src || !s.dst || !aligned(s.src, 16) || !aligned(s.dst, 16) || !aligned(s.weight, 16))
                return ENGRAM_EINVAL;
            if (!good_strides(s.st, s.sh) || !good_strides(s.dt, s.dh)) return ENGRAM_EINVAL;
        }
        a.src[i] = static_cast<const uint8_t*>(s.src);
        a.dst[i] = static_cast<uint8_t*>(const_cast<void*>(s.dst));
        a.weight[i] = static_cast<const uint8_t*>(s.weight);
        a.heads[i] = s.heads;
        a.src_tok[i] = s.st;
        a.src_head[i] = s.sh;
        a.dst_tok[i] = s.dt;
        a.dst_head[i] = s.dh;
    }
    if (d->n_tok == 0 || d->n_q_heads + d->n_k_heads == 0) return ENGRAM_OK;
    a.positions = d->positions;
    a.inv_freq = d->inv_freq;
    a.n_tok = static_cast<uint32_t>(d->n_tok);
    a.rotary = d->rotary_dim;
    a.interleaved = d->interleaved;
    a.eps = d->eps;
    const hipError_t e = launch_norm_rope(a, d->head_dim, d->type, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ENGRAM_OK : ENGRAM_EHIP;
}

int engram_kv_append(const engram_append_desc* d, void* stream) {
    if (!d) return ENGRAM_EINVAL;
    AppendArgs a;
    int st = view_of(d->cache, &a.cache);
    if (st != ENGRAM_OK) return st;
    if (!good_type(d->type)) return ENGRAM_EUNSUPPORTED;
    if (d->cache->type != ENGRAM_E4M3 && d->cache->type != d->type) return ENGRAM_EUNSUPPORTED;
    if (d->n_tok < 0 || d->reserved0 != 0 || d->reserved1 != 0) return ENGRAM_EINVAL;
    if (d->n_tok > kMaxTokens) return ENGRAM_ERANGE;
    st = check_rotation(d->rotary_dim, d->cache->head_dim, d->n_tok, d->positions, d->inv_freq, d->interleaved, d->eps);
    if (st != ENGRAM_OK) return st;
    if (d->n_tok == 0) return ENGRAM_OK;
    if (!d->k || !d->v || !d->slots || !aligned(d->k, 16) || !aligned(d->v, 16) || !aligned(d->slots, 8) ||
        !aligned(d->k_weight, 16))
        return ENGRAM_EINVAL;
    if (!good_strides(d->k_token_stride, d->k_head_stride) || !good_strides(d->v_token_stride, d->v_head_stride))
        return ENGRAM_EINVAL;
    a.src[0] = static_cast<const uint8_t*>(d->k);
    a.src[1] = static_cast<const uint8_t*>(d->v);
    a.src_tok[0] = d->k_token_stride;
    a.src_head[0] = d->k_head_stride;
    a.src_tok[1] = d->v_token_stride;
    a.src_head[1] = d->v_head_stride;
    a.weight = static_cast<const uint8_t*>(d->k_weight);
    a.positions = d->positions;
    a.inv_freq = d->inv_freq;
    a.slots = d->slots;
    a.n_tok = static_cast<uint32_t>(d->n_tok);
    a.rotary = d->rotary_dim;
    a.interleaved = d->interleaved;
    a.eps = d->eps;
    const hipError_t e = launch_append(a, d->cache->head_dim, d->type, d->cache->type == ENGRAM_E4M3,
                                       static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ENGRAM_OK : ENGRAM_EHIP;
}

int engram_kv_append_pages(const engram_append_pages_desc* d, void* stream) {
    if (!d) return ENGRAM_EINVAL;
    AppendPagesArgs a;
    int st = view_of(d->cache, &a.cache);
    if (st != ENGRAM_OK) return st;
    if (!good_type(d->type) || !of_pages(d->cache->type)) return ENGRAM_EUNSUPPORTED;
    if (d->n_seq < 0 || d->n_tok < 0 || d->table_width < 0 || d->max_q_len < 0 || d->reserved0 != 0) return ENGRAM_EINVAL;
    if (d->n_tok > INT32_MAX || d->n_seq > (1 << 24) || d->table_width > INT32_MAX) return ENGRAM_ERANGE;
    st = check_rotation(d->rotary_dim, d->cache->head_dim, d->n_tok, d->positions, d->inv_freq, d->interleaved, d->eps);
    if (st != ENGRAM_OK) return st;
    if (d->n_tok == 0) return ENGRAM_OK;
    if (d->n_seq == 0) return ENGRAM_EINVAL;
    if (!d->cu_q && d->n_tok % d->n_seq != 0) return ENGRAM_EINVAL;
    if (!d->k || !d->v || !d->kv_len || !aligned(d->k, 16) || !aligned(d->v, 16) || !aligned(d->kv_len, 4) ||
        !aligned(d->cu_q, 4) || !aligned(d->k_weight, 16))
        return ENGRAM_EINVAL;
    if (!good_strides(d->k_token_stride, d->k_head_stride) || !good_strides(d->v_token_stride, d->v_head_stride))
        return ENGRAM_EINVAL;
    if (d->table_stride < 0 || d->table_stride > (int64_t(1) << 40)) return ENGRAM_EINVAL;
    if (d->table_width == 0) return ENGRAM_OK;  // no request has a page
    if (!d->block_table || !aligned(d->block_table, 4) || d->table_stride < d->table_width) return ENGRAM_EINVAL;
    a.src[0] = static_cast<const uint8_t*>(d->k);
    a.src[1] = static_cast<const uint8_t*>(d->v);
    a.src_tok[0] = d->k_token_stride;
    a.src_head[0] = d->k_head_stride;
    a.src_tok[1] = d->v_token_stride;
    a.src_head[1] = d->v_head_stride;
    a.weight = static_cast<const uint8_t*>(d->k_weight);
    a.positions = d->positions;
    a.inv_freq = d->inv_freq;
    a.table = d->block_table;
    a.kv_len = d->kv_len;
    a.cu_q = d->cu_q;
    a.table_stride = d->table_stride;
    a.table_width = static_cast<uint32_t>(d->table_width);
    a.n_seq = static_cast<uint32_t>(d->n_seq);
    a.n_tok = static_cast<uint32_t>(d->n_tok);
    a.uniform_q = d->cu_q ? 0u : static_cast<uint32_t>(d->n_tok / d->n_seq);
    const uint64_t bound = d->cu_q ? (d->max_q_len ? std::min<uint64_t>(d->max_q_len, a.n_tok) : d->n_seq == 1 ? a.n_tok : 0)
                                   : a.uniform_q;
    a.most_q = static_cast<uint32_t>(bound);
    // A run of n tokens touches at most (n + page - 2) / page + 1 pages; set aside for each request where that is fewer than
    // room for any lengths.
    const uint64_t page = uint64_t(1) << a.cache.page_shift, any = (a.n_tok >> a.cache.page_shift) + 2 * uint64_t(a.n_seq);
    const uint64_t per = bound ? (bound + page - 2) / page + 1 : 0;
    const bool each = per && (per * a.n_seq <= any || !d->cu_q);
    a.pages_per = each ? static_cast<uint32_t>(per) : 0u;
    // workgroups of 256 threads, and a grid has less than 2^32
    const uint64_t pages = each ? per * a.n_seq : any;
    const uint32_t heads = append_heads(pages, a.cache.n_kv_heads, d->rotary_dim > 0);
    if (pages * (2 * ((uint64_t(a.cache.n_kv_heads) + heads - 1) / heads)) >> 23) return ENGRAM_ERANGE;
    if (bound == 1 && uint64_t(a.n_seq) * 2 * a.cache.n_kv_heads >> 24) return ENGRAM_ERANGE;
    a.rotary = d->rotary_dim;
    a.interleaved = d->interleaved;
    a.eps = d->eps;
    const hipError_t e = launch_append_pages(a, d->cache->head_dim, d->type, d->cache->type == ENGRAM_I8_PAGE,
                                             static_cast<hipStream_t>(stream));
    return e == hipSuccess ? ENGRAM_OK : ENGRAM_EHIP;
}

int engram_paged_attention_workspace(const engram_attention_desc* d, size_t* bytes) {
    if (!bytes) return ENGRAM_EINVAL;
    Launches l;
    size_t need = 0;
    const int st = attention_args(d, &l, &need);
    if (st == ENGRAM_OK) *bytes = need;
    return st;
}

int engram_paged_attention(const engram_attention_desc* d, void* ws, size_t ws_bytes, void* stream) {
    Launches l;
    size_t need = 0;
    const int st = attention_args(d, &l, &need);
    if (st != ENGRAM_OK) return st;
    if (d->n_tok == 0) return ENGRAM_OK;
    if (need) {
        if (!ws || ws_bytes < need || !aligned(ws, 256)) return ENGRAM_EWORKSPACE;
        uint8_t* at = static_cast<uint8_t*>(ws);
        l.few.part_o = reinterpret_cast<float*>(at);
        l.few.part_ml = reinterpret_cast<float*>(at + l.few_o);
        l.few.part_job = reinterpret_cast<int4*>(at + l.few_o + l.few_ml);
        at += l.few_o + l.few_ml + l.few_job;
        l.many.part_o = reinterpret_cast<float*>(at);
        l.many.part_ml = reinterpret_cast<float*>(at + l.many_o);
    }
    const hipStream_t to = static_cast<hipStream_t>(stream);
    const uint32_t dim = d->cache->head_dim;
    const Held held = d->cache->type == ENGRAM_E4M3        ? kE4m3Rows
                      : d->cache->type == ENGRAM_E4M3_PAGE ? kE4m3Pages
                      : d->cache->type == ENGRAM_I8_PAGE   ? kI8Pages
                                                           : kHalves;
    hipError_t e = hipSuccess;
    if (l.any_many) {
        e = launch_paged_tile(l.many, dim, d->type, held, to);
        if (e == hipSuccess && l.many.n_split > 1) e = launch_paged_join(l.many, dim, d->type, to);
    }
    if (e == hipSuccess && l.any_few) e = launch_paged_rows(l.few, dim, d->type, held, to);
    return e == hipSuccess ? ENGRAM_OK : ENGRAM_EHIP;
}

}  // extern "C"
