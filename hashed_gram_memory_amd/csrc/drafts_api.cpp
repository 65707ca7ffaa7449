// Host side of the calls between two steps of a decoding batch (page tables
// and slots, verification of drafts): validation and launches, as in
// engram_api.cpp.
#include <algorithm>

#include "drafts.h"
#include "engram_internal.h"

using namespace engram;

namespace {

constexpr int64_t kMostRequests = int64_t(1) << 20;
constexpr int64_t kMost = int64_t(1) << 30;  // tokens, pages

int tables_args(const engram_page_tables_desc* d, TablesArgs* a, size_t* bytes) {
    if (!d) return ENGRAM_EINVAL;
    if (d->n_seq < 0 || d->n_tok < 0 || d->table_width < 0 || d->n_pages < 0 || d->reserved0 != 0) return ENGRAM_EINVAL;
    const uint32_t p = d->page_size;
    if (p < 8 || p > 1024 || (p & (p - 1)) != 0) return ENGRAM_EUNSUPPORTED;
    if (d->n_seq > kMostRequests || d->n_tok >= kMost || d->table_width > INT32_MAX || d->n_pages > kMost) return ENGRAM_ERANGE;
    if (!d->new_tokens && d->n_seq && d->n_tok % d->n_seq != 0) return ENGRAM_EINVAL;
    if (d->n_seq && (!d->lengths || !d->held || !d->kv_len || !aligned(d->lengths, 4) || !aligned(d->new_tokens, 4) ||
                     !aligned(d->held, 4) || !aligned(d->kv_len, 4)))
        return ENGRAM_EINVAL;
    if (d->n_tok && (!d->slots || !d->positions || !aligned(d->slots, 8) || !aligned(d->positions, 4))) return ENGRAM_EINVAL;
    if (!d->cu_q || !d->n_short || !d->n_free || !aligned(d->cu_q, 4) || !aligned(d->n_short, 4) || !aligned(d->n_free, 4))
        return ENGRAM_EINVAL;
    if (d->n_pages && (!d->free_pages || !aligned(d->free_pages, 4))) return ENGRAM_EINVAL;
    if (d->table_width && d->n_seq && (!d->block_table || !aligned(d->block_table, 4) || d->table_stride < d->table_width))
        return ENGRAM_EINVAL;
    if (d->table_stride < 0 || d->table_stride > (int64_t(1) << 40)) return ENGRAM_EINVAL;
    a->lengths = d->lengths;
    a->fresh = d->new_tokens;
    a->table = d->block_table;
    a->held = d->held;
    a->stack = d->free_pages;
    a->n_free = d->n_free;
    a->slots = d->slots;
    a->positions = d->positions;
    a->cu_q = d->cu_q;
    a->kv_len = d->kv_len;
    a->n_short = d->n_short;
    a->ws = nullptr;
    a->table_stride = d->table_stride;
    a->n_seq = static_cast<uint32_t>(d->n_seq);
    a->n_tok = static_cast<uint32_t>(d->n_tok);
    a->width = static_cast<uint32_t>(d->table_width);
    a->n_stack = static_cast<uint32_t>(d->n_pages);
    a->uniform_new = d->n_seq ? static_cast<uint32_t>(d->n_tok / d->n_seq) : 0u;
    a->page_shift = static_cast<uint32_t>(__builtin_ctz(p));
    *bytes = tables_workspace(a->n_seq, a->n_tok);
    return ENGRAM_OK;
}

int verify_args(const engram_verify_draft_desc* d, VerifyArgs* a, size_t* bytes) {
    if (!d) return ENGRAM_EINVAL;
    if (d->type != ENGRAM_F32 && d->type != ENGRAM_BF16 && d->type != ENGRAM_F16) return ENGRAM_EUNSUPPORTED;
    if (d->n_seq < 0 || d->n_draft < 0 || d->vocab < 0 || d->reserved0 != 0) return ENGRAM_EINVAL;
    if (d->n_seq > kMostRequests || d->n_draft > kMost || d->vocab > kMost) return ENGRAM_ERANGE;
    *bytes = 0;
    if (d->n_seq == 0) return d->n_draft ? ENGRAM_EINVAL : ENGRAM_OK;
    if (d->vocab == 0) return ENGRAM_EINVAL;
    if (!d->cu_draft && d->n_draft % d->n_seq != 0) return ENGRAM_EINVAL;
    const uintptr_t size = d->type == ENGRAM_F32 ? 4 : 2;
    if (!d->target || !d->last_uniform || !d->tokens || !d->n_accepted || !aligned(d->target, size) ||
        !aligned(d->draft_probs, size) || !aligned(d->last_uniform, 4) || !aligned(d->tokens, 4) || !aligned(d->n_accepted, 4) ||
        !aligned(d->cu_draft, 4))
        return ENGRAM_EINVAL;
    if (d->n_draft && (!d->draft || !d->uniform || !aligned(d->draft, 4) || !aligned(d->uniform, 4))) return ENGRAM_EINVAL;
    const int64_t most = int64_t(1) << 40;
    if (d->target_stride < 0 || d->target_stride > most || d->draft_stride < 0 || d->draft_stride > most) return ENGRAM_EINVAL;
    a->target = static_cast<const uint8_t*>(d->target);
    a->drafter = static_cast<const uint8_t*>(d->draft_probs);
    a->draft = d->draft;
    a->uniform = d->uniform;
    a->last = d->last_uniform;
    a->cu_draft = d->cu_draft;
    a->tokens = d->tokens;
    a->accepted = d->n_accepted;
    a->ws = nullptr;
    a->target_stride = d->target_stride;
    a->drafter_stride = d->draft_stride;
    a->n_seq = static_cast<uint32_t>(d->n_seq);
    a->n_draft = static_cast<uint32_t>(d->n_draft);
    a->vocab = static_cast<uint32_t>(d->vocab);
    a->uniform_drafts = static_cast<uint32_t>(d->n_draft / d->n_seq);
    a->blocks = verify_blocks(a->n_seq, a->vocab);
    if (uint64_t(a->n_seq) * std::max(a->blocks, 1u) > (uint64_t(1) << 23)) return ENGRAM_ERANGE;  // a grid has less than 2^32 threads
    *bytes = verify_workspace(a->n_seq, a->vocab);
    return ENGRAM_OK;
}

int as_status(hipError_t e) { return e == hipSuccess ? ENGRAM_OK : ENGRAM_EHIP; }

}  // namespace

extern "C" {

int engram_page_tables_workspace(const engram_page_tables_desc* d, size_t* bytes) {
    if (!bytes) return ENGRAM_EINVAL;
    TablesArgs a;
    size_t need = 0;
    const int st = tables_args(d, &a, &need);
    if (st == ENGRAM_OK) *bytes = need;
    return st;
}

int engram_page_tables(const engram_page_tables_desc* d, void* ws, size_t ws_bytes, void* stream) {
    TablesArgs a;
    size_t need = 0;
    const int st = tables_args(d, &a, &need);
    if (st != ENGRAM_OK) return st;
    if (need) {
        if (!ws || ws_bytes < need || !aligned(ws, 256)) return ENGRAM_EWORKSPACE;
        a.ws = static_cast<uint32_t*>(ws);
    }
    return as_status(launch_page_tables(a, static_cast<hipStream_t>(stream)));
}

int engram_verify_draft_workspace(const engram_verify_draft_desc* d, size_t* bytes) {
    if (!bytes) return ENGRAM_EINVAL;
    VerifyArgs a;
    size_t need = 0;
    const int st = verify_args(d, &a, &need);
    if (st == ENGRAM_OK) *bytes = need;
    return st;
}

int engram_verify_draft(const engram_verify_draft_desc* d, void* ws, size_t ws_bytes, void* stream) {
    VerifyArgs a;
    size_t need = 0;
    const int st = verify_args(d, &a, &need);
    if (st != ENGRAM_OK) return st;
    if (d->n_seq == 0) return ENGRAM_OK;
    if (need) {
        if (!ws || ws_bytes < need || !aligned(ws, 256)) return ENGRAM_EWORKSPACE;
        a.ws = static_cast<double*>(ws);
    }
    return as_status(launch_verify_draft(a, d->type, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
