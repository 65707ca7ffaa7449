// Shared by the calls between two steps of a decoding batch (page tables and
// slots, verification of drafts): arguments and launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "engram.h"

namespace engram {

struct TablesArgs {
    const int32_t* lengths;   // [n_seq]
    const int32_t* fresh;     // [n_seq], or nullptr: uniform_new each
    int32_t* table;           // [n_seq][width], row stride table_stride
    int32_t* held;            // [n_seq]
    int32_t* stack;           // [n_stack]
    int32_t* n_free;          // [1]
    int64_t* slots;           // [n_tok]
    int32_t* positions;       // [n_tok]
    int32_t* cu_q;            // [n_seq + 1]
    int32_t* kv_len;          // [n_seq]
    int32_t* n_short;         // [1]
    uint32_t* ws;             // nullptr: one workgroup does it all
    int64_t table_stride;
    uint32_t n_seq, n_tok, width, n_stack;
    uint32_t uniform_new;
    uint32_t page_shift;
};

// Whether one workgroup does it all, without a workspace: a request to a thread, and up to eight tokens.  (64 requests of 6
// tokens take 5.9 us so and 9.0 in two launches, 1,024 of 8 tokens 11.9 and 11.3, 512 of 16 10.0 and 9.7.)
constexpr uint32_t kOneRequests = 1024, kOneTokens = 8192;
inline bool tables_in_one(uint64_t n_seq, uint64_t n_tok) { return n_seq <= kOneRequests && n_tok <= kOneTokens; }
inline size_t tables_workspace(uint64_t n_seq, uint64_t n_tok) {
    return tables_in_one(n_seq, n_tok) ? 0 : ((3 * n_seq + 2 + 4) * 4 + 255) & ~size_t(255);
}
hipError_t launch_page_tables(const TablesArgs& a, hipStream_t stream);

struct VerifyArgs {
    const uint8_t* target;    // [n_draft + n_seq][vocab], rows target_stride elements apart
    const uint8_t* drafter;   // [n_draft][vocab], or nullptr: each draft was certain
    const int32_t* draft;     // [n_draft]
    const float* uniform;     // [n_draft]
    const float* last;        // [n_seq]
    const int32_t* cu_draft;  // [n_seq + 1], or nullptr: uniform_drafts each
    int32_t* tokens;          // [n_draft + n_seq]
    int32_t* accepted;        // [n_seq]
    double* ws;               // sums of blocks, nullptr: a workgroup reads a request's row by itself
    int64_t target_stride, drafter_stride;
    uint32_t n_seq, n_draft, vocab;
    uint32_t uniform_drafts;
    uint32_t blocks;          // of a row
};

size_t verify_workspace(uint64_t n_seq, uint64_t vocab);
// Blocks of a row that the workspace has sums of; 0: none, a workgroup reads a request's row by itself.
uint32_t verify_blocks(uint64_t n_seq, uint64_t vocab);
hipError_t launch_verify_draft(const VerifyArgs& a, uint32_t type, hipStream_t stream);

}  // namespace engram
