/*
 * engram.h -- C ABI of the Engram n-gram memory lookup for AMD Instinct
 * MI355X (gfx950).
 *
 * Sources, cited by page title and section:
 *   [VRAM]  "DeepSeek V4.1 Flash: The VRAM Killer. Can You Run It Locally?",
 *           section "What makes up the 511 GB of weights?"
 *   [GUIDE] "How to Run DeepSeek-V4.1-Flash: 510 GB, and 203 GB of It Is a
 *           Lookup Table", sections "The architecture", "Where the 510 GB
 *           goes" and "Engram: the table that is never multiplied"
 *   [REQ]   "Running DeepSeek V4.1 Flash locally: the numbers beyond 552B",
 *           section "Backbone, Engram, and active parameters describe
 *           different scales"
 *   [X]     "How DeepSeek V4.1 Flash's 763B weights run on consumer GPUs"
 *   [BLOG]  stondo.github.io, "deepseek-v41-flash-552b-exl3-two-rtx-pro-6000",
 *           section "What eager-plus-NVMe actually delivers"
 *
 * The operation.  Two Engram modules each hash the suffix n-grams of order
 * 2, 3 and 4 of the token-id stream with 8 independent heads and read one
 * row per (order, head): 24 rows per module, 48 per token [GUIDE "Engram";
 * VRAM].  Rows are 256 bytes of FP8 [GUIDE "Engram"; REQ]; each carries one
 * fp32 scale, or 8 E8M0 exponents (one per 32 elements), as the plan says.
 * The row addresses depend on the token ids alone, so the
 * whole prompt is hashed before any row is read [VRAM; GUIDE "Engram"]: the
 * library exposes the hash and the gather as separate calls.  The 24
 * dequantised rows of a module are summed into one fp32 vector of 256
 * elements; the pages' learned gate that follows (row vs. hidden state,
 * [GUIDE "The architecture"]) is not part of this library.
 *
 * Conventions for every call:
 *   - Return value: ENGRAM_OK (0) or a negative engram_status.  No call
 *     throws, aborts or prints.
 *   - All arguments are validated on the host before anything is launched;
 *     on an error return nothing has been launched and no output was
 *     written.
 *   - Calls that take a stream are asynchronous on that stream (a
 *     hipStream_t passed as void*; NULL is the null stream).  They never
 *     synchronise and never allocate device memory.
 *   - Device pointers are owned by the caller and must stay valid until the
 *     work queued on the stream has finished.
 *   - Device-side faults (e.g. a table pointer that is not device memory)
 *     surface at the caller's next synchronisation, as usual in HIP.
 */
#ifndef ENGRAM_H
#define ENGRAM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Geometry of the lookup [GUIDE "Engram"; VRAM]. */
#define ENGRAM_N_MODULES 2        /* Engram modules (layers) per token           */
#define ENGRAM_MIN_ORDER 2        /* shortest suffix n-gram                      */
#define ENGRAM_MAX_ORDER 4        /* longest suffix n-gram, = id window length    */
#define ENGRAM_N_HEADS 8          /* hash heads per (module, order)              */
#define ENGRAM_ROWS_PER_MODULE 24 /* 3 orders x 8 heads                          */
#define ENGRAM_N_SUB 48           /* sub-tables = rows read per token            */
#define ENGRAM_ROW_BYTES 256      /* FP8 E4M3 codes per row = output width       */
#define ENGRAM_N_MULT 192         /* hash multipliers: 2 x 3 x 8 x 4             */

/* Row scale formats (engram_plan_desc.scale_format). */
#define ENGRAM_SCALE_F32_ROW 0       /* one fp32 scale per row                          */
#define ENGRAM_SCALE_E8M0_BLOCK32 1  /* 8 E8M0 bytes per row, one per 32 elements      */

/* Seed of the default hash multipliers: the bytes "ENGRAM" followed by 0x0001. */
#define ENGRAM_DEFAULT_HASH_SEED 0x454E4752414D0001ULL

typedef enum engram_status {
    ENGRAM_OK = 0,
    ENGRAM_EINVAL = -1,      /* NULL or misaligned pointer, bad shape or flag       */
    ENGRAM_ERANGE = -2,      /* row count 0 or > 2^32, token count out of range     */
    ENGRAM_EWORKSPACE = -3,  /* workspace NULL or smaller than required             */
    ENGRAM_EHIP = -4,        /* the HIP runtime refused a launch                    */
    ENGRAM_EUNSUPPORTED = -5 /* a geometry other than the one above                 */
} engram_status;

/*
 * Plan description.  Sub-table s = 24*m + 8*(n-2) + h holds module m, order
 * n, head h (module-major, then order, then head).
 *
 *   n_modules, min_order, max_order, n_heads, row_bytes
 *       Must equal 2, 2, 4, 8, 256 (else ENGRAM_EUNSUPPORTED).
 *   vocab_size
 *       Exclusive upper bound of the token ids (the vocabulary the ids are
 *       drawn from), or 0 when ids may take any value in [0, 2^31).  It is
 *       the length of vocab_map when there is one.  engram_dedup uses it to
 *       size its sort keys: 4*ceil(log2(vocab_size)) bits per window, or, for
 *       2^16 < vocab_size <= 2^18, 4*ceil(log2(D+1)) bits where D is the
 *       number of distinct ids the call uses.  Ids at or above vocab_size
 *       break the dedup grouping and, with a vocab_map, the hash (see
 *       engram_hash); engram_check_inputs counts them.
 *   hash_seed
 *       Seeds the 192 hash multipliers: M[i] is output i+1 of splitmix64
 *       (Steele, Lea and Flood 2014) seeded with hash_seed, with bit 0 set;
 *       i runs over (module, order, head, k) in that nesting, k = 0..3.
 *   rows[48]   (host array, copied)
 *       Rows R_s of sub-table s, 1 <= R_s <= 2^32.
 *   tables[48] (host array of device pointers, copied)
 *       Sub-table s as row-major uint8 [R_s][256] of FP8 E4M3 codes (OCP
 *       encoding: bias 7, no infinities, 0x7F/0xFF are NaN).  16-byte aligned.
 *   scales[48] (host array of device pointers, copied)
 *       ENGRAM_SCALE_F32_ROW: fp32 [R_s], the scale of each row; 4-byte
 *       aligned.
 *       ENGRAM_SCALE_E8M0_BLOCK32: uint8 [R_s][8], the 8 bytes of scales a
 *       row carries [GUIDE "Engram"], read as one E8M0 exponent per block of
 *       32 elements (element j uses byte j/32; e stands for 2^(e-127), 255
 *       is NaN), the microscaling form of FP8 named for these tables [X];
 *       8-byte aligned.
 *   scale_format
 *       ENGRAM_SCALE_F32_ROW (0, the default) or ENGRAM_SCALE_E8M0_BLOCK32
 *       (else ENGRAM_EUNSUPPORTED).
 *   reserved1
 *       Must be 0.
 *   vocab_map  (device pointer, not copied; NULL = none)
 *       uint32 [vocab_size]: the id normalisation applied before hashing.
 *       The pages' engines fold ids that differ only in case, accents or
 *       spacing into one id of a smaller vocabulary before hashing [GUIDE
 *       "Engram"]; the map is that table.  Every id of a window (history and
 *       the pad id 0 included) is replaced by vocab_map[id] before the
 *       multiply-xor.  Needs vocab_size > 0 (the map's length) and 4-byte
 *       alignment.  engram_dedup still groups raw windows: equal raw windows
 *       have equal mapped windows, so its groups stay valid.
 *
 * The plan copies the description; the tables themselves are not copied and
 * must outlive every call that uses the plan.
 */
typedef struct engram_plan_desc {
    uint32_t n_modules;
    uint32_t min_order;
    uint32_t max_order;
    uint32_t n_heads;
    uint32_t row_bytes;
    uint32_t vocab_size;           /* exclusive bound of token ids; 0 = any id in [0, 2^31) */
    uint64_t hash_seed;
    const uint64_t* rows;
    const uint8_t* const* tables;
    const void* const* scales;
    uint32_t scale_format;
    uint32_t reserved1;            /* must be 0 */
    const uint32_t* vocab_map;     /* device uint32 [vocab_size] or NULL */
} engram_plan_desc;

typedef struct engram_plan_s* engram_plan_t;

/* Fill a description with the default geometry and hash seed; the caller
 * still sets rows, tables and scales.  Returns ENGRAM_EINVAL on NULL. */
int engram_plan_desc_init(engram_plan_desc* desc);

/*
 * Validate a description and build an immutable plan: copies the row counts
 * and pointers, derives the multipliers and the exact division constants of
 * each R_s.  The geometry it accepts is the pages' one: two modules, orders
 * 2 to 4, 8 heads per order, 256-byte FP8 rows, 48 sub-tables [GUIDE
 * "Engram"; VRAM].  The pages print no hash constants; the multipliers are
 * this library's own (see hash_seed).  Host-only: touches no device and may
 * run before any device exists.  *out is set only on ENGRAM_OK.  A plan may
 * be used from several host threads and streams at once.  Errors: EINVAL
 * (NULL argument, pointer, misaligned pointer, reserved1 != 0, a vocab_map
 * without vocab_size), ERANGE (a row count of 0 or above 2^32),
 * EUNSUPPORTED (another geometry or scale format).
 */
int engram_plan(const engram_plan_desc* desc, engram_plan_t* out);

/* Release a plan (NULL is accepted).  No work using it may be in flight. */
int engram_plan_destroy(engram_plan_t plan);

/* Copy the 192 hash multipliers of a plan into host memory out[192], in
 * (module, order, head, k) order. */
int engram_plan_multipliers(engram_plan_t plan, uint64_t* out);

/*
 * Hash: 48 row addresses per token [GUIDE "Engram"; VRAM].
 *
 * Token tok = s*seq_len + t has the id window w_k = id at position t-k,
 * k = 0..3; positions before 0 read history[s][3 + (t-k)] (history[s][2] is
 * the id just before position 0) or, with history == NULL, id 0.  With a
 * vocab_map in the plan each w_k is then replaced by vocab_map[w_k].  For
 * module m, order n, head h, with u64 the zero-extension of the 32-bit id:
 *     x = XOR_{k<n} ( u64(w_k) * M[m][n][h][k] )   (mod 2^64)
 *     addr[tok][24*m + 8*(n-2) + h] = x mod R_s
 *
 *   ids      device int32 [n_seq][seq_len], ids in [0, 2^31), and below the
 *            plan's vocab_size when it has a vocab_map (the map is read at
 *            every window id, history and pad included, without a bounds
 *            check: a larger or negative id reads outside the map).  Not
 *            checked on the device; engram_check_inputs counts violations.
 *   history  device int32 [n_seq][3] or NULL; the same bounds as ids.
 *   addr     device uint32 [n_seq*seq_len][48], 16-byte aligned (output).
 *
 * n_seq*seq_len == 0 is a no-op.  Errors: EINVAL (NULL/misaligned pointer,
 * negative sizes), ERANGE (n_seq*seq_len >= 2^31).
 */
int engram_hash(engram_plan_t plan, const int32_t* ids, const int32_t* history,
                int64_t n_seq, int64_t seq_len, uint32_t* addr, void* stream);

/*
 * Gather, dequantise and sum [GUIDE "Engram"; REQ].
 *
 * For token tok, module m and element j:
 *     out[tok][m][j] = sum_{q=0..23} fp8(T_{24m+q}[a][j]) * scale_{24m+q}(a, j),
 *     a = addr[tok][24m+q],
 * scale(a, j) = scales[a] (fp32 per row) or 2^(scales[a][j/32] - 127) (E8M0
 * per 32-element block),
 * accumulated in fp32 in ascending q (fused multiply-add), starting at +0.
 *
 *   addr    device uint32 [n_tok][48] (as written by engram_hash); every
 *           address must be < R_s (not checked on the device).
 *   out     device fp32 [n_tok][2][256], 16-byte aligned (output).
 *
 * Direct mode: perm, offsets and n_unique all NULL.
 * Dedup mode: perm, offsets, n_unique as written by engram_dedup for the
 * same tokens; each group of tokens with equal windows is looked up once
 * and its vector stored to every member.  The result is bitwise identical
 * to direct mode.  In dedup mode the grid covers n_tok groups and exits
 * early past *n_unique, which stays on the device.
 *
 * n_tok == 0 is a no-op.  Errors: EINVAL (NULL/misaligned pointer, a partial
 * set of dedup pointers), ERANGE (n_tok < 0 or >= 2^31).
 */
int engram_gather_reduce(engram_plan_t plan, const uint32_t* addr, int64_t n_tok,
                         const int32_t* perm, const int32_t* offsets,
                         const int32_t* n_unique, float* out, void* stream);

/*
 * engram_gather_reduce in direct mode for a batch of n_seq sequences of
 * seq_len tokens whose addresses engram_hash wrote (addr[n_seq*seq_len][48],
 * token-major).  Same results, bitwise; the tokens are visited in tiles of 64
 * positions, up to 8 sequences at the same position per workgroup, so that
 * sequences sharing a prefix gather each prefix window once per workgroup
 * (in a batch of 8,192 tokens or more, tokens with equal addresses share one
 * gather) and read its rows from L2 after their first fetch (the pages hash
 * every address before the lookup [VRAM; GUIDE "Engram"], and batched prompts
 * often share a system prefix).
 *
 *   addr     device uint32 [n_seq*seq_len][48], 16-byte aligned.
 *   out      device fp32 [n_seq*seq_len][2][256], 16-byte aligned (output).
 *
 * n_seq*seq_len == 0 is a no-op.  Errors: EINVAL (NULL/misaligned pointer,
 * negative count), ERANGE (n_seq*seq_len above 2^31 - 1).
 */
int engram_gather_reduce_batched(engram_plan_t plan, const uint32_t* addr, int64_t n_seq, int64_t seq_len,
                                 float* out, void* stream);

/*
 * Inputs for the learned gate that follows the lookup: each retrieved row is
 * weighed against the hidden state before the module's rows are combined
 * [GUIDE "The architecture", "Engram"].  The gate itself (trained weights,
 * hidden states) is outside this library.
 *
 * engram_gather_weighted: as engram_gather_reduce (direct mode) with one
 * caller weight per row:
 *     out[tok][m][j] = sum_q fp8(T_{24m+q}[a][j]) * fp32(scale_{24m+q}(a, j) * w[tok][24m+q])
 * accumulated in fp32 in ascending q; with every weight 1 the result is
 * bitwise that of engram_gather_reduce.
 *   weights  device fp32 [n_tok][48] (same order as addr), 16-byte aligned.
 *   out      device fp32 [n_tok][2][256], 16-byte aligned (output).
 *
 * engram_gather_rows: the 48 dequantised rows of every token, un-reduced:
 *     rows[tok][s][j] = fp32(fp8(T_s[a][j]) * scale_s(a, j)),  a = addr[tok][s]
 *   rows     device fp32 [n_tok][48][256] (48 KiB per token), 16-byte aligned.
 *
 * n_tok == 0 is a no-op.  Errors: EINVAL (NULL/misaligned pointer), ERANGE.
 */
int engram_gather_weighted(engram_plan_t plan, const uint32_t* addr, int64_t n_tok,
                           const float* weights, float* out, void* stream);
int engram_gather_rows(engram_plan_t plan, const uint32_t* addr, int64_t n_tok, float* rows,
                       void* stream);

/*
 * Fused lookup: engram_hash followed by engram_gather_reduce (direct mode)
 * in one launch, without the address buffer.  The addresses depend on the
 * ids alone [VRAM; GUIDE "Engram"], so each (token, module) computes its own
 * 24 rows and gathers them.  Bitwise identical to the two calls.  A batch
 * of sequences is visited in the order of engram_gather_reduce_batched, so
 * sequences that share a prefix gather each prefix window once per workgroup
 * and read its rows from L2 after their first fetch: passing such sequences
 * in one call is cheaper than one call each.
 *
 *   ids, history, n_seq, seq_len   as for engram_hash.
 *   out       device fp32 [n_seq*seq_len][2][256], 16-byte aligned (output).
 *
 * n_seq*seq_len == 0 is a no-op.  Errors: EINVAL, ERANGE as engram_hash.
 */
int engram_lookup(engram_plan_t plan, const int32_t* ids, const int32_t* history,
                  int64_t n_seq, int64_t seq_len, float* out, void* stream);

/*
 * engram_lookup in dedup mode: one hash and one gather per group of tokens
 * with equal windows, the vector stored to every member of the group.  Equal
 * windows hash to equal rows [VRAM; GUIDE "Engram"], so the result is bitwise
 * that of engram_lookup (and of engram_hash + engram_gather_reduce in either
 * mode); the address buffer and the separate hash launch are gone, and a
 * window repeated across a batch (a shared prefix [BLOG]) is hashed once.
 *
 *   ids, history, n_seq, seq_len   as for engram_lookup, and the same tokens
 *             that engram_dedup grouped.
 *   perm, offsets, n_unique        as written by engram_dedup for those
 *             tokens (device int32, 4-byte aligned); *n_unique stays on the
 *             device.  *n_unique < 0 (a failed dedup call) writes nothing.
 *   out       device fp32 [n_seq*seq_len][2][256], 16-byte aligned (output).
 *
 * The grid covers n_seq*seq_len groups and exits early past *n_unique.  A
 * perm or offsets entry out of [0, n_tok) is skipped, never dereferenced.
 * n_seq*seq_len == 0 is a no-op.  Errors: EINVAL (NULL/misaligned pointer),
 * ERANGE as engram_hash.
 */
int engram_lookup_dedup(engram_plan_t plan, const int32_t* ids, const int32_t* history,
                        int64_t n_seq, int64_t seq_len, const int32_t* perm, const int32_t* offsets,
                        const int32_t* n_unique, float* out, void* stream);

/*
 * Workspace bytes engram_dedup needs for n_tok tokens under this plan
 * (host-only).  The size depends on the plan's vocab_size, which bounds the
 * width of the sort keys.  Errors: EINVAL (NULL plan or bytes), ERANGE
 * (n_tok < 0 or > 2^22).
 */
int engram_dedup_workspace(engram_plan_t plan, int64_t n_tok, size_t* bytes);

/*
 * Group the tokens whose id windows (w_0, w_1, w_2, w_3) are equal.
 *
 * The pages hash every row address from the token ids alone, before the
 * forward pass, so a whole batch's addresses are known up front and can be
 * fetched together [VRAM]; and in the serving setups they describe, most of
 * a prompt is a prefix other requests already sent [BLOG "What eager-plus-
 * NVMe actually delivers"].  Tokens with equal windows hash to the same 48
 * rows, so one lookup serves a whole group (engram_gather_reduce in dedup
 * mode).  Groups are ordered by ascending window (w_0 most significant, ids
 * compared as unsigned), tokens within a group by ascending index: the
 * result is unique.
 *
 *   ids, history, n_seq, seq_len   as for engram_hash.  Every id should be
 *             < the plan's vocab_size (when it is not 0); a larger or negative
 *             id is a contract violation: its grouping is then unspecified,
 *             but the call reads and writes nothing out of bounds.
 *   perm      device int32 [n_tok]: the tokens, group by group (output).
 *   offsets   device int32 [n_tok + 1]: offsets[u] is where group u starts
 *             in perm; offsets[n_unique] = n_tok; entries past n_unique are
 *             left unspecified (output).
 *   n_unique  device int32 [1]: the number of groups (output).  -1 reports
 *             that a bounded device-side wait of the sort gave up (the sort's
 *             tiles wait for the ones started before them; this does not
 *             happen unless the device stalls a running workgroup for
 *             milliseconds): perm and offsets are then invalid, and
 *             engram_gather_reduce in dedup mode treats the groups as empty.
 *             The bound is 262,144 polls per wait; the environment variable
 *             ENGRAM_DEDUP_SPIN_LIMIT, read at each call, overrides it (a
 *             test forces the give-up path with a small value).
 *   ws        device workspace of ws_bytes >= engram_dedup_workspace(plan,
 *             n_tok), 256-byte aligned, owned by the caller.  It keeps a
 *             small state between calls (no clearing needed, initial
 *             contents arbitrary); one call at a time may use it.
 *
 * n_tok == 0 writes offsets[0] = 0 and *n_unique = 0.  Errors: EINVAL,
 * ERANGE (n_tok > 2^22 = 4,194,304: split larger batches), EWORKSPACE.
 */
int engram_dedup(engram_plan_t plan, const int32_t* ids, const int32_t* history,
                 int64_t n_seq, int64_t seq_len, int32_t* perm, int32_t* offsets,
                 int32_t* n_unique, void* ws, size_t ws_bytes, void* stream);

/*
 * Opt-in input check: count, on the device and without faulting, the
 * contract violations the lookup calls do not check: the row addresses are
 * read as given [GUIDE "Engram"], and ids index the vocabulary map.  Reads
 * only ids, history and addr (never a table or the map), so it is safe on
 * any values.
 *
 *   ids, history, n_seq, seq_len   as for engram_hash, or ids == NULL (then
 *             history must be NULL too) to skip the id check.
 *   addr      device uint32 [n_addr_tok][48] as engram_hash writes it,
 *             16-byte aligned, or NULL to skip the address check.
 *   counts    device int32 [3], 4-byte aligned (output, overwritten):
 *             counts[0] = ids and history ids below 0,
 *             counts[1] = ids and history ids >= the plan's vocab_size
 *                         (always 0 when vocab_size is 0),
 *             counts[2] = addresses addr[t][s] >= R_s.
 *
 * Two launches on the stream (clear, count); no synchronisation.  Errors:
 * EINVAL (NULL plan or counts, misaligned pointer, history without ids),
 * ERANGE (a token count out of range).
 */
int engram_check_inputs(engram_plan_t plan, const int32_t* ids, const int32_t* history,
                        int64_t n_seq, int64_t seq_len, const uint32_t* addr, int64_t n_addr_tok,
                        int32_t* counts, void* stream);

/*
 * engram_dedup for callers that cannot allocate device memory (code under
 * HIP graph capture that forbids allocation, tight serving loops, harnesses
 * that disallow hipMalloc): the same kernels and results, with the workspace
 * in a fixed array of ENGRAM_DEDUP_SCRATCH_BYTES that the library holds on
 * every GPU it runs on until the process ends.  The call itself allocates
 * nothing.  Arguments, outputs and errors are those of engram_dedup, without
 * ws and ws_bytes; a batch whose workspace (engram_dedup_workspace) exceeds
 * the fixed size returns ENGRAM_EWORKSPACE before anything is launched
 * (524,288 tokens fit under any plan).  All calls on one GPU share that
 * GPU's array: calls that overlap in time on one GPU (two streams, two host
 * threads) race and give wrong groups; serialise them.  The first call on a
 * device looks up the array's address there (hipGetSymbolAddress).
 */
#define ENGRAM_DEDUP_SCRATCH_BYTES (32u << 20)
int engram_dedup_noalloc(engram_plan_t plan, const int32_t* ids, const int32_t* history,
                         int64_t n_seq, int64_t seq_len, int32_t* perm, int32_t* offsets,
                         int32_t* n_unique, void* stream);

/*
 * Serving operators: the attention layer that reads the same tokens as the
 * lookup.  With the tables resident, the rest of a GPU's memory is the
 * requests' KV cache [VRAM; GUIDE "Where the 510 GB goes"]; these calls norm
 * and rotate the heads of new tokens, append keys and values to a paged cache
 * and attend over it.  They use no plan.  Conventions as above; descriptions
 * are host structures read during the call, and every reserved field must
 * be 0.  q, k, v and out are [n_tok][heads][head_dim] with any token and head
 * stride (elements, multiples of 8, not negative) and 16-byte aligned, so
 * that the slices of one projection's output can be passed as they are.
 */

/* Element types.  The 8-bit ones only as a cache's type, fp32 only for probabilities. */
#define ENGRAM_BF16 0
#define ENGRAM_F16 1
#define ENGRAM_E4M3 2      /* OCP, a scale for each row                  */
#define ENGRAM_E4M3_PAGE 4 /* OCP, a scale for each page and head        */
#define ENGRAM_I8_PAGE 5   /* int8, a scale for each page and head       */
#define ENGRAM_F32 6

/*
 * A paged cache: K and V each [n_pages][n_kv_heads][page_size][head_dim] of
 * `type`; pages are k_page_stride and v_page_stride elements apart (multiples
 * of 16, at least one page's size; K and V may be halves of one allocation).
 * An ENGRAM_E4M3 cache holds FP8 codes and one fp32 scale for each (page,
 * head, slot), k_scale and v_scale [n_pages][n_kv_heads][page_size]: a row
 * stands for codes * scale, as a table row does.  ENGRAM_E4M3_PAGE and
 * ENGRAM_I8_PAGE have one fp32 scale for each (page, head), k_scale and
 * v_scale [n_pages][n_kv_heads], and codes of FP8 or int8; any finite scale is
 * read, and engram_kv_append_pages writes powers of two.
 *
 *   page_size   a power of two from 8 to 1024; head_dim 64, 128 or 256;
 *               n_kv_heads 1 to 65535; n_pages 1 to 2^31 - 1.
 * All pointers 16-byte aligned.
 */
typedef struct engram_kv_cache {
    void* k;
    void* v;
    float* k_scale;               /* NULL for BF16 and F16 */
    float* v_scale;
    int64_t k_page_stride;
    int64_t v_page_stride;
    int64_t n_pages;
    uint32_t n_kv_heads;
    uint32_t page_size;
    uint32_t head_dim;
    uint32_t type;
} engram_kv_cache;

/*
 * Norm and rotation of query and key heads, in one pass:
 *     y = x * rsqrt(mean(x^2) + eps) * weight        (no weight: y = x)
 *     (y_a, y_b) -> (y_a cos t - y_b sin t, y_a sin t + y_b cos t),
 *     t = positions[tok] * inv_freq[i], i = 0 .. rotary_dim/2 - 1,
 * (a, b) = (i, i + rotary_dim/2), or (2i, 2i + 1) with interleaved = 1;
 * elements from rotary_dim on are not rotated.  fp32 arithmetic (angles,
 * cosines and sines in fp64, these rounded to fp32), rounded once to `type`.  An output may be its input (same strides);
 * otherwise they must not overlap.
 *
 *   head_dim    64, 128 or 256.  rotary_dim: a multiple of 16, at most
 *               head_dim; 0 for none (positions and inv_freq may be NULL).
 *   n_q_heads, n_k_heads   0 to 65535; 0 leaves that side out.
 *   q_weight, k_weight     device [head_dim] of `type`, 16-byte aligned, or NULL.
 *   positions   device int32 [n_tok], any value.
 *   inv_freq    device double [rotary_dim / 2]; |t| below 2^50.
 *
 * n_tok == 0 is a no-op.  Errors: EINVAL, ERANGE (n_tok > 2^31 - 1, a head
 * count above 65535), EUNSUPPORTED (type, head_dim).
 */
typedef struct engram_norm_rope_desc {
    const void* q;
    const void* k;
    void* q_out;
    void* k_out;
    const void* q_weight;
    const void* k_weight;
    const int32_t* positions;
    const double* inv_freq;
    int64_t n_tok;
    int64_t q_token_stride, q_head_stride;
    int64_t k_token_stride, k_head_stride;
    int64_t q_out_token_stride, q_out_head_stride;
    int64_t k_out_token_stride, k_out_head_stride;
    uint32_t n_q_heads, n_k_heads;
    uint32_t head_dim;
    uint32_t rotary_dim;
    uint32_t interleaved;
    uint32_t type;
    float eps;
    uint32_t reserved0;
} engram_norm_rope_desc;

int engram_qk_norm_rope(const engram_norm_rope_desc* desc, void* stream);

/*
 * Append new keys and values to a paged cache.  The key of token i (normed
 * if k_weight is given, rotated if rotary_dim > 0, both as above) and its
 * value go to page slots[i] / page_size, place slots[i] % page_size.  A
 * negative slot, or one past the pool, writes nothing (a batch's padding).
 * Two tokens of one call must not name the same slot.
 *   type of k, v and the cache: equal, or an ENGRAM_E4M3 cache, where each
 * row x is stored as scale = max|x| / 448 and the codes nearest to
 * x * 448 / max|x| (ties to even); a row of zeros has scale 0, and a NaN in
 * a row makes its scale NaN.  Nothing but the named rows (and their scales) is
 * written.
 *
 *   slots       device int64 [n_tok], 8-byte aligned.
 *
 * n_tok == 0 is a no-op.  Errors: EINVAL, ERANGE, EUNSUPPORTED (a type or
 * geometry other than the above).
 */
typedef struct engram_append_desc {
    const engram_kv_cache* cache;
    const void* k;
    const void* v;
    const void* k_weight;
    const int32_t* positions;
    const double* inv_freq;
    const int64_t* slots;
    int64_t n_tok;
    int64_t k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
    uint32_t rotary_dim;
    uint32_t interleaved;
    uint32_t type;
    float eps;
    uint32_t reserved0;
    uint32_t reserved1;
} engram_append_desc;

int engram_kv_append(const engram_append_desc* desc, void* stream);

/*
 * The append for caches with a scale for each page and head (ENGRAM_E4M3_PAGE,
 * ENGRAM_I8_PAGE).  As in the attention below, request b has the tokens
 * cu_q[b] .. cu_q[b + 1] - 1 (cu_q NULL: n_tok / n_seq each), which are the
 * last of its kv_len[b] keys, on the pages of block_table[b].  Keys are normed
 * and rotated as in engram_kv_append.  For every page, head and side with new
 * rows x (fp32, M = 448 for e4m3, 127 for int8):
 *     need  = the least power of two (2^-126 at least) with max|x| <= need * M,
 *             0 for a page of zeros, NaN where an x is infinite or NaN
 *     scale = need where the first new row is the page's first, else need where
 *             that is above the magnitude of the scale held, else that scale; a
 *             NaN stays
 *     codes = x / scale, rounded to nearest, ties to even; where the scale grew,
 *             codes of the rows held before are multiplied by old / new and
 *             rounded again (codes under a scale that is 0 or NaN: unspecified
 *             but for zeros under 0).  Under a scale from elsewhere that is no
 *             power of two x is multiplied by 1 / scale, rounded to fp32, so that
 *             next to a border it may have the neighbouring code; int8 codes of
 *             -128 count as -127 where a negative scale gives way.
 * Rows of a page before a request's first new token count as held, those after
 * its last do not and are left as they are: a request whose tokens were
 * refused appends over them.  A token before the request's first key, and one
 * on a page number outside the pool, is left out; those past the first max_q_len
 * (0: not known) of a request may be.  kv_len is bounded by table_width *
 * page_size, by 2^31 - 4096 and by 0.  A page is written for one request:
 * two requests of a call must not append to the same page.
 *
 * A token that is taken back, as a refused draft is, leaves its mark on its
 * page: the scale that it raised stays, for the rows held, which were rounded
 * again under it, and for those that follow; an infinity or NaN in it leaves the
 * page's scale, and so all rows of that page and head, NaN.  Both end when the
 * page's first row is written anew.
 *
 * n_tok == 0 is a no-op.  Errors: EINVAL, ERANGE (n_tok / page_size + 2 n_seq
 * pages times n_kv_heads / 2, or n_seq * n_kv_heads of single tokens, may be
 * refused above 2^23: split the batch), EUNSUPPORTED (a type
 * or geometry other than the above).
 */
typedef struct engram_append_pages_desc {
    const engram_kv_cache* cache;
    const void* k;
    const void* v;
    const void* k_weight;
    const int32_t* positions;
    const double* inv_freq;
    const int32_t* block_table;
    const int32_t* kv_len;
    const int32_t* cu_q;
    int64_t n_seq;
    int64_t n_tok;
    int64_t max_q_len;
    int64_t table_width;
    int64_t table_stride;
    int64_t k_token_stride, k_head_stride;
    int64_t v_token_stride, v_head_stride;
    uint32_t rotary_dim;
    uint32_t interleaved;
    uint32_t type;
    float eps;
    uint32_t reserved0;
} engram_append_pages_desc;

int engram_kv_append_pages(const engram_append_pages_desc* desc, void* stream);

/*
 * Attention of new tokens over a paged cache that already holds them.
 * Request b has the q_len tokens cu_q[b] .. cu_q[b + 1] - 1 of q (cu_q NULL:
 * n_tok / n_seq each) and kv_len[b] cached keys; key j lies on page
 * block_table[b][j / page_size], place j % page_size.  Its token i is at
 * position p = kv_len[b] - q_len + i and sees the keys j <= p, with a window
 * w > 0 those with j > p - w.  Query head h reads KV head
 * h / (n_q_heads / n_kv_heads):
 *     out = sum_j a_j v_j / sum_j a_j,  a_j = exp(scale * q . k_j - max),
 *     lse = log(sum_j exp(scale * q . k_j))            (natural)
 * A token that sees no key gets out = 0 and lse = -infinity.  What a token
 * does not see never reaches its result, NaN and infinities included.
 * Products of 16-bit operands with fp32 sums; softmax in fp32.  For the second
 * product a_j is held in about 16 bits where a request has at most 32 rows (new
 * tokens * n_q_heads / n_kv_heads), and rounded once to `type` where it has
 * more.  There, with bf16 queries over pages of codes with one scale, K's codes
 * times their page's scale are held as bf16: exactly where the scale is a power of
 * two, as the append writes them, else rounded once.  V's codes are exact, and a_j
 * is rounded to fp16's 11 bits, where the scales of V's pages that some hundred
 * rows see are 0 or powers of two from 2^-100 to 2^60, the largest 2^10 times the
 * smallest at most (2^27 / n where they see n > 2^17 keys).  Else V is held as K
 * is, and a_j rounded to bf16.
 *
 *   lse         device fp32 [n_tok][n_q_heads], or NULL.
 *   block_table device int32 [n_seq][table_width], rows table_stride apart.  A
 *               page number outside the pool is never read: its keys count
 *               as unseen.  kv_len is bounded by table_width * page_size, by
 *               2^31 - 4096 and by 0; entries past a request's last page are not read.
 *   max_q_len   a bound of the requests' q_len where cu_q is given, 0 if not
 *               known.  It and the requests' lengths decide which kernels run
 *               and how they divide the keys, and so the last bits of a
 *               result.  A request that is longer than it says may be left out
 *               (out and lse unwritten).
 *   window      0 for none.
 *   scale       finite.
 *   cu_q        device int32 [n_seq + 1], ascending from 0 to n_tok at most:
 *               tokens from cu_q[n_seq] on are no request's, and their out
 *               and lse are not written.  Other values leave results
 *               unspecified; nothing out of bounds is read or written.
 *   ws          device workspace of engram_paged_attention_workspace bytes
 *               (host-only; 0 for few keys), 256-byte aligned.  It holds
 *               nothing between calls; one call at a time may use it.
 *
 * Results are the same on every call with the same arguments.  n_tok == 0
 * is a no-op.  Errors: EINVAL, ERANGE (n_tok * n_q_heads > 2^31 - 1, or
 * n_tok * n_q_heads / 16 + n_seq * n_kv_heads > 2^23: split the batch),
 * EUNSUPPORTED, EWORKSPACE.
 */
typedef struct engram_attention_desc {
    const engram_kv_cache* cache;
    const void* q;
    void* out;
    float* lse;
    const int32_t* block_table;
    const int32_t* kv_len;
    const int32_t* cu_q;
    int64_t n_seq;
    int64_t n_tok;
    int64_t max_q_len;
    int64_t table_width;
    int64_t table_stride;
    int64_t window;
    int64_t q_token_stride, q_head_stride;
    int64_t out_token_stride, out_head_stride;
    uint32_t n_q_heads;
    uint32_t type;
    float scale;
    uint32_t reserved0;
} engram_attention_desc;

int engram_paged_attention_workspace(const engram_attention_desc* desc, size_t* bytes);
int engram_paged_attention(const engram_attention_desc* desc, void* ws, size_t ws_bytes, void* stream);

/*
 * Between two steps of a batch that decodes with drafted tokens: what a
 * server's bookkeeping would otherwise fetch to the host.  With these, a step
 * of lookup, attention and verification can be captured and replayed while the
 * requests grow.
 *
 * Page tables and slots.  Every request gets the pages that its length needs,
 * and its new tokens their slots.  Request b has lengths[b] keys and gets
 * new_tokens[b] more (new_tokens NULL: n_tok / n_seq each; negative numbers
 * count as 0), and holds the first held[b] pages of block_table[b]:
 *     need    = ceil((lengths + new_tokens) / page_size)
 *     tokens  = cu_q[b] .. cu_q[b + 1] - 1, cu_q the sum of new_tokens before
 *               b, n_tok at most
 *     pool    = pages past `need` of all requests, in order of request and
 *               place, then free_pages from free_pages[n_free - 1] down
 * A request that holds fewer than it needs takes the pool's next pages.  Pages
 * of the pool that came back and were not taken go on free_pages[n_free ..],
 * in order.  A request is served unless its tokens do not all fit into n_tok,
 * need exceeds table_width, its keys exceed 2^31 - 4096, or the pages that it
 * and those before it take are more than the pool has (one that takes none is
 * served all the same).  One that is not served keeps what it holds.
 * Outputs (of served requests, tokens i = 0 .. new - 1):
 *     slots[cu_q[b] + i]     = block_table[b][p / page_size] * page_size +
 *                              p % page_size, p = lengths + i
 *     positions[cu_q[b] + i] = p
 *     kv_len[b]              = lengths + new_tokens
 * else slot -1, position 0 and kv_len 0: the appends leave such tokens out, and
 * the attention gives them 0.  Tokens from cu_q[n_seq] on get slot -1 too.
 *     n_short = the number of requests that were not served
 * block_table, held, free_pages and n_free are brought up to date; entries of a
 * table past `held` are left as they are.
 *
 *   lengths, new_tokens, held, kv_len   device int32 [n_seq].  held is bounded
 *               by 0 and table_width.
 *   block_table device int32 [n_seq][table_width], rows table_stride apart.
 *   free_pages  device int32 [n_pages], n_free int32 [1] (bounded by 0 and
 *               n_pages): a stack; pages past its room are dropped.
 *   cu_q        device int32 [n_seq + 1]; slots int64, positions int32 [n_tok];
 *               n_short int32 [1].
 *   page_size   a power of two from 8 to 1024.
 *   ws          device workspace of engram_page_tables_workspace bytes
 *               (host-only; 0 for small batches), 256-byte aligned; holds
 *               nothing between calls; one call at a time may use it.
 * No output may overlap another or an input.  Errors: EINVAL, ERANGE (n_seq >
 * 2^20, n_tok >= 2^30, n_pages > 2^30), EUNSUPPORTED (page_size), EWORKSPACE.
 */
typedef struct engram_page_tables_desc {
    const int32_t* lengths;
    const int32_t* new_tokens;
    int32_t* block_table;
    int32_t* held;
    int32_t* free_pages;
    int32_t* n_free;
    int64_t* slots;
    int32_t* positions;
    int32_t* cu_q;
    int32_t* kv_len;
    int32_t* n_short;
    int64_t n_seq;
    int64_t n_tok;
    int64_t table_width;
    int64_t table_stride;
    int64_t n_pages;
    uint32_t page_size;
    uint32_t reserved0;
} engram_page_tables_desc;

int engram_page_tables_workspace(const engram_page_tables_desc* desc, size_t* bytes);
int engram_page_tables(const engram_page_tables_desc* desc, void* ws, size_t ws_bytes, void* stream);

/*
 * Verification of drafted tokens (speculative sampling): the tokens that a
 * step emits are distributed as the target's own.  Request b has the K drafts
 * cu_draft[b] .. cu_draft[b + 1] - 1 (cu_draft NULL: n_draft / n_seq each) and
 * the K + 1 target rows from cu_draft[b] + b on: row i the probabilities of
 * the token after i drafts.  With p_i a target row, q_i the drafter's
 * probabilities that draft d_i came from, u_i in [0, 1) its random number and v in
 * [0, 1) the request's:
 *     a     = the first i with not (u_i * q_i(d_i) < p_i(d_i)), else K
 *     w_j   = max(p_a(j) - q_a(j), 0) where a < K and their sum is not 0, else p_a(j)
 *     next  = the first j with w_0 + .. + w_j > v * (w_0 + .. + w_{vocab-1})
 *     tokens[cu_draft[b] + b ..] = d_0 .. d_{a-1}, next, then -1;  n_accepted[b] = a
 * draft_probs NULL: the drafts were certain (q_i is 1 at d_i, 0 elsewhere).
 * Products, differences and sums are fp64.  Rows need not be normalised.  A
 * draft that is no word (negative, or vocab and above) is refused; a negative
 * or NaN probability counts as 0, the target's and the drafter's; next is -1
 * where the row's sum is not positive and finite, and always a word with a weight
 * where it is.
 *
 *   target      device [n_draft + n_seq][vocab] of `type` (ENGRAM_F32, BF16 or
 *               F16), rows target_stride elements apart, aligned as its elements.
 *   draft_probs device [n_draft][vocab] of `type`, rows draft_stride apart.
 *   draft       device int32 [n_draft]; uniform fp32 [n_draft]; last_uniform
 *               fp32 [n_seq].
 *   cu_draft    device int32 [n_seq + 1], ascending from 0 to n_draft; other
 *               values leave results unspecified, and nothing out of bounds is
 *               read or written.
 *   tokens      device int32 [n_draft + n_seq], n_accepted int32 [n_seq].
 *   ws          device workspace of engram_verify_draft_workspace bytes
 *               (host-only; 0 for small vocabularies), 256-byte aligned; holds
 *               nothing between calls; one call at a time may use it.
 *
 * Results are the same on every call with the same arguments.  n_seq == 0 is a
 * no-op.  Errors: EINVAL, ERANGE (n_seq > 2^20, n_draft or vocab > 2^30, n_seq *
 * vocab / 4096 > 2^23: split the batch), EUNSUPPORTED (type), EWORKSPACE.
 */
typedef struct engram_verify_draft_desc {
    const void* target;
    const void* draft_probs;
    const int32_t* draft;
    const float* uniform;
    const float* last_uniform;
    const int32_t* cu_draft;
    int32_t* tokens;
    int32_t* n_accepted;
    int64_t n_seq;
    int64_t n_draft;
    int64_t vocab;
    int64_t target_stride;
    int64_t draft_stride;
    uint32_t type;
    uint32_t reserved0;
} engram_verify_draft_desc;

int engram_verify_draft_workspace(const engram_verify_draft_desc* desc, size_t* bytes);
int engram_verify_draft(const engram_verify_draft_desc* desc, void* ws, size_t ws_bytes, void* stream);

/* Static, human-readable name of a status code. */
const char* engram_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* ENGRAM_H */
