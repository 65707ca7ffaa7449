// Page tables and slots of a step, from the requests' lengths.
//
//     need_b = ceil((length_b + new_b) / page)
//     surplus_b = max(held_b - need_b, 0),  take_b = max(need_b - held_b, 0)
//
// Page k of all that are taken, request after request, is page k of the pool:
// first the surplus pages that come back in this call, in their order, then
// the stack of free pages from its top.  So no entry of the table or the stack
// is both read and written in a call: what is read are places below held_b and
// the stack's top (only where fewer pages come back than are taken), what is
// written are places from held_b on and the stack above its top (only where
// more come back).  Every page can be dealt by itself, and a token's slot does
// not wait for the table.
//
// The lengths are read once and three sums run over the requests (tokens;
// pages that come back and that are taken): latency, not bandwidth, for any
// batch of a few tokens a request.  What grows with the tokens is the 12 bytes
// that each gets.
//
// Mapping: one workgroup makes the sums, a request to each of its 1,024
// threads (a run of requests where there are more).  In a small batch it also
// deals the pages and writes the slots, with the sums in LDS.  Else a second
// launch does that with the whole chip, a token or a page to a thread, which
// finds its request by bisection (of the offsets in LDS where they fit).
#include <algorithm>

#include "drafts.h"

namespace engram {
namespace {

constexpr uint32_t kThreads = 1024, kWaves = kThreads / 64;
constexpr uint32_t kCap = INT32_MAX;  // sums end here: more tokens or pages than a call may have, and two do not wrap
constexpr uint64_t kMostLength = INT32_MAX - 4095;  // keys of a request, as the attention takes them

__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return min(a + b, kCap); }

struct Before {
    uint32_t mine, all;  // the sum over the threads before this one, and over all
};

// sums: LDS of this scan alone.
__device__ __forceinline__ Before scan(uint32_t x, uint32_t* sums) {
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    uint32_t upto = min(x, kCap);
#pragma unroll
    for (uint32_t k = 1; k < 64; k <<= 1) {
        const uint32_t y = __shfl_up(upto, k);
        upto = add(upto, lane >= k ? y : 0u);
    }
    if (lane == 63u) sums[wave] = upto;
    const uint32_t prev = __shfl_up(upto, 1);
    __syncthreads();
    Before r = {lane ? prev : 0u, 0u};
#pragma unroll
    for (uint32_t w = 0; w < kWaves; ++w) {
        const uint32_t s = sums[w];
        r.mine = add(r.mine, w < wave ? s : 0u);
        r.all = add(r.all, s);
    }
    return r;
}

struct Asked {
    int32_t length, fresh, held;
};
__device__ __forceinline__ Asked asked(const TablesArgs& A, uint32_t b) {
    return {A.lengths[b], A.fresh ? A.fresh[b] : static_cast<int32_t>(A.uniform_new), A.held[b]};
}
__device__ __forceinline__ uint32_t new_of(const Asked& a) { return static_cast<uint32_t>(max(a.fresh, 0)); }

// What a request holds and gets; `upto` counts the tokens to its end.
struct Wish {
    uint32_t keys, need, held, surplus, take;
    bool fits;
};
__device__ __forceinline__ Wish wish(const TablesArgs& A, const Asked& a, uint32_t upto) {
    const uint32_t n = new_of(a);
    const uint64_t keys = static_cast<uint64_t>(max(a.length, 0)) + n;
    const uint64_t need = (keys + (uint64_t(1) << A.page_shift) - 1u) >> A.page_shift;
    Wish w;
    w.fits = (upto <= A.n_tok || n == 0u) && need <= A.width && keys <= kMostLength;
    w.keys = static_cast<uint32_t>(keys);
    w.need = static_cast<uint32_t>(need);
    w.held = min(static_cast<uint32_t>(max(a.held, 0)), A.width);
    w.surplus = w.fits && w.held > w.need ? w.held - w.need : 0u;
    w.take = w.fits && w.need > w.held ? w.need - w.held : 0u;
    return w;
}

// The sums as both launches see them, in LDS or in the workspace.
struct Sums {
    const uint32_t* cu;      // [n_seq + 1], tokens before a request
    const uint32_t* taken;   // [n_seq + 1], pages taken
    const uint32_t* back;    // [n_seq + 1], pages that come back
    const uint32_t* before;  // [n_seq], pages held before the call
    const uint32_t* keys;    // [n_seq], kv_len
    uint32_t n_taken, n_back, n_free;
};

// The last of the requests 0 .. n - 1 that begins at or before x (sums[0] <= x).
__device__ __forceinline__ uint32_t find(const uint32_t* sums, uint32_t n, uint32_t x) {
    uint32_t lo = 0;
    while (n > 1u) {
        const uint32_t half = n >> 1;
        const bool right = sums[lo + half] <= x;
        lo += right ? half : 0u;
        n = right ? n - half : half;
    }
    return lo;
}

__device__ __forceinline__ int32_t returned(const TablesArgs& A, const Sums& s, uint32_t r) {
    const uint32_t b = find(s.back, A.n_seq, r);
    const uint32_t place = s.before[b] - (s.back[b + 1] - s.back[b]) + (r - s.back[b]);
    return A.table[b * A.table_stride + min(place, A.width - 1u)];
}

__device__ __forceinline__ int32_t from_pool(const TablesArgs& A, const Sums& s, uint32_t k) {
    if (k < s.n_back) return returned(A, s, k);
    const uint32_t at = s.n_free - 1u - (k - s.n_back);
    return at < A.n_stack ? A.stack[at] : -1;
}

// Page k of the pool to its request, or (past those taken) back to the stack.
__device__ __forceinline__ void deal(const TablesArgs& A, const Sums& s, uint32_t k) {
    if (k < s.n_taken) {
        const uint32_t b = find(s.taken, A.n_seq, k);
        const uint32_t place = s.before[b] + (k - s.taken[b]);
        if (place < A.width) A.table[b * A.table_stride + place] = from_pool(A, s, k);
    } else {
        const uint32_t at = s.n_free + (k - s.n_taken);
        if (at < A.n_stack) A.stack[at] = returned(A, s, k);
    }
}

// kRun neighbouring tokens from t on: their request is looked for once, and then followed.
constexpr uint32_t kRun = 4;
__device__ __forceinline__ void place_tokens(const TablesArgs& A, const Sums& s, uint32_t t) {
    const uint32_t end = A.n_seq ? s.cu[A.n_seq] : 0u;
    uint32_t b = 0, b_end = 0, keys = 0, before = 0, taken = 0;
    if (t < end) b = find(s.cu, A.n_seq, t);
#pragma unroll
    for (uint32_t i = 0; i < kRun; ++i, ++t) {
        if (t >= A.n_tok) return;
        int64_t slot = -1;
        uint32_t pos = 0;
        if (t < end) {
            if (t >= b_end) {
                if (i) {
                    do ++b;
                    while (s.cu[b + 1] <= t);
                }
                b_end = s.cu[b + 1];
                keys = s.keys[b];
                before = s.before[b];
                taken = s.taken[b];
            }
            if (keys) {
                pos = keys - (b_end - t);
                const uint32_t j = pos >> A.page_shift;
                const int32_t page = j < before ? A.table[b * A.table_stride + j] : from_pool(A, s, taken + (j - before));
                slot = (static_cast<int64_t>(page) << A.page_shift) + (pos & ((1u << A.page_shift) - 1u));
            }
        }
        A.slots[t] = slot;
        A.positions[t] = static_cast<int32_t>(pos);
    }
}

template <bool kOne>
__global__ __launch_bounds__(kThreads) void tables_kernel(const TablesArgs A) {
    __shared__ uint32_t sm_sums[4][kWaves];
    __shared__ uint32_t sm_cu[kOne ? kOneRequests + 1 : 1], sm_taken[kOne ? kOneRequests + 1 : 1],
        sm_back[kOne ? kOneRequests + 1 : 1], sm_before[kOne ? kOneRequests : 1], sm_keys[kOne ? kOneRequests : 1];
    __shared__ uint32_t sm_taken_all;
    const uint32_t tid = threadIdx.x;
    const uint32_t per = kOne ? 1u : (A.n_seq + kThreads - 1u) / kThreads;
    const uint32_t b0 = min(tid * per, A.n_seq), b1 = min(b0 + per, A.n_seq);
    uint32_t* const taken = kOne ? sm_taken : A.ws;
    uint32_t* const back = kOne ? sm_back : A.ws + A.n_seq + 1;
    uint32_t* const before = kOne ? sm_before : A.ws + 2 * (A.n_seq + 1);
    const uint32_t n_free = min(static_cast<uint32_t>(max(*A.n_free, 0)), A.n_stack);
    Asked mine = {0, 0, 0};
    if (kOne && b0 < b1) mine = asked(A, b0);
    const auto request = [&](uint32_t b) { return kOne ? mine : asked(A, b); };

    uint32_t tokens = 0;
    for (uint32_t b = b0; b < b1; ++b) tokens = add(tokens, min(new_of(request(b)), kCap));
    const Before tok = scan(tokens, sm_sums[0]);

    uint32_t n_back = 0, n_take = 0, upto = tok.mine;
    for (uint32_t b = b0; b < b1; ++b) {
        const Asked a = request(b);
        upto = add(upto, min(new_of(a), kCap));
        const Wish w = wish(A, a, upto);
        n_back = add(n_back, w.surplus);
        n_take = add(n_take, w.take);
    }
    const Before backs = scan(n_back, sm_sums[1]), takes = scan(n_take, sm_sums[2]);

    const uint32_t there = add(n_free, backs.all);
    uint32_t back_at = backs.mine, take_at = takes.mine, dealt = 0, missed = 0;
    upto = tok.mine;
    for (uint32_t b = b0; b < b1; ++b) {
        const Asked a = request(b);
        const uint32_t from = upto;
        upto = add(upto, min(new_of(a), kCap));
        const Wish w = wish(A, a, upto);
        // those that take and are served come before those that take and are not
        const bool served = w.fits && (w.take == 0u || add(take_at, w.take) <= there);
        const uint32_t cu = min(from, A.n_tok), keys = served ? w.keys : 0u;
        taken[b] = take_at;
        back[b] = back_at;
        before[b] = w.held;
        if constexpr (kOne) {
            sm_cu[b] = cu;
            sm_keys[b] = keys;
        }
        A.cu_q[b] = static_cast<int32_t>(cu);
        A.kv_len[b] = static_cast<int32_t>(keys);
        if (served) A.held[b] = static_cast<int32_t>(w.need);
        dealt += served ? w.take : 0u;
        missed += served ? 0u : 1u;
        back_at = add(back_at, w.surplus);
        take_at = add(take_at, w.take);
    }
    if (tid == 0) {
        A.cu_q[A.n_seq] = static_cast<int32_t>(min(tok.all, A.n_tok));
        if constexpr (kOne) sm_cu[A.n_seq] = min(tok.all, A.n_tok);
        taken[A.n_seq] = takes.all;
        back[A.n_seq] = backs.all;
    }
    // the pages dealt and the requests that got none
    {
        const uint32_t lane = tid & 63u;
        uint32_t d = dealt, m = missed;
#pragma unroll
        for (int k = 1; k < 64; k <<= 1) {
            d = add(d, __shfl_xor(d, k));
            m += __shfl_xor(m, k);
        }
        if (lane == 0) {
            sm_sums[3][tid >> 6] = d;
            sm_sums[0][tid >> 6] = m;
        }
        __syncthreads();
        if (tid == 0) {
            uint32_t all = 0, none = 0;
            for (uint32_t w = 0; w < kWaves; ++w) {
                all = add(all, sm_sums[3][w]);
                none += sm_sums[0][w];
            }
            *A.n_short = static_cast<int32_t>(none);
            *A.n_free = static_cast<int32_t>(min(add(n_free, backs.all) - min(all, there), A.n_stack));
            if constexpr (kOne) {
                sm_taken_all = all;
            } else {
                uint32_t* const totals = before + A.n_seq;
                totals[0] = all;
                totals[1] = backs.all;
                totals[2] = n_free;
            }
        }
    }
    if constexpr (kOne) {
        __syncthreads();
        const Sums s = {sm_cu, sm_taken, sm_back, sm_before, sm_keys, sm_taken_all, backs.all, n_free};
        for (uint32_t t = tid * kRun; t < A.n_tok; t += kThreads * kRun) place_tokens(A, s, t);
        for (uint32_t k = tid; k < max(s.n_taken, s.n_back); k += kThreads) deal(A, s, k);
    }
}

constexpr uint32_t kSpreadThreads = 256, kSpreadTokens = kSpreadThreads * kRun;  // of a workgroup
constexpr uint32_t kStaged = 4096;  // requests whose offsets lie in LDS

__global__ __launch_bounds__(kSpreadThreads) void spread_kernel(const TablesArgs A, uint32_t token_groups) {
    __shared__ uint32_t sm_cu[kStaged + 1];
    const uint32_t* const cu = reinterpret_cast<const uint32_t*>(A.cu_q);
    const uint32_t* const before = A.ws + 2 * (A.n_seq + 1);
    const uint32_t* const totals = before + A.n_seq;
    Sums s = {cu, A.ws, A.ws + A.n_seq + 1, before, reinterpret_cast<const uint32_t*>(A.kv_len), totals[0], totals[1], totals[2]};
    if (blockIdx.x < token_groups) {
        if (A.n_seq <= kStaged) {
            for (uint32_t i = threadIdx.x; i <= A.n_seq; i += kSpreadThreads) sm_cu[i] = cu[i];
            __syncthreads();
            s.cu = sm_cu;
        }
        place_tokens(A, s, (blockIdx.x * kSpreadThreads + threadIdx.x) * kRun);
    } else {
        const uint32_t step = (gridDim.x - token_groups) * kSpreadThreads;
        for (uint32_t k = (blockIdx.x - token_groups) * kSpreadThreads + threadIdx.x; k < max(s.n_taken, s.n_back); k += step)
            deal(A, s, k);
    }
}

}  // namespace

hipError_t launch_page_tables(const TablesArgs& a, hipStream_t stream) {
    if (!a.ws) {
        hipLaunchKernelGGL(tables_kernel<true>, dim3(1), dim3(kThreads), 0, stream, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(tables_kernel<false>, dim3(1), dim3(kThreads), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const uint32_t tokens = (a.n_tok + kSpreadTokens - 1u) / kSpreadTokens;
    // pages that a batch is expected to deal; more take further turns
    const uint32_t pages = std::min((a.n_tok >> a.page_shift) + a.n_seq, 1u << 18);
    hipLaunchKernelGGL(spread_kernel, dim3(tokens + (pages + kSpreadThreads - 1u) / kSpreadThreads), dim3(kSpreadThreads), 0,
                       stream, a, tokens);
    return hipGetLastError();
}

}  // namespace engram
