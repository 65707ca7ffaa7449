// Verification of drafted tokens.
//
// Request b has drafts d_0 .. d_{K-1}, the drafter's probabilities q_0 ..
// q_{K-1}, the target's p_0 .. p_K and random numbers u_0 .. u_{K-1}, v.
//     a = the first i < K with not (u_i q_i(d_i) < p_i(d_i)), else K
//     w_j = max(p_a(j) - q_a(j), 0)  (a < K),  p_K(j)  (a = K)
//     token = the first j with w_0 + .. + w_j > v (w_0 + .. + w_{V-1})
// Without q a draft was certain: q_i = 1 at d_i and 0 elsewhere.  Products,
// differences and sums are fp64: every product and comparison is exact, and a
// sum of a whole vocabulary is off by 1e-16 of itself, where the weight of one
// word may be 1e-6 and fp32 sums would now and then name its neighbour.
//
// The work is the reading of one row of p, and of q where a draft was refused:
// HBM-bound for a batch, latency for one request.  64 requests of 5 drafts over
// 129,280 words in fp32, 9 of 10 with a refused draft, take 19 to 20 us: 12 us of
// sums (62 MB, 5.3 TB/s) and 7.6 to choose the word; one request over 32,768
// words takes 9.5 to 10 us, over 4,096 words 6.4.
//
// Mapping: a row is taken in blocks of 4,096 words, 16 neighbours to each of
// 256 threads.  One launch sums the blocks, a second finds the block in which
// the sum passes v times the whole and reads that block again, thread sums
// first and then the words of one thread.  Both launches sum in the same order,
// so the block's end is the same number in both.  Rows of up to 16,384 words
// take one launch, a workgroup of 1,024 threads to a row (256 requests of 8,192
// words 8.1 us against 12.9 in two launches, one of 4,096 6.4 against 9.9, 64 of
// 16,384 9.7 against 10.7).  Eight words to a thread, or four waves on a SIMD
// for five, take the same.
// Which drafts are kept is a gather of K words, found anew by every workgroup
// of the first launch.
#include "drafts.h"
#include "serving.h"

namespace engram {
namespace {

constexpr uint32_t kWords = 16;             // of a thread
constexpr uint32_t kBlock = 256 * kWords;   // words of a block
constexpr uint32_t kWhole = 1024 * kWords;  // words of a row that one workgroup takes

struct F32 {
    static constexpr uint32_t kBytes = 4;
    static __device__ __forceinline__ float at(const uint8_t* row, uint32_t j) {
        return reinterpret_cast<const float*>(row)[j];
    }
};
template <class T>
struct Half {
    static constexpr uint32_t kBytes = 2;
    static __device__ __forceinline__ float at(const uint8_t* row, uint32_t j) {
        return T::lo(reinterpret_cast<const uint16_t*>(row)[j]);
    }
};

// kWords neighbouring words of a row as floats.  Rows start at any element: an odd vocabulary leaves them on none of the
// 16-byte lines, and the loads say so.
template <class E>
struct Words16 {
    float x[kWords];
};
typedef uint32_t u32x4a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4a2 __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ Words16<F32> load16(const uint8_t* row, uint32_t j0, F32) {
    Words16<F32> r;
    const u32x4a4* p = reinterpret_cast<const u32x4a4*>(row + static_cast<uint64_t>(j0) * 4);
#pragma unroll
    for (uint32_t i = 0; i < kWords / 4; ++i) {
        const u32x4a4 w = p[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) r.x[4 * i + e] = __builtin_bit_cast(float, static_cast<uint32_t>(w[e]));
    }
    return r;
}
template <class T>
__device__ __forceinline__ Words16<Half<T>> load16(const uint8_t* row, uint32_t j0, Half<T>) {
    Words16<Half<T>> r;
    const u32x4a2* p = reinterpret_cast<const u32x4a2*>(row + static_cast<uint64_t>(j0) * 2);
#pragma unroll
    for (uint32_t i = 0; i < kWords / 8; ++i) {
        const u32x4a2 w = p[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r.x[8 * i + 2 * e] = T::lo(w[e]);
            r.x[8 * i + 2 * e + 1] = T::hi(w[e]);
        }
    }
    return r;
}

// What a probability weighs: nothing if it is negative or NaN.
__device__ __forceinline__ float weighs(float x) { return fmaxf(x, 0.0f); }

// The drafts of a request, and what became of them.
struct Verdict {
    uint32_t first, count;   // drafts first .. first + count - 1
    uint32_t accepted;
    bool refused;
    uint32_t row;            // of the target, where the next token comes from
    uint32_t certain;        // the refused draft of a drafter that was certain, else none of the vocabulary
};

__device__ __forceinline__ Verdict drafts_of(const VerifyArgs& A, uint32_t b) {
    Verdict r = {};
    if (A.cu_draft) {
        const int32_t n = static_cast<int32_t>(A.n_draft);
        const int32_t from = min(max(A.cu_draft[b], 0), n), to = min(max(A.cu_draft[b + 1], from), n);
        r.first = static_cast<uint32_t>(from);
        r.count = static_cast<uint32_t>(to - from);
    } else {
        r.first = b * A.uniform_drafts;
        r.count = A.uniform_drafts;
    }
    return r;
}

// With `accepted` of them kept.
__device__ __forceinline__ Verdict kept(const VerifyArgs& A, Verdict r, uint32_t b, uint32_t accepted) {
    r.accepted = accepted;
    r.refused = accepted < r.count;
    r.row = r.first + accepted + b;
    r.certain = r.refused && !A.drafter ? static_cast<uint32_t>(A.draft[r.first + accepted]) : UINT32_MAX;
    return r;
}

template <class E>
__device__ __forceinline__ Verdict verdict_of(const VerifyArgs& A, uint32_t b) {
    const Verdict r = drafts_of(A, b);
    const uint32_t lane = threadIdx.x & 63u;
    uint32_t accepted = r.count;
    for (uint32_t i0 = 0; i0 < r.count; i0 += 64u) {
        const uint32_t i = i0 + lane;
        bool no = false;
        if (i < r.count) {
            const uint32_t t = r.first + i, d = static_cast<uint32_t>(A.draft[t]);
            float p = 0.0f, q = 1.0f;
            if (d < A.vocab) {
                p = weighs(E::at(A.target + static_cast<uint64_t>(t + b) * A.target_stride * E::kBytes, d));
                if (A.drafter) q = weighs(E::at(A.drafter + static_cast<uint64_t>(t) * A.drafter_stride * E::kBytes, d));
            }
            no = !(static_cast<double>(A.uniform[t]) * static_cast<double>(q) < static_cast<double>(p));
        }
        const uint64_t any = __ballot(no);
        if (any) {
            accepted = i0 + static_cast<uint32_t>(__builtin_ctzll(any));
            break;
        }
    }
    return kept(A, r, b, accepted);
}

// The two kinds of weights of a word.
struct Weight {
    double w, p;
};
__device__ __forceinline__ Weight weight_of(float p, float q, bool certain) {
    p = weighs(p);
    q = weighs(q);
    return {certain ? 0.0 : p > q ? static_cast<double>(p) - static_cast<double>(q) : 0.0, static_cast<double>(p)};
}

struct Rows {
    const uint8_t *p, *q;  // q: nullptr where the weights are p's
};
template <class E>
__device__ __forceinline__ Rows rows_of(const VerifyArgs& A, const Verdict& v) {
    return {A.target + static_cast<uint64_t>(v.row) * A.target_stride * E::kBytes,
            v.refused && A.drafter ? A.drafter + static_cast<uint64_t>(v.first + v.accepted) * A.drafter_stride * E::kBytes
                                   : nullptr};
}

// The sums of kWords words from j0 on.
template <class E>
__device__ __forceinline__ Weight sums_of(const VerifyArgs& A, const Rows& rows, uint32_t certain, uint32_t j0) {
    Weight s = {0.0, 0.0};
    if (j0 + kWords <= A.vocab) {
        const Words16<E> p = load16(rows.p, j0, E());
        if (rows.q) {
            const Words16<E> q = load16(rows.q, j0, E());
#pragma unroll
            for (uint32_t i = 0; i < kWords; ++i) {
                const Weight x = weight_of(p.x[i], q.x[i], false);
                s.w += x.w;
                s.p += x.p;
            }
        } else {
#pragma unroll
            for (uint32_t i = 0; i < kWords; ++i) {
                const Weight x = weight_of(p.x[i], 0.0f, j0 + i == certain);
                s.w += x.w;
                s.p += x.p;
            }
        }
    } else {
        for (uint32_t j = j0; j < A.vocab; ++j) {
            const Weight x = weight_of(E::at(rows.p, j), rows.q ? E::at(rows.q, j) : 0.0f, j == certain);
            s.w += x.w;
            s.p += x.p;
        }
    }
    return s;
}

__device__ __forceinline__ double shfl_up(double x, uint32_t k) { return __shfl_up(x, k); }

// Sums up to and with this thread, and of all; the same order of sums in every launch of kThreads.
template <uint32_t kThreads>
struct Scan {
    double wave_w[kThreads / 64], wave_p[kThreads / 64];
};
template <uint32_t kThreads>
__device__ __forceinline__ void scan(Scan<kThreads>& sm, Weight mine, Weight& upto, Weight& all) {
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    upto = mine;
#pragma unroll
    for (uint32_t k = 1; k < 64; k <<= 1) {
        const double w = shfl_up(upto.w, k), p = shfl_up(upto.p, k);
        upto.w += lane >= k ? w : 0.0;
        upto.p += lane >= k ? p : 0.0;
    }
    if (lane == 63u) {
        sm.wave_w[wave] = upto.w;
        sm.wave_p[wave] = upto.p;
    }
    __syncthreads();
    Weight before = {0.0, 0.0};
    all = {0.0, 0.0};
#pragma unroll
    for (uint32_t i = 0; i < kThreads / 64; ++i) {
        if (i == wave) before = all;
        all.w += sm.wave_w[i];
        all.p += sm.wave_p[i];
    }
    upto.w += before.w;
    upto.p += before.p;
}

__device__ __forceinline__ bool sound(double sum) { return sum > 0.0 && sum < __builtin_huge_val(); }

// The first of kWords words from j0 on, a lane's each, whose sum passes `goal`, else the last with a weight; `from`: the sum
// before j0.
template <class E>
__device__ __forceinline__ uint32_t word_of(const VerifyArgs& A, const Rows& rows, uint32_t certain, bool of_w, uint32_t j0,
                                            double from, double goal) {
    const uint32_t lane = threadIdx.x & 63u, j = j0 + lane;
    double w = 0.0;
    if (lane < kWords && j < A.vocab) {
        const Weight x = weight_of(E::at(rows.p, j), rows.q ? E::at(rows.q, j) : 0.0f, j == certain);
        w = of_w ? x.w : x.p;
    }
    double upto = w;
#pragma unroll
    for (uint32_t k = 1; k < kWords; k <<= 1) {
        const double y = __shfl_up(upto, k);
        upto += lane >= k ? y : 0.0;
    }
    const uint64_t pass = __ballot(w > 0.0 && from + upto > goal), some = __ballot(w > 0.0);
    return j0 + static_cast<uint32_t>(pass ? __builtin_ctzll(pass) : 63 - __builtin_clzll(some | 1u));
}

// The word at which a workgroup's sums pass the goal: the thread that holds it is found first (`w` its sum, `end` the sum to
// its end), and its wave takes its words apart.
template <class E>
__device__ __forceinline__ uint32_t choose(const VerifyArgs& A, const Rows& rows, uint32_t certain, bool of_w, uint32_t first,
                                           double w, double end, double goal, uint32_t* sm_found) {
    // the first thread that passes; else the last that holds anything
    const uint32_t rank = w > 0.0 ? (end > goal ? 4096u - threadIdx.x : 1u + threadIdx.x) : 0u;
    if (rank) atomicMax(sm_found, rank);
    __syncthreads();
    const uint32_t best = *sm_found;
    const uint64_t mine = __ballot(rank && rank == best);
    __syncthreads();
    if (mine) {
        const int l = __builtin_ctzll(mine);
        const uint32_t t = (threadIdx.x & ~63u) + static_cast<uint32_t>(l);
        const uint32_t word = word_of<E>(A, rows, certain, of_w, first + t * kWords, __shfl(end - w, l), goal);
        if ((threadIdx.x & 63u) == 0u) *sm_found = word;
    }
    __syncthreads();
    return *sm_found;
}

__device__ __forceinline__ double goal_of(float v, double all) { return v > 0.0f ? static_cast<double>(v) * all : 0.0; }

// Tokens of a request, by its first threads; `next`: the one after those accepted.
__device__ __forceinline__ void put(const VerifyArgs& A, const Verdict& v, uint32_t b, int32_t next, uint32_t threads) {
    for (uint32_t i = threadIdx.x; i <= v.count; i += threads)
        A.tokens[v.first + b + i] = i < v.accepted ? A.draft[v.first + i] : i == v.accepted ? next : -1;
    if (threadIdx.x == 0) A.accepted[b] = static_cast<int32_t>(v.accepted);
}

template <class E>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(5))) void sum_blocks_kernel(const VerifyArgs A) {
    __shared__ Scan<256> sm;
    const uint32_t b = blockIdx.x / A.blocks, block = blockIdx.x - b * A.blocks;
    const Verdict v = verdict_of<E>(A, b);
    Weight upto, all;
    scan(sm, sums_of<E>(A, rows_of<E>(A, v), v.certain, block * kBlock + threadIdx.x * kWords), upto, all);
    if (threadIdx.x == 0) {
        double* const to = A.ws + 2 * static_cast<uint64_t>(blockIdx.x);
        to[0] = all.w;
        to[1] = all.p;
        if (block == 0) A.accepted[b] = static_cast<int32_t>(v.accepted);
    }
}

template <class E>
__global__ __launch_bounds__(256) void choose_kernel(const VerifyArgs A) {
    __shared__ Scan<256> sm;
    __shared__ uint32_t sm_found;
    const uint32_t b = blockIdx.x, lane = threadIdx.x & 63u;
    const Verdict v = kept(A, drafts_of(A, b), b, static_cast<uint32_t>(A.accepted[b]));
    const Rows rows = rows_of<E>(A, v);
    const double* const sums = A.ws + 2 * static_cast<uint64_t>(b) * A.blocks;
    // every wave for itself: the whole sum, in a fixed order, then the block in which it passes the goal
    Weight whole = {0.0, 0.0};
    for (uint32_t i = lane; i < A.blocks; i += 64u) {
        whole.w += sums[2 * i];
        whole.p += sums[2 * i + 1];
    }
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
        whole.w += __shfl_xor(whole.w, k);
        whole.p += __shfl_xor(whole.p, k);
    }
    const bool of_w = v.refused && whole.w > 0.0;
    const double all = of_w ? whole.w : whole.p;
    if (!sound(all)) {
        put(A, v, b, -1, 256);
        return;
    }
    const double goal = goal_of(A.last[b], all);
    uint32_t block = 0;
    double before = 0.0, at = 0.0;
    bool done = false;
    for (uint32_t i0 = 0; i0 < A.blocks && !done; i0 += 64u) {
        const uint32_t i = i0 + lane;
        const double mine = i < A.blocks ? sums[2 * i + (of_w ? 0 : 1)] : 0.0;
        double upto = mine;
#pragma unroll
        for (uint32_t k = 1; k < 64; k <<= 1) {
            const double x = shfl_up(upto, k);
            upto += lane >= k ? x : 0.0;
        }
        upto += at;
        const uint64_t pass = __ballot(mine > 0.0 && upto > goal), some = __ballot(mine > 0.0);
        done = pass != 0;
        const uint64_t from = pass ? pass & (~pass + 1u) : some;  // the first that passes, else the last that holds anything
        if (from) {
            const int l = 63 - __builtin_clzll(from);
            block = i0 + static_cast<uint32_t>(l);
            before = __shfl(upto - mine, l);
        }
        at = __shfl(upto, 63);
    }
    const uint32_t j0 = block * kBlock + threadIdx.x * kWords;
    if (threadIdx.x == 0) sm_found = 0;
    const Weight mine = sums_of<E>(A, rows, v.certain, j0);
    Weight upto, of_block;
    scan(sm, mine, upto, of_block);
    const double w = of_w ? mine.w : mine.p, end = before + (of_w ? upto.w : upto.p);
    const uint32_t word = choose<E>(A, rows, v.certain, of_w, block * kBlock, w, end, goal, &sm_found);
    put(A, v, b, static_cast<int32_t>(word), 256);
}

template <class E>
__global__ __launch_bounds__(1024) void whole_kernel(const VerifyArgs A) {
    __shared__ Scan<1024> sm;
    __shared__ uint32_t sm_found;
    const uint32_t b = blockIdx.x;
    const Verdict v = verdict_of<E>(A, b);
    const Rows rows = rows_of<E>(A, v);
    const Weight mine = sums_of<E>(A, rows, v.certain, threadIdx.x * kWords);
    if (threadIdx.x == 0) sm_found = 0;
    Weight upto, whole;
    scan(sm, mine, upto, whole);
    const bool of_w = v.refused && whole.w > 0.0;
    const double all = of_w ? whole.w : whole.p;
    if (!sound(all)) {
        put(A, v, b, -1, 1024);
        return;
    }
    const double goal = goal_of(A.last[b], all);
    const double w = of_w ? mine.w : mine.p, end = of_w ? upto.w : upto.p;
    const uint32_t word = choose<E>(A, rows, v.certain, of_w, 0, w, end, goal, &sm_found);
    put(A, v, b, static_cast<int32_t>(word), 1024);
}

template <class E>
hipError_t verify_one(const VerifyArgs& a, hipStream_t stream) {
    if (!a.blocks) {
        hipLaunchKernelGGL(whole_kernel<E>, dim3(a.n_seq), dim3(1024), 0, stream, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(sum_blocks_kernel<E>, dim3(a.n_seq * a.blocks), dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(choose_kernel<E>, dim3(a.n_seq), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

uint32_t verify_blocks(uint64_t, uint64_t vocab) {
    return vocab <= kWhole ? 0u : static_cast<uint32_t>((vocab + kBlock - 1) / kBlock);
}

size_t verify_workspace(uint64_t n_seq, uint64_t vocab) {
    return (n_seq * verify_blocks(n_seq, vocab) * 16 + 255) & ~size_t(255);
}

hipError_t launch_verify_draft(const VerifyArgs& a, uint32_t type, hipStream_t stream) {
    switch (type) {
        case ENGRAM_F32: return verify_one<F32>(a, stream);
        case ENGRAM_BF16: return verify_one<Half<Bf16>>(a, stream);
        default: return verify_one<Half<F16>>(a, stream);
    }
}

}  // namespace engram
