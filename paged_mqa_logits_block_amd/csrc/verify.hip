// Verification of drafted tokens: of each request's drafts the first ones with
// u q(x) < p(x) are kept, and one token more is taken from max(p - q, 0) where a draft
// was rejected, else from the last p, by the inverse of its cumulative sums.
//
// A row of weights is added up in spans of kVerifySpan entries, one wave to a span, in
// 64 bits (of softmax rows of 50,021 normal numbers, sums in 32 bits from the first entry on
// moved 3 tokens in a hundred, of 131,072 19), always in the same order; the token lies in
// the first span whose cumulative sum passes u * total, which is read once more for its
// place inside.  A weight p - q is rounded once to 32 bits, as p and q are: it is exact where they
// are within a factor of 2, else off by at most 2^-24 of itself.
//
// What bounds it is the bytes of one row of p, and of q where a draft was rejected, per
// request: rows of drafts that were kept or not reached are not read.  Measured, spans over
// the chip and then the search: 257 requests of 100,003 entries (161 MB) 29 us at 5.6 TB/s,
// and 4.8; 9 of 131,072 4.7 and 4.1, 1 of 50,021 4.4 and 3.6, where latency bounds both: the
// starts, the drafts' entries, the row and its sum follow one another.
#include "qsa_device.h"
#include "step_internal.h"

namespace qsa {
namespace {

constexpr int kMaxSpans = kVerifyMaxVocab / kVerifySpan;

struct Verdict {
    int row0, rows, kept;  // rows: at most max_tokens are looked at
    bool every;            // all drafts were kept
};

__device__ __forceinline__ Verdict rows_of(const VerifyArgs &a, int req) {
    Verdict v = {};
    v.row0 = min(max(a.q_starts[req], 0), a.num_rows);
    v.rows = min(min(max(a.q_starts[req + 1], 0), a.num_rows) - v.row0, a.max_tokens);
    return v;
}

// by a whole wave
__device__ __forceinline__ Verdict judge(const VerifyArgs &a, int req) {
    Verdict v = rows_of(a, req);
    const int drafts = v.rows - 1;
    while (v.kept < drafts) {
        const int j = v.kept + lane_id();
        bool good = false;
        if (j < drafts) {
            const int64_t row = v.row0 + j;
            const int x = a.tokens[row + 1];
            if (x >= 0 && x < a.vocab) {
                const double q = a.draft_probs ? (double)a.draft_probs[row * a.draft_row + x] : 1.0;
                good = (double)a.uniforms[row] * q < (double)a.probs[row * a.prob_row + x];
            }
        }
        const uint64_t bad = ~ballot(good);
        if (bad) {
            v.kept += __builtin_ctzll(bad);
            break;
        }
        v.kept += kWave;
    }
    v.every = v.kept >= drafts;
    return v;
}

// The weights of a request's next token: p, less q where that is not null.
struct Weights {
    const float *p, *q;
    int without;  // an entry of weight 0, or -1
};
__device__ __forceinline__ Weights weights_of(const VerifyArgs &a, const Verdict &v) {
    const int64_t row = v.row0 + v.kept;
    Weights w = {a.probs + row * a.prob_row, nullptr, -1};
    if (!v.every) {
        if (a.draft_probs) w.q = a.draft_probs + row * a.draft_row;
        else w.without = a.tokens[row + 1];
    }
    return w;
}

// What is not a positive number has no weight: as unsigned numbers, the bits of infinity,
// of NaN and of everything with a sign are not below those of infinity.
__device__ __forceinline__ float weight(float x) { return __float_as_uint(x) < 0x7F800000u ? x : 0.0f; }

typedef float Entries __attribute__((ext_vector_type(4), aligned(4)));  // rows start at any element

// the weights of 4 entries from `at` on, 0 behind the vocabulary
__device__ __forceinline__ void load_weights(const Weights &w, int vocab, int at, float (&x)[4]) {
    if (at + 4 <= vocab) {
        const Entries p = *reinterpret_cast<const Entries *>(w.p + at);
        if (w.q) {
            const Entries q = *reinterpret_cast<const Entries *>(w.q + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = p[i] - q[i];
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = p[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = 0.0f;
            if (at + i < vocab) x[i] = w.p[at + i] - (w.q ? w.q[at + i] : 0.0f);
        }
    }
    if (w.without >= 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = at + i == w.without ? 0.0f : x[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = weight(x[i]);
}

// v plus v of the lane that the DPP pattern takes from (0 where there is none)
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
    const int64_t b = __builtin_bit_cast(int64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, ROWS, 0xF, false);
    return v + __builtin_bit_cast(double, (int64_t)((uint64_t)hi << 32 | lo));
}
// Inclusive sums over the wave, in the order of the six steps (LDS permutations and two
// sums per entry in their place took 1 us more per call).  All lanes active.
__device__ __forceinline__ double wave_incl_sum_d(double v) {
    v = dpp_add<kDppRowShr1, 0xF>(v);
    v = dpp_add<kDppRowShr2, 0xF>(v);
    v = dpp_add<kDppRowShr4, 0xF>(v);
    v = dpp_add<kDppRowShr8, 0xF>(v);
    v = dpp_add<kDppRowBcast15, 0xA>(v);
    return dpp_add<kDppRowBcast31, 0xC>(v);
}
// the value of the lane before, 0 in lane 0
__device__ __forceinline__ double lane_before_d(double v) {
    constexpr int kDppWaveShr1 = 0x138;
    const int64_t b = __builtin_bit_cast(int64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)b, kDppWaveShr1, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), kDppWaveShr1, 0xF, 0xF, false);
    return __builtin_bit_cast(double, (int64_t)((uint64_t)hi << 32 | lo));
}

// a span's sum, by one wave; in the last lane
__device__ __forceinline__ double span_sum(const Weights &w, int vocab, int span) {
    constexpr int kSteps = kVerifySpan / (4 * kWave);
    double sum[2] = {0.0, 0.0};
    float x[kSteps][4];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) load_weights(w, vocab, span * kVerifySpan + 4 * (kWave * i + lane_id()), x[i]);
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j & 1] += (double)x[i][j];
    return wave_incl_sum_d(sum[0] + sum[1]);
}

// What the workgroup's threads share while they look for the token.
template <int THREADS>
struct Search {
    double wave_sum[2][THREADS / kWave], base;
    uint32_t key[2][THREADS / kWave];
    double spans[kMaxSpans];
};

// Of the threads' `first` (an index, or INT_MAX) the least, or where none has one the
// largest `last` (-1: none).
template <int THREADS>
__device__ __forceinline__ int block_pick(uint32_t (&key)[THREADS / kWave], int first, int last) {
    uint32_t k = wave_total_umax(first != 0x7FFFFFFF ? 0xFFFFFFFFu - (uint32_t)first : (uint32_t)(last + 1));
    if (lane_id() == 0) key[threadIdx.x >> 6] = k;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / kWave; ++i) k = max(k, key[i]);
    return k & 0x80000000u ? (int)(0xFFFFFFFFu - k) : (int)k - 1;
}

// the sum of the threads before this one; total: of all
template <int THREADS>
__device__ __forceinline__ double block_before(double (&wave_sum)[THREADS / kWave], double v, double &total) {
    const int wave = threadIdx.x >> 6;
    const double inc = wave_incl_sum_d(v);
    if (lane_id() == kWave - 1) wave_sum[wave] = inc;
    __syncthreads();
    double before = 0.0;
    total = 0.0;
#pragma unroll
    for (int i = 0; i < THREADS / kWave; ++i) {
        const double x = wave_sum[i];
        before += i < wave ? x : 0.0;
        total += x;
    }
    return before + lane_before_d(inc);
}

// The entry of the weights in which u falls, from their spans' sums, by the workgroup: the
// first one whose cumulative weight passes u * total, or the last one with weight; -1
// where none has any.
template <int THREADS>
__device__ __forceinline__ int find(const VerifyArgs &a, Search<THREADS> &sh, const double *spans, const Weights &w,
                                    float u) {
    constexpr int kPer = (kMaxSpans + THREADS - 1) / THREADS, kEach = kVerifySpan / THREADS;
    const int t = threadIdx.x;
    double s[kPer], sum = 0.0, total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        s[i] = kPer * t + i < a.spans ? spans[kPer * t + i] : 0.0;
        sum += s[i];
    }
    const double begin = block_before<THREADS>(sh.wave_sum[0], sum, total);
    if (!(total > 0.0)) return -1;
    const double goal = (double)u * total;
    int first = 0x7FFFFFFF, last = -1;
    double at = begin;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        at += s[i];
        if (s[i] > 0.0) {
            last = kPer * t + i;
            if (at > goal) first = min(first, last);
        }
    }
    const int span = block_pick<THREADS>(sh.key[0], first, last);
    if (span / kPer == t) {  // this thread has the cumulative weight before the span
        at = begin;
#pragma unroll
        for (int i = 0; i < kPer - 1; ++i)
            if (i < span % kPer) at += s[i];
        sh.base = at;
    }
    static_assert(kEach % 4 == 0, "whole loads of 4 entries");
    float x[kEach / 4][4];
    double in = 0.0;
#pragma unroll
    for (int i = 0; i < kEach / 4; ++i) {
        load_weights(w, a.vocab, span * kVerifySpan + kEach * t + 4 * i, x[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) in += (double)x[i][j];
    }
    at = block_before<THREADS>(sh.wave_sum[1], in, total);
    at += sh.base;
    first = 0x7FFFFFFF;
    last = -1;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const float v = x[i / 4][i % 4];
        at += (double)v;
        if (v > 0.0f) {
            last = span * kVerifySpan + kEach * t + i;
            if (at > goal) first = min(first, last);
        }
    }
    return block_pick<THREADS>(sh.key[1], first, last);
}

// all spans' sums, by the workgroup
template <int THREADS>
__device__ __forceinline__ void all_spans(const VerifyArgs &a, Search<THREADS> &sh, const Weights &w) {
    for (int s = threadIdx.x >> 6; s < a.spans; s += THREADS / kWave) {
        const double x = span_sum(w, a.vocab, s);
        if (lane_id() == kWave - 1) sh.spans[s] = x;
    }
    __syncthreads();
}

// A request's next token; spans: their sums, or null.
template <int THREADS>
__device__ __forceinline__ int next_token(const VerifyArgs &a, Search<THREADS> &sh, const Verdict &v, int req,
                                          const double *spans) {
    Weights w = weights_of(a, v);
    const float u = a.sample_uniforms[req];
    int token;
    if (!spans) all_spans<THREADS>(a, sh, w);
    token = find<THREADS>(a, sh, spans ? spans : sh.spans, w, u);
    if (token >= 0 || v.every) return token;
    // p is nowhere above q (or has no weight but the rejected draft's): a token of p
    w.q = nullptr;
    w.without = -1;
    __syncthreads();  // find has returned before its second use of what it shares
    all_spans<THREADS>(a, sh, w);
    return find<THREADS>(a, sh, sh.spans, w, u);
}

template <int THREADS>
__device__ __forceinline__ void write_tokens(const VerifyArgs &a, int req, const Verdict &v, int token) {
    int32_t *out = a.out_tokens + (int64_t)req * a.max_tokens;
    for (int j = threadIdx.x; j < a.max_tokens; j += THREADS)
        out[j] = v.rows <= 0 || j > v.kept ? -1 : j < v.kept ? a.tokens[v.row0 + j + 1] : token;
    if (threadIdx.x == 0) a.num_tokens[req] = v.rows <= 0 ? 0 : v.kept + 1;
}

// one workgroup per request
constexpr int kWholeThreads = 512;
__global__ __launch_bounds__(kWholeThreads) void verify_kernel(VerifyArgs a) {
    __shared__ Search<kWholeThreads> sh;
    const int req = blockIdx.x;
    const Verdict v = judge(a, req);
    const int token = v.rows > 0 ? next_token<kWholeThreads>(a, sh, v, req, nullptr) : -1;
    write_tokens<kWholeThreads>(a, req, v, token);
}

// Split launch: a wave per span of every request, then a workgroup per request that looks
// for the token.  The workspace holds the spans' sums, then the drafts that each
// request keeps.
constexpr int kSplitThreads = 256;
__device__ __forceinline__ int32_t *kept_of(const VerifyArgs &a) {
    return reinterpret_cast<int32_t *>(a.part + (int64_t)a.num_reqs * a.spans);
}

__global__ __launch_bounds__(kSplitThreads) void verify_sums_kernel(VerifyArgs a) {
    const int req = blockIdx.y, span = (int)blockIdx.x * (kSplitThreads / kWave) + (threadIdx.x >> 6);
    if (span >= a.spans) return;
    const Verdict v = judge(a, req);
    if (span == 0 && lane_id() == 0) kept_of(a)[req] = v.kept;
    if (v.rows <= 0) return;
    const double x = span_sum(weights_of(a, v), a.vocab, span);
    if (lane_id() == kWave - 1) a.part[(int64_t)req * a.spans + span] = x;
}

__global__ __launch_bounds__(kSplitThreads) void verify_find_kernel(VerifyArgs a) {
    __shared__ Search<kSplitThreads> sh;
    const int req = blockIdx.x;
    Verdict v = rows_of(a, req);
    v.kept = kept_of(a)[req];
    v.every = v.kept >= v.rows - 1;
    const int token = v.rows > 0 ? next_token<kSplitThreads>(a, sh, v, req, a.part + (int64_t)req * a.spans) : -1;
    write_tokens<kSplitThreads>(a, req, v, token);
}

}  // namespace

hipError_t launch_verify(const VerifyArgs &a, hipStream_t s) {
    if (!a.part) {
        hipLaunchKernelGGL(verify_kernel, dim3((unsigned)a.num_reqs), dim3(kWholeThreads), 0, s, a);
        return hipGetLastError();
    }
    constexpr int kSpansPer = kSplitThreads / kWave;
    hipLaunchKernelGGL(verify_sums_kernel, dim3((unsigned)((a.spans + kSpansPer - 1) / kSpansPer), (unsigned)a.num_reqs),
                       dim3(kSplitThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(verify_find_kernel, dim3((unsigned)a.num_reqs), dim3(kSplitThreads), 0, s, a);
    return hipGetLastError();
}

int64_t verify_workspace_bytes(int64_t num_reqs, int64_t spans) { return num_reqs * (spans * (int64_t)sizeof(double) + 4); }

}  // namespace qsa
