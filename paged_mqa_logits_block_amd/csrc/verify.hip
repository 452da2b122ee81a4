// Verification of drafted tokens: of each request's drafts the first ones with
// u q(x) < p(x) are kept, and one token more is taken from max(p - q, 0) where a draft
// was rejected, else from the last p, by the inverse of its cumulative sums.
//
// A row of weights is added up in spans of kVerifySpan entries, one wave to a span, in
// 64 bits (a sum of 100,000 probabilities in 32 would move the chosen token), always in
// the same order; the token lies in the first span whose cumulative sum passes
// u * total, which is read once more for its place inside.
//
// What bounds it is the bytes of one row of p, and of q where a draft was rejected, per
// request: rows of drafts that were kept or not reached are not read.
#include "qsa_device.h"
#include "step_internal.h"

namespace qsa {
namespace {

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWaves = kVerifyThreads / kWave;
constexpr int kMaxSpans = kVerifyMaxVocab / kVerifySpan;
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));  // rows start at any element

struct Verdict {
    int row0, rows, kept;  // rows: at most max_tokens are looked at
    bool every;            // all drafts were kept
};

// by a whole wave
__device__ __forceinline__ Verdict judge(const VerifyArgs &a, int req) {
    Verdict v;
    v.row0 = min(max(a.q_starts[req], 0), a.num_rows);
    v.rows = min(min(max(a.q_starts[req + 1], 0), a.num_rows) - v.row0, a.max_tokens);
    const int drafts = v.rows - 1;
    v.kept = 0;
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

// The weights of a request's next token.
struct Weights {
    const float *p, *q;  // q null: none, or the draft's alone
    int without;         // an entry of weight 0, or -1
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

// what is not a positive number has no weight
__device__ __forceinline__ float weight(float x) { return x > 0.0f && x < __builtin_inff() ? x : 0.0f; }

// four entries from `at` on (behind the vocabulary: weight 0): what p has over q, and p
__device__ __forceinline__ void load4(const Weights &w, int vocab, int at, float (&rest)[4], float (&target)[4]) {
    float p[4] = {0.0f, 0.0f, 0.0f, 0.0f}, q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (at + 4 <= vocab) {
        const f32x4 x = *reinterpret_cast<const f32x4_a4 *>(w.p + at);
        f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
        if (w.q) y = *reinterpret_cast<const f32x4_a4 *>(w.q + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[i] = x[i];
            q[i] = y[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (at + i >= vocab) continue;
            p[i] = w.p[at + i];
            if (w.q) q[i] = w.q[at + i];
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        target[i] = weight(p[i]);
        rest[i] = at + i == w.without ? 0.0f : weight(p[i] - q[i]);
    }
}

__device__ __forceinline__ double xor_lane_d(double v, int m) {
    const int64_t b = __builtin_bit_cast(int64_t, v);
    const uint32_t lo = (uint32_t)xor_lane_i((int)b, m), hi = (uint32_t)xor_lane_i((int)(b >> 32), m);
    return __builtin_bit_cast(double, (int64_t)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ double shfl_d(double v, int src) {
    const int64_t b = __builtin_bit_cast(int64_t, v);
    const uint32_t lo = (uint32_t)shfl_i((int)b, src), hi = (uint32_t)shfl_i((int)(b >> 32), src);
    return __builtin_bit_cast(double, (int64_t)((uint64_t)hi << 32 | lo));
}

// a span's sums of both kinds of weights, by one wave
struct Sums {
    double rest, target;
};
__device__ __forceinline__ Sums span_sums(const Weights &w, int vocab, int span) {
    constexpr int kSteps = kVerifySpan / (4 * kWave);
    Sums s = {0.0, 0.0};
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        float rest[4], target[4];
        load4(w, vocab, span * kVerifySpan + 4 * (kWave * i + lane_id()), rest, target);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s.rest += (double)rest[j];
            s.target += (double)target[j];
        }
    }
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) {
        s.rest += xor_lane_d(s.rest, m);
        s.target += xor_lane_d(s.target, m);
    }
    return s;
}

// What the workgroup's threads share while they look for the token.
struct Search {
    double wave_sum[kVerifyWaves];
    int32_t first[kVerifyWaves], last[kVerifyWaves];
};

// The sum of the threads before this one, and the total, in a fixed order.
__device__ __forceinline__ double block_before(Search &sh, double v, double &total) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    double inc = v;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const double u = shfl_d(inc, lane >= d ? lane - d : lane);
        if (lane >= d) inc += u;
    }
    __syncthreads();
    if (lane == kWave - 1) sh.wave_sum[wave] = inc;
    __syncthreads();
    double before = 0.0;
    total = 0.0;
    for (int i = 0; i < kVerifyWaves; ++i) {
        if (i < wave) before += sh.wave_sum[i];
        total += sh.wave_sum[i];
    }
    const double in = shfl_d(inc, lane > 0 ? lane - 1 : 0);  // exclusive
    return lane > 0 ? before + in : before;
}

// The least of the threads' `first`, or where all are INT_MAX the largest `last`.
__device__ __forceinline__ int block_pick(Search &sh, int first, int last) {
    const int t = threadIdx.x;
    first = -wave_max_i(-first);
    last = wave_max_i(last);
    __syncthreads();
    if ((t & 63) == 0) {
        sh.first[t >> 6] = first;
        sh.last[t >> 6] = last;
    }
    __syncthreads();
    for (int i = 0; i < kVerifyWaves; ++i) {
        first = min(first, sh.first[i]);
        last = max(last, sh.last[i]);
    }
    return first != 0x7FFFFFFF ? first : last;
}

// The request's next token from its spans' sums, by the workgroup: the first entry whose
// cumulative weight passes u * total, or the last one with weight, or -1.
__device__ __forceinline__ int choose(const VerifyArgs &a, Search &sh, const Sums *spans, const Weights &w, float u) {
    constexpr int kPer = kMaxSpans / kVerifyThreads, kEach = kVerifySpan / kVerifyThreads;
    const int t = threadIdx.x;
    double rest[kPer], target[kPer], sums[2] = {0.0, 0.0};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int s = kPer * t + i;
        rest[i] = s < a.spans ? spans[s].rest : 0.0;
        target[i] = s < a.spans ? spans[s].target : 0.0;
        sums[0] += rest[i];
        sums[1] += target[i];
    }
    double total, all;
    double before = block_before(sh, sums[0], total);
    const double other = block_before(sh, sums[1], all);
    const bool use_target = !(total > 0.0);  // p is nowhere above q
    if (use_target) {
        before = other;
        total = all;
    }
    if (!(total > 0.0)) return -1;
    const double goal = (double)u * total;
    int first = 0x7FFFFFFF, last = -1;
    double at = before, base = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const double s = use_target ? target[i] : rest[i];
        if (s > 0.0) {
            last = kPer * t + i;
            if (at + s > goal) first = min(first, kPer * t + i);
        }
        at += s;
    }
    const int span = block_pick(sh, first, last);
    // the cumulative sum before the span, from the thread that has it
    if (span / kPer == t) {
        base = before;
        for (int i = 0; i < span % kPer; ++i) base += use_target ? target[i] : rest[i];
        sh.wave_sum[0] = base;
    }
    __syncthreads();
    base = sh.wave_sum[0];
    __syncthreads();
    float x[kEach];
    double sum = 0.0, unused;
#pragma unroll
    for (int i = 0; i < kEach; i += 4) {
        float r[4], p[4];
        load4(w, a.vocab, span * kVerifySpan + kEach * t + i, r, p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[i + j] = use_target ? p[j] : r[j];
            sum += (double)x[i + j];
        }
    }
    at = base + block_before(sh, sum, unused);
    first = 0x7FFFFFFF;
    last = -1;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        at += (double)x[i];
        if (x[i] > 0.0f) {
            last = span * kVerifySpan + kEach * t + i;
            if (at > goal) first = min(first, last);
        }
    }
    return block_pick(sh, first, last);
}

__device__ __forceinline__ void write_tokens(const VerifyArgs &a, int req, const Verdict &v, int token) {
    int32_t *out = a.out_tokens + (int64_t)req * a.max_tokens;
    for (int j = threadIdx.x; j < a.max_tokens; j += kVerifyThreads)
        out[j] = v.rows <= 0 || j > v.kept ? -1 : j < v.kept ? a.tokens[v.row0 + j + 1] : token;
    if (threadIdx.x == 0) a.num_tokens[req] = v.rows <= 0 ? 0 : v.kept + 1;
}

// one workgroup per request
__global__ __launch_bounds__(kVerifyThreads) void verify_kernel(VerifyArgs a) {
    __shared__ Search sh;
    __shared__ Sums spans[kMaxSpans];
    const int req = blockIdx.x, wave = threadIdx.x >> 6;
    const Verdict v = judge(a, req);
    int token = -1;
    if (v.rows > 0) {
        const Weights w = weights_of(a, v);
        for (int s = wave; s < a.spans; s += kVerifyWaves) {
            const Sums x = span_sums(w, a.vocab, s);
            if (lane_id() == 0) spans[s] = x;
        }
        __syncthreads();
        token = choose(a, sh, spans, w, a.sample_uniforms[req]);
    }
    write_tokens(a, req, v, token);
}

hipError_t run_verify(const VerifyArgs &a, hipStream_t s) {
    hipLaunchKernelGGL(verify_kernel, dim3((unsigned)a.num_reqs), dim3(kVerifyThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_verify(const VerifyArgs &a, hipStream_t s) { return run_verify(a, s); }

}  // namespace qsa
