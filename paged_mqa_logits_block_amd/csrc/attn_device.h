// Device-side parts shared by the attention kernels: operand types, the copies
// to LDS, the transposed reads and the score / output products of one wave.
//
// One wave works on 32 stacked (row, head) pairs and 32 keys at a time, with the
// 32x32x16 MFMA in transposed form:
//
//   S^T = K Q^T:  A = K (lane: key l & 31, elements 8 (l >> 5) .. + 7 of each 16),
//                 B = Q (lane: pair l & 31, the same elements)
//   O^T = V^T P^T: A = V^T (lane: output element l & 31), B = P^T
//
// A lane of the result holds one column, pair l & 31, and 16 of the 32 rows:
// register i is row 8 (i >> 2) + 4 (l >> 5) + (i & 3).  So each lane keeps the
// running maximum and sum of its own pair, a step's maximum needs one exchange
// (with lane l ^ 32), rescaling the output is a product by a value that the
// lane already has, and the scores feed the second product without moving
// between lanes: MFMA sums over its 16 inner elements in any order, so inner
// element 8 (l >> 5) + j of step t stands for key 16 t + 4 (l >> 5) + j (j < 4) or
// 16 t + 8 + 4 (l >> 5) + j - 4, which are registers 8 t .. 8 t + 7 of the scores.
#pragma once

#include "attn_internal.h"
#include "qsa_device.h"
#include "qsa_internal.h"

namespace qsa {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kNegInf = -__builtin_inff();
constexpr float kLn2 = 0.693147180559945f;

template <int DT>
struct Half;
template <>
struct Half<kBF16> {
    typedef __bf16 T;
    typedef bf16x8 V8;
};
template <>
struct Half<kFP16> {
    typedef _Float16 T;
    typedef f16x8 V8;
};

template <int DT>
__device__ __forceinline__ f32x16 mfma32(i32x4 a, i32x4 b, f32x16 c) {
    typedef typename Half<DT>::V8 V8;
    if constexpr (DT == kBF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(V8, a), __builtin_bit_cast(V8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(V8, a), __builtin_bit_cast(V8, b), c, 0, 0, 0);
}

// 8 values rounded to nearest into 16 bits.  The weights are rounded here to
// the caches' type, and the MFMA then runs at its 16-bit rate: each is off by at most
// half a step of that type relative to itself, as the output is, but for fp16's
// subnormal ones, which are off by up to 2^-25 (kLift keeps that to 2^-38 of the
// largest weight).  The sum of the weights is taken before the rounding.
template <int DT>
__device__ __forceinline__ i32x4 pack8(const f32x16 &p, int at) {
    typename Half<DT>::V8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (typename Half<DT>::T)p[at + j];
    return __builtin_bit_cast(i32x4, v);
}

template <int DT>
__device__ __forceinline__ float to_f32(uint16_t u) {
    return (float)__builtin_bit_cast(typename Half<DT>::T, u);
}

// max(v, v of lane l ^ 32)
__device__ __forceinline__ float xor32_max(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// max(v, v of lane l ^ 16)
__device__ __forceinline__ float xor16_max(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// 16 bytes per lane from global memory to LDS at lds_wave + 16 * lane (lds_wave
// wave-uniform); outstanding on the vector memory counter until wait_copies().
__device__ __forceinline__ void copy16(const void *src, uint32_t lds_wave) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, off\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "v"(src), "s"(lds_wave)
        : "memory");
}

// the same from base + off, base wave-uniform
__device__ __forceinline__ void copy16(const uint8_t *base, uint32_t off, uint32_t lds_wave) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %3\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, %2\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "v"(off), "s"(base), "s"(lds_wave)
        : "memory");
}

// the same with 4 bytes per lane, at lds_wave + 4 * lane
__device__ __forceinline__ void copy4(const void *src, uint32_t lds_wave) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %1, off\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "v"(src), "s"(lds_wave)
        : "memory");
}

__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint32_t lds_offset(const void *p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

// Keys and values lie in LDS as rows of D elements, the 16-byte chunks of a row
// permuted by an XOR with the row's number: the copies write LDS linearly, so
// each lane takes its chunk from the permuted place in global memory.  K rows
// are read by 32 lanes at the same chunk (16 bytes each): the permutation puts
// the rows of every 16 neighbouring lanes into different 16-byte columns of the
// banks.  V is read transposed, 4 rows x 16 elements by 16 lanes: the chunk
// pairs of 4 neighbouring rows are kept apart.
template <int D>
__device__ __forceinline__ int swz_k(int row) {
    return D == 128 ? (row & 15) : ((row >> 1) & 7);
}
template <int D>
__device__ __forceinline__ int swz_v(int row) {
    return D == 128 ? 2 * (row & 7) : 2 * ((row >> 1) & 3);
}

// scores S^T of 32 keys (LDS rows from kbase) against the wave's pairs
template <int DT, int D>
__device__ __forceinline__ f32x16 score_tile(const uint8_t *kbase, const i32x4 (&q)[D / 16], int lane) {
    const int row = lane & 31, h = lane >> 5;
    i32x4 k[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
        k[c] = *reinterpret_cast<const i32x4 *>(kbase + row * 2 * D + (((2 * c + h) ^ swz_k<D>(row)) << 4));
    __builtin_amdgcn_sched_barrier(0);  // all reads on their way before the first product waits for one
    f32x16 s = {};
#pragma unroll
    for (int c = 0; c < D / 16; ++c) s = mfma32<DT>(k[c], q[c], s);
    return s;
}

// four rows' elements as the transposing read gives them: lane i of 16 gets
// element i of the group's 16, rows 0..3
__device__ __forceinline__ s16x4 read_tr(const uint8_t *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)p);
}

// The output element (0..D - 1) of register i of output tile m: the tile's rows 0..15
// are elements of the lower half of the head, rows 16..31 of the upper half, so
// that the two 16-lane groups that read V together read different banks.
template <int D>
__device__ __forceinline__ int out_element(int m, int i, int lane) {
    return D / 2 * (i >> 3) + 16 * m + 8 * ((i >> 2) & 1) + 4 * (lane >> 5) + (i & 3);
}

// V^T operands of 16 keys (rows `row0` on of the LDS rows at vbase), output tiles 0.. D / 32 - 1
template <int D>
__device__ __forceinline__ void read_values(const uint8_t *vbase, int row0, i32x4 (&v)[D / 32], int lane) {
    const int h = lane >> 5, half = (lane >> 4) & 1, i = lane & 15;
#pragma unroll
    for (int m = 0; m < D / 32; ++m) {
        const int chunk = D / 16 * half + 2 * m + ((i & 3) >> 1);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int row = 8 * u + 4 * h + (i >> 2);  // swz_v depends on the low bits only
            const auto x = __builtin_bit_cast(
                i32x2, read_tr(vbase + (row0 + row) * 2 * D + ((chunk ^ swz_v<D>(row)) << 4) + 8 * (i & 1)));
            v[m][2 * u] = x[0];
            v[m][2 * u + 1] = x[1];
        }
    }
}

// O^T += V^T P^T over 32 keys (LDS rows from vbase), p the weights of score_tile's
// layout
template <int DT, int D>
__device__ __forceinline__ void output_tile(const uint8_t *vbase, const f32x16 &p, f32x16 (&o)[D / 32], int lane) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        i32x4 v[D / 32];
        read_values<D>(vbase, 16 * t, v, lane);
        const i32x4 b = pack8<DT>(p, 8 * t);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < D / 32; ++m) o[m] = mfma32<DT>(v[m], b, o[m]);
    }
}

// the key (0..31) that register i of a score tile holds in this lane
__device__ __forceinline__ int score_key(int i, int lane) { return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3); }

// What one MFMA leaves in a lane: 16 values of a 32x32 tile, or 4 of a 16x16 one.
template <bool NARROW>
struct Tile {
    typedef f32x16 V;
};
template <>
struct Tile<true> {
    typedef f32x4 V;
};

template <int DT>
__device__ __forceinline__ f32x4 mfma16(i32x4 a, i32x4 b, f32x4 c) {
    typedef typename Half<DT>::V8 V8;
    if constexpr (DT == kBF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V8, a), __builtin_bit_cast(V8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(V8, a), __builtin_bit_cast(V8, b), c, 0, 0, 0);
}

// The same as score_tile and output_tile with the 16x16x32 MFMA, for up to 16 pairs:
// with g = l >> 4, lane l holds elements 8 g .. + 7 of each 32 as an operand, and of
// the result pair l & 15 and rows 4 g + i.  Score tile u is keys 16 u .. 16 u + 15; the
// inner elements 8 g + j of the second product stand for keys 4 g + j (j < 4) and
// 16 + 4 g + j - 4, the lane's own scores.  Output tile m is elements 16 m .. + 15.
template <int DT, int D>
__device__ __forceinline__ void score_narrow(const uint8_t *kbase, const i32x4 (&q)[D / 32], f32x4 (&z)[2], int lane) {
    const int g = lane >> 4;
    i32x4 k[2][D / 32];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const int row = 16 * u + (lane & 15);
            k[u][c] = *reinterpret_cast<const i32x4 *>(kbase + row * 2 * D + (((4 * c + g) ^ swz_k<D>(row)) << 4));
        }
    __builtin_amdgcn_sched_barrier(0);
    z[0] = z[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int u = 0; u < 2; ++u) z[u] = mfma16<DT>(k[u][c], q[c], z[u]);
}

template <int DT, int D>
__device__ __forceinline__ void output_narrow(const uint8_t *vbase, const f32x4 (&p)[2], f32x4 (&o)[D / 16], int lane) {
    const int g = lane >> 4, i = lane & 15;
    i32x4 v[D / 16];
#pragma unroll
    for (int m = 0; m < D / 16; ++m)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int row = 16 * u + 4 * g + (i >> 2), chunk = 2 * m + ((i & 3) >> 1);
            const auto x = __builtin_bit_cast(
                i32x2, read_tr(vbase + row * 2 * D + ((chunk ^ swz_v<D>(row)) << 4) + 8 * (i & 1)));
            v[m][2 * u] = x[0];
            v[m][2 * u + 1] = x[1];
        }
    typename Half<DT>::V8 w;  // rounded as in pack8
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = (typename Half<DT>::T)p[j >> 2][j & 3];
    const i32x4 b = __builtin_bit_cast(i32x4, w);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 0; m < D / 16; ++m) o[m] = mfma16<DT>(v[m], b, o[m]);
}

// One step of a pair's softmax over U score tiles: the weights
// 2^(c z - ref) in place of the scores z (c = scale log2 e), their sum added to
// `total`.  `ref` (in log2 units, -inf before the first key) is put kLift below the
// running maximum, and follows the maximum only where that has risen by more than
// kLag since, for then every weight is still below 2^(kLift + kLag) and the outputs
// need no rescaling in most steps (with the exact maximum some of a wave's 32 pairs
// rises in nearly every step).  Sums and outputs are relative to ref throughout, so
// it cancels.
//
// c z - ref is one fma, c z itself unrounded, where ref is a rounded c z: they are
// apart by up to half a step of c z, which passes any exponent once scores are large
// (from about 2^30 on a row's only key had weight 0 or infinity).  Past 2^20 the
// products are rounded as ref is, and ref is not lifted (kLift may be less than a step).
//
// fp16 holds weights up to 2^15.9, and from 2^-14 down with fewer and fewer bits.
// With the largest weight between 2^13 and 2^15, keys down to 2^-27 of the largest
// have all theirs.  (Not lifted, 40,000 keys 16 below one whose value is 0 came out 6%
// off.  A lag of 8 with a lift of 7, down to 2^-21, takes 519 us for 2,048 rows at
// 16,384 tokens in fp16, these 525.)
template <int DT>
constexpr float kLag = DT == kFP16 ? 2.0f : 8.0f;
template <int DT>
constexpr float kLift = DT == kFP16 ? 13.0f : 0.0f;
template <int DT, int U, int N, class V>
__device__ __forceinline__ void softmax_step(V (&z)[U], float c, float &ref, float &total, V (&o)[N]) {
    constexpr int kRegs = sizeof(V) / 4;
    float top = z[0][0];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < kRegs; ++i) top = fmaxf(top, z[u][i]);
    if (kRegs == 4) top = xor16_max(top);
    top = xor32_max(top) * c;
    const bool large = fabsf(top) > 0x1p20f;
    if (ballot(large && top != kNegInf)) {
#pragma clang fp contract(off)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < kRegs; ++i) z[u][i] *= c;
        c = 1.0f;
    }
    if (ballot(top - ref > kLift<DT> + kLag<DT>)) {
        const float next = fmaxf(ref, large ? top : top - kLift<DT>);
        const float keep = next == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(ref - next);
        ref = next;
        total *= keep;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] *= keep;
    }
    const float use = ref == kNegInf ? 0.0f : -ref;
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < kRegs; ++i) {
            z[u][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[u][i], c, use));
            sum[i & 1] += z[u][i];
        }
    total += sum[0] + sum[1];
}

// tok / block_size for tok < 2^30 (see AttnArgs)
__device__ __forceinline__ uint32_t block_index(const AttnArgs &a, uint32_t tok) {
    return __umulhi(2 * tok, a.div_mul) >> a.div_shift;
}

// The tokens that a tile of rows works through, in steps of KEYS.  Without a window
// these are the first `keys`.  With one they are the first tokens and those from the
// oldest row's window on: `head` steps of the former, then `gap` steps left out, in
// whole steps, so that a step's tokens are neighbours.  Tokens of a step that no row
// sees may lie in blocks that have been freed: copies take a token that is seen in
// their place.
struct KeySpan {
    int keys;        // behind the last token that a row sees
    int first, old;  // tokens of [first, old) are not seen by any row
    int head, gap;
    int least;       // windows, streaming: the rows' smallest visible count
};

// hi: the rows' largest visible count, lo: the smallest one above 0
template <bool WINDOW, int KEYS>
__device__ __forceinline__ KeySpan key_span(const AttnArgs &a, int hi, int lo) {
    KeySpan s = {hi, 0, 0, 0, 0, 0};
    if constexpr (WINDOW) {
        if (hi <= 0) return s;
        s.first = min(a.sinks, hi);
        s.old = max(lo - a.window, 0);
        s.head = (s.first + KEYS - 1) / KEYS;
        s.gap = max(s.old / KEYS - s.head, 0);
    }
    return s;
}
template <int KEYS>
__device__ __forceinline__ int span_steps(const KeySpan &s) { return (s.keys + KEYS - 1) / KEYS - s.gap; }
// the step of a request's tokens that is step s of the span
template <bool WINDOW>
__device__ __forceinline__ int token_step(const KeySpan &k, int s) { return WINDOW && s >= k.head ? s + k.gap : s; }
// the token that is copied for `tok`
template <bool WINDOW>
__device__ __forceinline__ int copied_token(const KeySpan &k, int tok) {
    if (tok >= k.keys) return k.keys - 1;
    return WINDOW && tok >= k.first && tok < k.old ? k.old : tok;
}
// whether a row with ctx visible tokens sees token tok
template <bool WINDOW>
__device__ __forceinline__ bool sees(const AttnArgs &a, int ctx, int tok) {
    return tok < ctx && (!WINDOW || tok < a.sinks || tok >= ctx - a.window);
}
// whether the tokens [tok, tok + KEYS) are not seen by all rows, whose visible counts are
// from `least` to `most`
template <bool WINDOW, int KEYS>
__device__ __forceinline__ bool partly_seen(const AttnArgs &a, int tok, int least, int most) {
    return tok + KEYS > least || (WINDOW && tok < most - a.window && tok + KEYS > a.sinks);
}

// byte offset of place `in` of pool block `block`, kv head hk
__device__ __forceinline__ int64_t kv_offset(const AttnArgs &a, uint32_t block, uint32_t in, int hk) {
    return (int64_t)(((uint64_t)block * a.kv_block + (uint64_t)in * a.kv_slot + (uint64_t)(uint32_t)hk * a.kv_head) << 4);
}

// The request that takes row tile `slot`, and the tile's first row: request i,
// rows [s_i, s_{i+1}), owns the slots from s_i / T + i on.  These are strictly
// increasing in i and leave room for ceil(len / T) tiles each, so no prefix sum
// over the requests is needed.
struct RowTile {
    int req, row0, rows;
};
__device__ __forceinline__ int request_start(const AttnArgs &a, int i) { return min(max(a.q_starts[i], 0), a.num_rows); }
__device__ __forceinline__ int visible(const AttnArgs &a, int row) { return min(max(a.ctx_lens[row], 0), a.cap); }

// the tile of `slot` among the rows [s0, s1) of request req; rows 0: none
__device__ __forceinline__ RowTile request_tile(const AttnArgs &a, int req, int s0, int s1, int slot) {
    const int j = slot - (s0 / a.tile_rows + req);
    const int64_t row0 = (int64_t)s0 + (int64_t)j * a.tile_rows;
    RowTile t = {req, (int)row0, 0};
    if (j >= 0 && row0 < s1) t.rows = min(a.tile_rows, s1 - t.row0);
    return t;
}

// by one wave: false for a slot without rows
__device__ __forceinline__ bool find_tile(const AttnArgs &a, int slot, RowTile &t) {
    const int T = a.tile_rows, lane = lane_id();
    // 64-way search for the last i in [0, num_reqs) with start(i) / T + i <= slot
    int lo = 0, len = a.num_reqs;
    while (len > 1) {
        const int step = (len + kWave - 1) / kWave;
        const int off = lane * step, i = lo + off;
        const bool le = off < len && request_start(a, i) / T + i <= slot;
        const uint64_t b = ballot(le);
        const int last = b ? 63 - __builtin_clzll(b) : 0;
        lo += last * step;
        len = min(step, len - last * step);
    }
    t = request_tile(a, lo, request_start(a, lo), request_start(a, lo + 1), slot);
    return t.rows > 0;
}

// The requests' first rows and first slots, in LDS.
struct Requests {
    int32_t row[kMaxSlots + 1], slot[kMaxSlots + 1];
};

// the same by one thread
__device__ __forceinline__ RowTile find_tile(const AttnArgs &a, const Requests &q, int slot) {
    int lo = 0, hi = a.num_reqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q.slot[mid] <= slot) lo = mid;
        else hi = mid;
    }
    return request_tile(a, lo, q.row[lo], q.row[lo + 1], slot);
}

// By a whole workgroup: the requests into LDS, and each slot's largest visible
// count, or -1 for a slot without rows.  A thread takes consecutive rows, 8 counts on
// their way at once (one at a time, and with a division per row, this took 10 us for
// 3,163 rows).
// `lows`, with WINDOW: each slot's smallest visible count above 0.
template <int THREADS, bool WINDOW>
__device__ __forceinline__ void slot_counts(const AttnArgs &a, Requests &q, int32_t *counts, int32_t *lows) {
    constexpr int kBatch = 8;
    const int t = threadIdx.x, n = a.num_reqs, T = a.tile_rows;
    for (int i = t; i <= n; i += THREADS) {
        const int s = request_start(a, i);
        q.row[i] = s;
        q.slot[i] = s / T + i;
    }
    for (int i = t; i <= a.slots; i += THREADS) {
        counts[i] = -1;
        if constexpr (WINDOW) lows[i] = 0x7FFFFFFF;
    }
    __syncthreads();
    const int per = (a.num_rows + THREADS - 1) / THREADS, r0 = t * per, r1 = min(r0 + per, a.num_rows);
    int req = 0;
    for (int hi = n; hi - req > 1;) {  // the last request whose first row is at most r0
        const int mid = (req + hi) >> 1;
        if (q.row[mid] <= r0) req = mid;
        else hi = mid;
    }
    int s = q.row[req], e = q.row[req + 1], at = q.slot[req], in = 0;  // row r: slot `at`, its row `in`
    if (r0 > s) {
        at += (r0 - s) / T;
        in = (r0 - s) % T;
    }
    for (int b = r0; b < r1; b += kBatch) {
        int v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) v[j] = visible(a, min(b + j, a.num_rows - 1));
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int r = b + j;
            if (r >= r1) break;
            while (req + 1 < n && r >= e) {
                ++req;
                s = e;
                e = q.row[req + 1];
                at = q.slot[req];
                in = 0;
            }
            if (r < s || r >= e) continue;
            if (at < a.slots) {
                atomicMax(&counts[at], v[j]);
                if (WINDOW && v[j] > 0) atomicMin(&lows[at], v[j]);
            }
            if (++in == T) {
                in = 0;
                ++at;
            }
        }
    }
    __syncthreads();
}

// Exclusive prefix sums over the slots, kPer consecutive ones per thread: before[i]
// is the sum of the slots before i, before[slots] the total.
template <int THREADS>
__device__ __forceinline__ void slot_sums(int32_t *before, int slots, const int32_t (&u)[kMaxSlots / THREADS],
                                          int32_t *wave_sums) {
    constexpr int kPer = kMaxSlots / THREADS;
    const int t = threadIdx.x;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += u[i];
    const int inc = wave_incl_sum(sum);
    if ((t & 63) == 63) wave_sums[t >> 6] = inc;
    __syncthreads();
    int at = inc - sum;
    for (int i = 0; i < (t >> 6); ++i) at += wave_sums[i];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (t * kPer + i <= slots) before[t * kPer + i] = at;
        at += u[i];
    }
    if (t == THREADS - 1 && slots == kMaxSlots) before[slots] = at;
    __syncthreads();
}

__device__ __forceinline__ float wave_sum_f(float v) {
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) v += xor_lane_f(v, m);
    return v;
}

// The kernel's arguments where the launch put them.  A kernel that hands its own
// parameter by reference to a function that is not inlined keeps a copy of it in
// scratch memory and reads every field from there, in its loops too (the
// streaming kernel took 262 us that way over 539 MB of cache).
__device__ __forceinline__ const AttnArgs &launch_args() {
    return *(const AttnArgs *)__builtin_amdgcn_kernarg_segment_ptr();
}

// Outputs that are NaN though the pair's sum is a number.  The kernels multiply a zero
// weight with the values of keys that only other rows of the tile see, of the keys that
// fill up a step (the last one once more) and of those whose weight is below what the
// caches' type holds; where such a value is infinite or NaN, so is the product.  What the
// element is follows from the values that the pair itself sees: NaN, or infinities of
// both signs, make it NaN, infinities of one sign infinite, and otherwise the NaN is
// another row's and the pair is done again over its own keys (selected tokens: there
// are no other rows).  The first place of each of the three kinds is found once per
// wave, for all its pairs.  (Doing every such pair again, one NaN
// that all rows see took 168 ms for 2,048 rows at 16,384 tokens.)
//
// Places are tokens, or with SPARSE the entries of `idx` times `ratio`; a lane has the
// elements lane D / 64 on.  All this is cold.

// the lane's place: false if it has no token, or one behind a table entry outside the pool
template <bool SPARSE>
__device__ __forceinline__ bool place_offset(const AttnArgs &a, int req, int hk, const int32_t *idx, int limit, int place,
                                             int64_t &off, bool &bad) {
    int64_t key = place;
    if constexpr (SPARSE) {
        const int column = idx[place / a.ratio];
        key = (int64_t)column * a.ratio + place % a.ratio;
        if (column < 0 || key >= limit) return false;
    }
    const uint32_t at = block_index(a, (uint32_t)key);
    const int e = a.block_table[(int64_t)req * a.max_blocks + at];
    bad = e < 0 || e >= a.num_blocks;
    if (!bad) off = kv_offset(a, e, (uint32_t)key - at * (uint32_t)a.block_size, hk);
    return true;
}

// The lane's elements of the values at off of lanes j .. j + 7; any lane's off is in the
// pool (0 where it has no token).
template <int D>
__device__ __forceinline__ void value_rows(const AttnArgs &a, int64_t off, int j, uint16_t (&x)[8][D / 64]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t at = ((int64_t)readlane((int)(off >> 32), j + i) << 32) | (uint32_t)readlane((int)off, j + i);
        const uint16_t *v = reinterpret_cast<const uint16_t *>(a.vcache + at) + lane_id() * (D / 64);
        if constexpr (D == 128) *reinterpret_cast<uint32_t *>(x[i]) = *reinterpret_cast<const uint32_t *>(v);
        else x[i][0] = v[0];
    }
}

// first places of values that are NaN, infinite and minus infinite
template <int D>
struct FirstPlaces {
    int nan[D / 64], inf[D / 64], minus[D / 64];
};

// adds the places [k0, k1)
template <int DT, int D, bool SPARSE>
__device__ __forceinline__ void find_places(const AttnArgs &a, int req, int hk, const int32_t *idx, int limit, int k0,
                                            int k1, FirstPlaces<D> &f) {
    for (int base = k0; base < k1; base += kWave) {
        int64_t off = 0;
        bool bad = false;
        const bool seen = base + lane_id() < k1 && place_offset<SPARSE>(a, req, hk, idx, limit, base + lane_id(), off, bad);
        const uint64_t mine = ballot(seen && !bad);
        for (int j = 0; j < kWave; j += 8) {
            uint16_t x[8][D / 64];
            value_rows<D>(a, off, j, x);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (!(mine >> (j + u) & 1)) continue;
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const float v = to_f32<DT>(x[u][i]);
                    if (v != v) f.nan[i] = min(f.nan[i], base + j + u);
                    if (v == -kNegInf) f.inf[i] = min(f.inf[i], base + j + u);
                    if (v == kNegInf) f.minus[i] = min(f.minus[i], base + j + u);
                }
            }
        }
    }
}

template <int D>
__device__ __forceinline__ FirstPlaces<D> no_places() {
    FirstPlaces<D> f;
    for (int i = 0; i < D / 64; ++i) f.nan[i] = f.inf[i] = f.minus[i] = 0x7FFFFFFF;
    return f;
}

template <int DT, int D, bool SPARSE>
__device__ __forceinline__ FirstPlaces<D> first_places(const AttnArgs &a, int req, int hk, const int32_t *idx, int limit,
                                                       int k0, int k1) {
    FirstPlaces<D> f = no_places<D>();
    find_places<DT, D, SPARSE>(a, req, hk, idx, limit, k0, k1, f);
    return f;
}

// Adds a pair's own keys [k0, k1) to its softmax state, by one wave with plain loads and
// 32-bit weights: no other key's value is touched.
template <int DT, int D>
__device__ __forceinline__ void own_range(const AttnArgs &a, int req, const uint16_t *q, int hk, int k0, int k1, float &m,
                                          float &l, float (&o)[D / 64]) {
    for (int base = k0; base < k1; base += kWave) {
        int64_t off = 0;
        bool bad = false;
        const bool seen = base + lane_id() < k1 && place_offset<false>(a, req, hk, nullptr, 0, base + lane_id(), off, bad);
        float s = kNegInf;
        if (seen) {
            const i32x4 *k = reinterpret_cast<const i32x4 *>(a.kcache + off);
            float dot = 0.0f;
            for (int c = 0; c < D / 8; ++c) {
                const i32x4 x = k[c];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dot += to_f32<DT>(q[8 * c + e]) * to_f32<DT>((uint16_t)((uint32_t)x[e >> 1] >> (16 * (e & 1))));
            }
            s = bad ? __builtin_nanf("") : dot * a.scale_log2;
        }
        const uint64_t mine = ballot(seen);
        const float top = fmaxf(m, wave_max_f(s));
        const float ref = top == kNegInf ? 0.0f : top;
        const float p = __builtin_amdgcn_exp2f(s - ref), keep = __builtin_amdgcn_exp2f(m - ref);
        l = l * keep + wave_sum_f(p);
        for (int i = 0; i < D / 64; ++i) o[i] *= keep;
        m = top;
        for (int j = 0; j < kWave; j += 8) {
            uint16_t x[8][D / 64];
            value_rows<D>(a, off, j, x);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (!(mine >> (j + u) & 1)) continue;
                const float pj = readlane_f(p, j + u);
#pragma unroll
                for (int i = 0; i < D / 64; ++i) o[i] += pj * to_f32<DT>(x[u][i]);
            }
        }
    }
}

// A pair's place in the outputs, or with `state` in a cut tile's part.
struct PairPlace {
    const uint16_t *q;
    void *out;
    float *lse;                   // or null
    float *state, *top, *total;   // all null, or the state's outputs, reference and sum
};

// The places that a pair sees: [k0, k1), and with a window [k2, k3) before them.
struct OwnPlaces {
    int k0, k1, k2, k3;
};

// What a row with ctx visible tokens sees of steps [s0, s1) of KEYS keys of its tile's span.
template <int KEYS>
__device__ __forceinline__ OwnPlaces window_places(const AttnArgs &a, const KeySpan &span, int ctx, int s0, int s1) {
    const int first = min(a.sinks, ctx), old = max(ctx - a.window, first);
    // the window's steps are behind the gap, the first tokens' before it
    const int gap = span.gap * KEYS;
    return {max(s0 * KEYS + gap, old), min(s1 * KEYS + gap, ctx), s0 * KEYS, min(s1 * KEYS, first)};
}

// first places over all that a pair sees
template <int DT, int D>
__device__ __forceinline__ FirstPlaces<D> own_first_places(const AttnArgs &a, int req, int hk, const OwnPlaces &k) {
    FirstPlaces<D> f = no_places<D>();
#pragma unroll 1
    for (int i = 0; i < 2; ++i)
        find_places<DT, D, false>(a, req, hk, nullptr, 0, i ? k.k0 : k.k2, i ? k.k1 : k.k3, f);
    return f;
}

// Mends what the wave has written of one pair over its places `k`, of which k1 is the
// end, or does the pair anew (`anew`).
template <int DT, int D, bool SPARSE>
__device__ __forceinline__ void mend_pair(const AttnArgs &a, int req, int hk, const OwnPlaces &k, const FirstPlaces<D> &f,
                                          bool anew, const PairPlace &p) {
    const int k1 = k.k1;
    typedef typename Half<DT>::T T;
    const int at = lane_id() * (D / 64);
    T *out = static_cast<T *>(p.out) + at;
    float o[D / 64], inv = 1.0f;
    bool others = anew, write = false;
    const auto settle = [&]() {  // NaN elements by the values that the pair sees
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const bool inf = f.inf[i] < k1, minus = f.minus[i] < k1;
            if (o[i] == o[i] || f.nan[i] < k1 || (inf && minus)) continue;
            if (inf || minus) {
                o[i] = inf ? -kNegInf : kNegInf;
                write = true;
            } else {
                others = true;
            }
        }
    };
    if (!anew) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) o[i] = p.state ? p.state[at + i] : (float)out[i];
        settle();
    }
    if constexpr (!SPARSE) {
        if (ballot(others)) {
            float top = kNegInf, total = 0.0f;
            for (int i = 0; i < D / 64; ++i) o[i] = 0.0f;
#pragma unroll 1
            for (int i = 0; i < 2; ++i)
                own_range<DT, D>(a, req, p.q, hk, i ? k.k0 : k.k2, i ? k1 : k.k3, top, total, o);
            if (!anew) settle();
            write = true;
            if (lane_id() == 0 && p.state) {
                *p.top = top;
                *p.total = total;
            }
            if (lane_id() == 0 && !p.state && p.lse) *p.lse = (top + __builtin_amdgcn_logf(total)) * kLn2;
            if (!p.state) inv = total == 0.0f ? 0.0f : 1.0f / total;
        }
    }
    if (!write) return;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        if (p.state) p.state[at + i] = o[i];
        else out[i] = (T)(o[i] * inv);
    }
}

// Joins the parts of a cut tile for one pair, D / 4 threads to a pair with 4 output
// elements each: the parts' states (outputs [PAIRS][D], references, sums) are read 8
// parts at a time, all of a batch on their way at once.  Part i is at p + i stride.
template <int DT, int D, int PAIRS>
__device__ __forceinline__ void join_parts(const float *parts, int64_t stride, int used, int m, int d0,
                                           typename Half<DT>::T *out, float *lse) {
    constexpr int kBatch = 8;
    typedef typename Half<DT>::T T;
    typedef T V4 __attribute__((ext_vector_type(4)));
    float top = kNegInf, total = 0.0f;
    f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < used; i += kBatch) {
        float ref[kBatch], l[kBatch];
        f32x4 x[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const float *p = parts + min(i + j, used - 1) * stride;
            ref[j] = p[PAIRS * D + m];
            l[j] = p[PAIRS * (D + 1) + m];
            x[j] = *reinterpret_cast<const f32x4 *>(p + m * D + d0);
        }
        float next = top;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) next = fmaxf(next, ref[j]);
        const float use = next == kNegInf ? 0.0f : next;
        const float keep = __builtin_amdgcn_exp2f(top - use);
        top = next;
        total *= keep;
        v *= keep;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const float f = i + j < used ? __builtin_amdgcn_exp2f(ref[j] - use) : 0.0f;
            if (i + j < used) {
                total += l[j] * f;
                v += x[j] * f;
            }
        }
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    V4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = (T)(v[j] * inv);
    *reinterpret_cast<V4 *>(out + d0) = r;
    if (lse && d0 == 0) *lse = (top + __builtin_amdgcn_logf(total)) * kLn2;
}
constexpr int kJoinThreads = 256;

}  // namespace qsa
