// Attention of few stacked rows over long key ranges: decode and verify rows
// over the paged cache (dense), and single rows over selected tokens (SPARSE).
//
//   o = sum_c softmax_c(scale q . k_c) v_c,  lse = log sum_c exp(scale q . k_c)
//
// One workgroup takes up to 32 (row, head) pairs that share a kv head and a
// range of keys; its four waves take the range's 32-key steps in turn, each
// with a softmax state of its own, joined in LDS at the end.  Where the row
// tiles do not fill the chip, the keys are split over several workgroups, which
// leave their states (32-bit maximum, sum and unnormalised output) in the
// workspace for a joining kernel.
//
// What bounds it is the cache's bytes: 32 keys and values of one head are 16 KB
// at D = 128, against 16 MFMAs.  Each wave owns two 16 KB buffers and copies the
// next step straight to LDS while it works on the current one, so the loads
// need no registers and no barriers; the table entries (and selected columns)
// behind the copies are loaded one step (two steps) further ahead.

#include "attn_device.h"

namespace qsa {
namespace {

constexpr int kStreamThreads = 64 * kStreamWaves;

struct TileWork {
    int req, row0, rows;  // dense: a request's tile; sparse: one row
    int hk, head0, heads;
};

// The pair m of a tile: row m / sub_heads, head m % sub_heads.
struct Pair {
    int row, head;
    bool live;
};
__device__ __forceinline__ Pair pair_of(const AttnArgs &a, const TileWork &w, int m) {
    Pair p;
    const int r = m / a.sub_heads;
    p.row = w.row0 + r;
    p.head = w.head0 + m - r * a.sub_heads;
    p.live = r < w.rows && p.head < w.head0 + w.heads;
    return p;
}

template <bool SPARSE>
__device__ __forceinline__ bool tile_work(const AttnArgs &a, int slot, int hs, TileWork &w) {
    w.hk = hs / a.num_subs;
    const int sub = hs - w.hk * a.num_subs;
    w.head0 = w.hk * a.group + sub * a.sub_heads;
    w.heads = min(a.sub_heads, a.group - sub * a.sub_heads);
    if (SPARSE) {
        w.row0 = slot;
        w.rows = 1;
        const int r = a.row_to_req[slot];
        w.req = r >= 0 && r < a.num_reqs ? r : -1;
        return true;
    }
    RowTile t;
    if (!find_tile(a, slot, t)) return false;
    w.req = t.req;
    w.row0 = t.row0;
    w.rows = t.rows;
    return true;
}

// keys the tile works through: the largest visible count of its rows, or the
// selected tokens
template <bool SPARSE>
__device__ __forceinline__ int visible(const AttnArgs &a, int row) {
    if (SPARSE) return a.k * a.ratio;
    return min(max(a.ctx_lens[row], 0), a.cap);
}

template <bool SPARSE>
__device__ __forceinline__ int tile_keys(const AttnArgs &a, const TileWork &w) {
    if (SPARSE) return a.k * a.ratio;
    int most = 0;
    for (int r = 0; r < w.rows; ++r) most = max(most, visible<SPARSE>(a, w.row0 + r));
    return most;
}

// 32-key steps of a split: one for each wave at least
__device__ __forceinline__ int split_steps(int steps, int splits) {
    return max((steps + splits - 1) / splits, kStreamWaves);
}

template <int DT, int D, bool SPARSE>
__global__ __launch_bounds__(kStreamThreads, 1) void attn_stream_kernel(AttnArgs a) {
    constexpr int kTileBytes = kStreamKeys * D * 2;          // keys (or values) of one step
    constexpr int kWaveBytes = 4 * kTileBytes;               // two buffers of keys and values
    constexpr int kCopies = kTileBytes / (16 * kWave);       // copy instructions for each of the two
    constexpr int kLanesPerKey = D / 8, kKeysPerCopy = kWave / kLanesPerKey;
    constexpr int kPad = D + 4;                              // floats between rows of the waves' outputs
    __shared__ __align__(16) uint8_t ring[kStreamWaves * kWaveBytes];
    __shared__ float top_of[kStreamWaves][kAttnTile], sum_of[kStreamWaves][kAttnTile];

    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int slot = blockIdx.x, hs = blockIdx.y, split = blockIdx.z;
    TileWork w;
    if (!tile_work<SPARSE>(a, slot, hs, w)) return;
    const Pair pair = pair_of(a, w, lane & 31);
    const int keys = __builtin_amdgcn_readfirstlane(tile_keys<SPARSE>(a, w));
    const int steps = (keys + kStreamKeys - 1) / kStreamKeys;
    const int per = a.splits > 1 ? split_steps(steps, a.splits) : steps;
    const int t0 = min(split * per, steps), t1 = min(t0 + per, steps);
    if (a.splits > 1 && t0 >= t1) return;

    const int ctx = SPARSE ? 0 : (pair.live ? visible<SPARSE>(a, pair.row) : 0);
    int least = 0, limit = 0;
    if (SPARSE) {
        limit = a.ctx_lens ? min(max(a.ctx_lens[w.row0], 0), a.cap) : a.cap;
    } else {
        least = keys;  // the smallest visible count: steps below it need no mask
        for (int r = 0; r < w.rows; ++r) least = min(least, visible<SPARSE>(a, w.row0 + r));
    }

    i32x4 q[D / 16];
    const uint16_t *qrow = static_cast<const uint16_t *>(a.q) + pair.row * a.q_row + pair.head * a.q_head;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        q[c] = i32x4{0, 0, 0, 0};
        if (pair.live) q[c] = *reinterpret_cast<const i32x4 *>(qrow + 16 * c + 8 * (lane >> 5));
    }

    uint8_t *mine = ring + wave * kWaveBytes;
    const uint32_t mine_lds = lds_offset(mine);
    const int32_t *table = a.block_table + (int64_t)max(w.req, 0) * a.max_blocks;
    const int32_t *idx = SPARSE ? a.idx + (int64_t)w.row0 * a.k : nullptr;

    // a step's tokens, one per lane of each half wave
    struct Token {
        int32_t entry, in;
        bool seen;
    };
    const auto load_column = [&](int s) -> int32_t {
        if constexpr (!SPARSE) return 0;
        const int pos = s * kStreamKeys + (lane & 31);
        return s < t1 && pos < keys ? idx[pos / a.ratio] : -1;
    };
    const auto load_entry = [&](int s, int32_t column) -> Token {
        Token k = {0, 0, false};
        if (s >= t1) return k;
        const int pos = s * kStreamKeys + (lane & 31);
        uint32_t tok;
        if constexpr (SPARSE) {
            const int64_t wide = (int64_t)column * a.ratio + pos % a.ratio;
            k.seen = column >= 0 && wide < limit;
            tok = k.seen ? (uint32_t)wide : 0u;
        } else {
            // behind the last visible key the copies take that key again
            k.seen = true;
            tok = (uint32_t)min(pos, keys - 1);
        }
        const uint32_t e = tok / (uint32_t)a.block_size;
        k.in = (int32_t)(tok - e * (uint32_t)a.block_size);
        if (k.seen && w.req >= 0) k.entry = table[e];
        if (w.req < 0) k.entry = -1;
        return k;
    };
    // starts the copies of a step; returns which keys take part and which are
    // behind table entries outside the pool
    struct Masks {
        uint32_t seen, bad;
    };
    const auto start_copies = [&](const Token &k, int buf) -> Masks {
        Masks mk;
        mk.seen = (uint32_t)ballot(k.seen);
        const bool bad = k.entry < 0 || k.entry >= a.num_blocks;
        mk.bad = (uint32_t)ballot(bad && k.seen);
        if (SPARSE && mk.seen == 0) return mk;
        int64_t off = (bad ? 0 : (int64_t)k.entry * a.kv_block) + (int64_t)k.in * a.kv_slot + (int64_t)w.hk * a.kv_head;
        int lo = (int)off, hi = (int)(off >> 32);
        if (SPARSE && mk.seen != 0xFFFFFFFFu) {  // places without a token take the first seen token's key
            const int first = __builtin_ctz(mk.seen);
            const int flo = readlane(lo, first), fhi = readlane(hi, first);
            lo = k.seen ? lo : flo;
            hi = k.seen ? hi : fhi;
        }
        const uint32_t lds = mine_lds + buf * 2 * kTileBytes;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const int row = i * kKeysPerCopy + lane / kLanesPerKey, chunk = lane % kLanesPerKey;
            const int64_t at = ((int64_t)shfl_i(hi, row) << 32) | (uint32_t)shfl_i(lo, row);
            copy16(a.kcache + 2 * (at + 8 * (chunk ^ swz_k<D>(row))), lds + i * 16 * kWave);
            copy16(a.vcache + 2 * (at + 8 * (chunk ^ swz_v<D>(row))), lds + kTileBytes + i * 16 * kWave);
        }
        return mk;
    };

    f32x16 o[D / 32] = {};
    float m = kNegInf, l = 0.0f;  // l: this lane's half of the sum
    int s = t0 + wave, buf = 0;
    Masks now = {0, 0};
    Token next;
    int32_t column;
    {
        const Token first = load_entry(s, load_column(s));
        const int32_t c1 = load_column(s + kStreamWaves);
        if (s < t1) now = start_copies(first, 0);
        next = load_entry(s + kStreamWaves, c1);
        column = load_column(s + 2 * kStreamWaves);
    }
    for (; s < t1; s += kStreamWaves) {
        wait_copies();
        const Masks cur = now;
        if (s + kStreamWaves < t1) {
            now = start_copies(next, buf ^ 1);
            next = load_entry(s + 2 * kStreamWaves, column);
            column = load_column(s + 3 * kStreamWaves);
        }
        const uint8_t *kb = mine + buf * 2 * kTileBytes;
        buf ^= 1;
        if (SPARSE && cur.seen == 0) continue;
        f32x16 z = score_tile<DT, D>(kb, q, lane);
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] *= a.scale_log2;
        if (cur.bad) {
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = (cur.bad >> score_key(i, lane)) & 1 ? __builtin_nanf("") : z[i];
        }
        if (SPARSE) {
            if (cur.seen != 0xFFFFFFFFu) {
#pragma unroll
                for (int i = 0; i < 16; ++i) z[i] = (cur.seen >> score_key(i, lane)) & 1 ? z[i] : kNegInf;
            }
        } else if ((s + 1) * kStreamKeys > least) {
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = s * kStreamKeys + score_key(i, lane) < ctx ? z[i] : kNegInf;
        }
        float top = z[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, z[i]);
        top = fmaxf(m, xor32_max(top));
        const float ref = top == kNegInf ? 0.0f : top;
        const float keep = __builtin_amdgcn_exp2f(m - ref);
        m = top;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            z[i] = __builtin_amdgcn_exp2f(z[i] - ref);
            sum += z[i];
        }
        l = l * keep + sum;
        if (ballot(keep != 1.0f)) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) o[c] *= keep;
        }
        output_tile<DT, D>(kb + kTileBytes, z, o, lane);
    }
    l = xor32_sum(l);

    // join the waves' states: each leaves its output in its own part of the ring
    float *left = reinterpret_cast<float *>(mine);
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const f32x4 v = {o[c][4 * g], o[c][4 * g + 1], o[c][4 * g + 2], o[c][4 * g + 3]};
            *reinterpret_cast<f32x4 *>(left + (lane & 31) * kPad + 32 * c + 8 * g + 4 * (lane >> 5)) = v;
        }
    if (lane < kAttnTile) {
        top_of[wave][lane] = m;
        sum_of[wave][lane] = l;
    }
    __syncthreads();
    constexpr int kPer = D / 8;  // outputs per thread: 8 threads to a pair
    const int pm = t >> 3, d0 = (t & 7) * kPer;
    float top = kNegInf, total = 0.0f, r[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) r[i] = 0.0f;
#pragma unroll
    for (int i = 0; i < kStreamWaves; ++i) top = fmaxf(top, top_of[i][pm]);
    const float ref = top == kNegInf ? 0.0f : top;
#pragma unroll
    for (int i = 0; i < kStreamWaves; ++i) {
        const float f = __builtin_amdgcn_exp2f(top_of[i][pm] - ref);
        total += sum_of[i][pm] * f;
        const float *src = reinterpret_cast<const float *>(ring + i * kWaveBytes) + pm * kPad + d0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) r[j] += src[j] * f;
    }
    const Pair pp = pair_of(a, w, pm);
    if (!SPARSE && least < keys) {
        // A NaN can come from a value that only other rows of the tile see (zero
        // weight times a value that is not finite): then every pair is done
        // again over its own keys.
        bool nan = false;
#pragma unroll
        for (int i = 0; i < kPer; ++i) nan |= r[i] != r[i];
        if (__syncthreads_or(nan && pp.live)) {
            float *again = reinterpret_cast<float *>(ring);
            for (int p = wave; p < kAttnTile; p += kStreamWaves) {
                const Pair x = pair_of(a, w, p);
                if (!x.live) continue;
                float pm2, pl2, po[D / 64];
                own_range<DT, D>(launch_args(), w.req, static_cast<const uint16_t *>(a.q) + x.row * a.q_row + x.head * a.q_head,
                                 w.hk, t0 * kStreamKeys, min(t1 * kStreamKeys, visible<SPARSE>(a, x.row)), pm2, pl2,
                                 po);
                for (int i = 0; i < D / 64; ++i) again[p * kPad + lane * (D / 64) + i] = po[i];
                if (lane == 0) {
                    top_of[0][p] = pm2;
                    sum_of[0][p] = pl2;
                }
            }
            __syncthreads();
            top = top_of[0][pm];
            total = sum_of[0][pm];
#pragma unroll
            for (int i = 0; i < kPer; ++i) r[i] = again[pm * kPad + d0 + i];
        }
    }
    if (!pp.live) return;
    if (a.splits > 1) {
        float *part = a.part + ((int64_t)(slot * gridDim.y + hs) * a.splits + split) * (kAttnTile * (D + 2));
#pragma unroll
        for (int i = 0; i < kPer; i += 4)
            *reinterpret_cast<f32x4 *>(part + pm * D + d0 + i) = f32x4{r[i], r[i + 1], r[i + 2], r[i + 3]};
        if ((t & 7) == 0) {
            part[kAttnTile * D + pm] = top;
            part[kAttnTile * (D + 1) + pm] = total;
        }
        return;
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    typedef typename Half<DT>::T T;
    T *out = static_cast<T *>(a.out) + pp.row * a.o_row + pp.head * a.o_head + d0;
#pragma unroll
    for (int i = 0; i < kPer; i += 8) {
        typename Half<DT>::V8 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (T)(r[i + j] * inv);
        *reinterpret_cast<i32x4 *>(out + i) = __builtin_bit_cast(i32x4, v);
    }
    if (a.lse && (t & 7) == 0)
        a.lse[(int64_t)pp.row * (a.num_kv_heads * a.group) + pp.head] = (top + __builtin_amdgcn_logf(total)) * kLn2;
}

// Joins the splits' states, one wave to a pair: lane i reads split i's maximum
// and sum, and the outputs are read 8 splits at a time, D / 64 elements per lane.
constexpr int kJoinPairs = 4;

template <int DT, int D, bool SPARSE>
__global__ __launch_bounds__(64 * kJoinPairs) void attn_join_kernel(AttnArgs a) {
    constexpr int kPer = D / 64, kBatch = 8;
    typedef float Vec __attribute__((ext_vector_type(kPer)));
    TileWork w;
    if (!tile_work<SPARSE>(a, blockIdx.x, blockIdx.y, w)) return;
    const int lane = threadIdx.x & 63;
    const int pm = __builtin_amdgcn_readfirstlane(blockIdx.z * kJoinPairs + (threadIdx.x >> 6));
    const Pair pp = pair_of(a, w, pm);
    if (!pp.live) return;
    const int keys = __builtin_amdgcn_readfirstlane(tile_keys<SPARSE>(a, w));
    constexpr int kPart = kAttnTile * (D + 2);
    const float *part = a.part + (int64_t)(blockIdx.x * gridDim.y + blockIdx.y) * a.splits * kPart;
    const int steps = (keys + kStreamKeys - 1) / kStreamKeys, per = split_steps(steps, a.splits);
    const int used = (steps + per - 1) / per;
    float m = kNegInf, l = 0.0f;
    if (lane < used) {
        m = part[lane * kPart + kAttnTile * D + pm];
        l = part[lane * kPart + kAttnTile * (D + 1) + pm];
    }
    const float top = wave_max_f(m), ref = top == kNegInf ? 0.0f : top;
    const float f = __builtin_amdgcn_exp2f(m - ref);
    const float total = wave_sum_f(l * f);
    Vec r = {};
    const float *src = part + pm * D + kPer * lane;
    for (int i = 0; i < used; i += kBatch) {
        Vec v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) v[j] = *reinterpret_cast<const Vec *>(src + min(i + j, used - 1) * kPart);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (i + j < used) r += v[j] * readlane_f(f, i + j);
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    typedef typename Half<DT>::T T;
    T *out = static_cast<T *>(a.out) + pp.row * a.o_row + pp.head * a.o_head + kPer * lane;
#pragma unroll
    for (int j = 0; j < kPer; ++j) out[j] = (T)(r[j] * inv);
    if (a.lse && lane == 0)
        a.lse[(int64_t)pp.row * (a.num_kv_heads * a.group) + pp.head] = (top + __builtin_amdgcn_logf(total)) * kLn2;
}

template <int DT, int D, bool SPARSE>
hipError_t run_stream(const AttnArgs &a, hipStream_t s) {
    const unsigned heads = (unsigned)(a.num_kv_heads * a.num_subs);
    hipLaunchKernelGGL((attn_stream_kernel<DT, D, SPARSE>), dim3((unsigned)a.slots, heads, (unsigned)a.splits),
                       dim3(kStreamThreads), 0, s, a);
    if (a.splits > 1)
        hipLaunchKernelGGL((attn_join_kernel<DT, D, SPARSE>),
                           dim3((unsigned)a.slots, heads, kAttnTile / kJoinPairs), dim3(64 * kJoinPairs), 0, s, a);
    return hipGetLastError();
}

template <int DT>
hipError_t run_dim(const AttnArgs &a, bool sparse, hipStream_t s) {
    if (a.head_dim == 128) return sparse ? run_stream<DT, 128, true>(a, s) : run_stream<DT, 128, false>(a, s);
    return sparse ? run_stream<DT, 64, true>(a, s) : run_stream<DT, 64, false>(a, s);
}

}  // namespace

hipError_t launch_attn_stream(const AttnArgs &a, bool sparse, hipStream_t s) {
    return a.dtype == kBF16 ? run_dim<kBF16>(a, sparse, s) : run_dim<kFP16>(a, sparse, s);
}

}  // namespace qsa
