// Attention of few stacked rows over long key ranges: decode and verify rows
// over the paged cache (dense), and single rows over selected tokens (SPARSE).
//
//   o = sum_c softmax_c(scale q . k_c) v_c,  lse = log sum_c exp(scale q . k_c)
//
// A tile is up to 32 (row, head) pairs that share a kv head.  A workgroup works
// on one tile's keys (or a range of them) with 8 waves that take 32-key steps in
// turn, each with a softmax state of its own, joined in LDS at the end.
//
// What bounds it is the bytes of keys and values: a step is 16 KB at D = 128
// against 16 MFMAs.  Each wave owns a key and a value buffer in LDS, filled
// straight from global memory; the next step's keys are fetched as soon as the
// scores are taken and the next values as soon as the output is, so that about
// 128 KB are on their way to a CU at any time, without registers or barriers.
// Table entries and selected columns reach the wave the same way, one and two
// steps ahead.  Every load of the loop is such a copy, so the waits can count
// them: copies complete in order, and the newest are always one buffer's.
//
// Cut launches (few tiles, a workspace): the tiles' key ranges are laid end
// to end and cut into kStreamGroups equal parts, one per workgroup and CU, so
// requests of mixed lengths keep the whole chip busy to the end.  A tile that is
// cut leaves its parts' states (32-bit maximum, sum, unnormalised output) in the
// workspace and a second kernel joins them; part (workgroup, tile) has place
// workgroup + tile, as both only grow along the line (tiles are numbered without the
// slots that have no rows).  With many tiles each gets a workgroup.
//
// Measured (kernel traces): a verify step of 9 requests with 4 rows, 16,000 to 65,600
// tokens, 539 MB of cache at D = 128, 32 over 4 heads, bf16: 109 us and 5 for the
// join, 4.8 TB/s of both, where a kernel that only reads as many bytes in order takes
// 87 (6.2 TB/s); 262 + 26 us with one wave per 32 keys' split and arguments in scratch,
// 198 + 10 without the scratch.  One row over 4,000 tokens: 10 + 4 us, latency: about
// six dependent loads, of which the launch, the join and the table make half.  Selected
// tokens of 36 rows (8,192 each, 605 MB): 106 + 5 us, 5.5 TB/s.  Of 1,000 rows (2,048
// each): 267 us for 4.2 GB through the L2s (15.7 TB/s; 78% of the requests hit), 299
// with 32-pair tiles of which these heads fill 8 (NARROW below).  A plain kernel that
// loads the same rows and multiplies nothing takes 230 us (18.2 TB/s): what bounds it
// is the gather.
#include "attn_device.h"

namespace qsa {
namespace {

constexpr int kStreamThreads = kWave * kStreamWaves;

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

// the query heads of head part `hs`
__device__ __forceinline__ void part_heads(const AttnArgs &a, int hs, TileWork &w) {
    w.hk = hs / a.num_subs;
    const int sub = hs - w.hk * a.num_subs;
    w.head0 = w.hk * a.group + sub * a.sub_heads;
    w.heads = min(a.sub_heads, a.group - sub * a.sub_heads);
}

// the tile of row tile `slot` and head part `hs`; false for a slot without rows
template <bool SPARSE>
__device__ __forceinline__ bool tile_work(const AttnArgs &a, int slot, int hs, TileWork &w) {
    part_heads(a, hs, w);
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

// keys the tile works through: up to the largest visible count of its rows, or the
// selected tokens
template <bool SPARSE>
__device__ __forceinline__ KeySpan tile_keys(const AttnArgs &a, int row0, int rows) {
    if (SPARSE) return {a.k * a.ratio, 0, 0, 0, 0, 0};
    int most = 0;
    for (int r = 0; r < rows; ++r) most = max(most, visible(a, row0 + r));
    return key_span<false, kStreamKeys>(a, __builtin_amdgcn_readfirstlane(most), 0);
}
// by a wave, the rows' counts read at once (one after the other they took 1 to 2 us)
__device__ __forceinline__ KeySpan window_keys(const AttnArgs &a, int row0, int rows) {
    const int r = lane_id(), v = r < rows ? visible(a, row0 + r) : 0;
    const int most = (int)wave_total_umax((uint32_t)v), low = 0x7FFFFFFF - (int)wave_total_umax(v > 0 ? 0x7FFFFFFFu - v : 0u);
    KeySpan s = key_span<true, kStreamKeys>(a, most, low);
    s.least = 0x7FFFFFFF - (int)wave_total_umax(r < rows ? 0x7FFFFFFFu - v : 0u);
    return s;
}

// 8 (D = 128) or 4 copies fill a buffer; wait until at most one buffer's are
// outstanding
template <int N>
__device__ __forceinline__ void wait_all_but() {
    static_assert(N == 8 || N == 4, "copies of a buffer");
    if constexpr (N == 8) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
}

// this wave's reads of LDS are done: what they read may be overwritten by copies
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// where a cut tile's state lies in the workspace
template <int D>
__device__ __forceinline__ float *part_of(const AttnArgs &a, int group, int tile) {
    return a.part + (int64_t)(group + tile) * (kAttnTile * (D + 2));
}

// NARROW (selected tokens of up to 16 heads): the 16x16x32 MFMA on 16 pairs instead of
// the 32x32x16 one on 32, with half the products and half the weights per key.
// WINDOW: the newest tokens and the first ones only (see KeySpan).
// WAVES: of the workgroup.
template <int DT, int D, bool SPARSE, bool NARROW, bool WINDOW, int WAVES = kStreamWaves>
struct Stream {
    static constexpr int kThreads = kWave * WAVES;
    static_assert(SPARSE || !NARROW, "dense tiles fill 32 pairs where they can");
    static_assert(!SPARSE || !WINDOW, "a selection is its own window");
    static constexpr int kTileBytes = kStreamKeys * D * 2;  // one buffer of keys or values
    static constexpr int kCopies = kTileBytes / (16 * kWave);
    static constexpr int kLanesPerKey = D / 8, kKeysPerCopy = kWave / kLanesPerKey;

    struct Shared {
        __align__(16) uint8_t ring[WAVES][2 * kTileBytes];
        int32_t entry[WAVES][2][kWave];
        int32_t column[WAVES][2][kWave];
        float top_of[WAVES][kAttnTile], sum_of[WAVES][kAttnTile];
    };

    // where f32 output chunk c (4 elements) of pair p lies in a wave's buffers,
    // which hold exactly the 32 x D outputs: chunks permuted so that neither the
    // lanes of a pair nor those of a chunk meet in one bank
    static __device__ __forceinline__ int left_at(int p, int c) { return p * D + 4 * (c ^ (p & (D / 4 - 1))); }

    // steps [t0, t1) of tile w's keys; dest: the workspace place of the state, or null to
    // write the outputs
    static __device__ __forceinline__ void run(const AttnArgs &a, Shared &sh, const TileWork &w, KeySpan span, int t0,
                                               int t1, float *dest) {
        const int keys = span.keys;
        int t = threadIdx.x;
        asm volatile("" : "+v"(t));  // addresses are made anew for each range, not kept live across them
        const int lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
        const Pair pair = pair_of(a, w, NARROW ? lane & 15 : lane & 31);
        const int ctx = SPARSE ? 0 : (pair.live ? visible(a, pair.row) : 0);
        int least = 0, limit = 0;
        if (SPARSE) {
            limit = a.ctx_lens ? visible(a, w.row0) : a.cap;
        } else {
            least = WINDOW ? span.least : keys;  // the smallest visible count: steps below it need no mask
            for (int r = 0; r < w.rows && !WINDOW; ++r) least = min(least, visible(a, w.row0 + r));
        }
        constexpr int kQ = NARROW ? D / 32 : D / 16;
        i32x4 q[kQ];
        const uint16_t *qrow = static_cast<const uint16_t *>(a.q) + pair.row * a.q_row + pair.head * a.q_head;
#pragma unroll
        for (int c = 0; c < kQ; ++c) {
            q[c] = i32x4{0, 0, 0, 0};
            if (pair.live)
                q[c] = *reinterpret_cast<const i32x4 *>(qrow + (NARROW ? 32 * c + 8 * (lane >> 4) : 16 * c + 8 * (lane >> 5)));
        }

        uint8_t *mine = sh.ring[wave];
        const uint32_t mine_lds = lds_offset(mine);
        const uint32_t entry_lds = lds_offset(sh.entry[wave]), column_lds = lds_offset(sh.column[wave]);
        const int32_t *table = a.block_table + (int64_t)max(w.req, 0) * a.max_blocks;
        const int32_t *idx = SPARSE ? a.idx + (int64_t)w.row0 * a.k : nullptr;
        // the wave's step j, and this lane's place in it (both half waves alike)
        const auto place = [&](int j) {
            return token_step<WINDOW>(span, t0 + wave + j * WAVES) * kStreamKeys + (lane & 31);
        };
        const auto have = [&](int j) { return t0 + wave + j * WAVES < t1; };

        struct Token {
            uint32_t entry, in;  // table column, place in the block
            bool seen;
        };
        const auto copy_column = [&](int j) {
            const int pos = min(place(j), keys - 1);
            copy4(idx + pos / a.ratio, column_lds + (j & 1) * 4 * kWave);
        };
        const auto token = [&](int j) {
            Token k;
            const int pos = place(j);
            uint32_t tok;
            if constexpr (SPARSE) {
                const int column = sh.column[wave][j & 1][lane];
                const int64_t wide = (int64_t)column * a.ratio + pos % a.ratio;
                k.seen = pos < keys && column >= 0 && wide < limit;
                tok = k.seen ? (uint32_t)wide : 0u;
            } else {
                // behind the last visible key the copies take that key again
                k.seen = true;
                tok = (uint32_t)max(copied_token<WINDOW>(span, pos), 0);
            }
            k.entry = block_index(a, tok);
            k.in = tok - k.entry * (uint32_t)a.block_size;
            return k;
        };
        const auto copy_entry = [&](int j, const Token &k) {
            uint32_t lds = entry_lds + (j & 1) * 4 * kWave;
            // (with the window's arithmetic the compiler keeps this in a vector register)
            if constexpr (WINDOW) lds = __builtin_amdgcn_readfirstlane(lds);
            copy4(table + k.entry, lds);
        };
        // byte offsets of the keys that this lane copies parts of, which keys take part, and which lie
        // behind table entries outside the pool
        struct Step {
            int64_t at[kCopies];
            uint32_t seen, bad;
        };
        const auto locate = [&](int j, const Token &k) {
            Step s;
            const int entry = sh.entry[wave][j & 1][lane];
            const bool bad = entry < 0 || entry >= a.num_blocks || w.req < 0;
            s.seen = (uint32_t)ballot(k.seen);
            s.bad = (uint32_t)ballot(bad && k.seen);
            const int64_t off = kv_offset(a, bad ? 0 : entry, k.in, w.hk);
            int lo = (int)off, hi = (int)(off >> 32);
            if (SPARSE && s.seen != 0xFFFFFFFFu && s.seen != 0) {
                // places without a token take the first seen token's key
                const int first = __builtin_ctz(s.seen);
                const int flo = readlane(lo, first), fhi = readlane(hi, first);
                lo = k.seen ? lo : flo;
                hi = k.seen ? hi : fhi;
            }
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int row = i * kKeysPerCopy + lane / kLanesPerKey;
                s.at[i] = ((int64_t)shfl_i(hi, row) << 32) | (uint32_t)shfl_i(lo, row);
            }
            return s;
        };
        const auto copy_rows = [&](const uint8_t *cache, const Step &s, bool values) {
            const uint32_t lds = mine_lds + (values ? kTileBytes : 0);
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const int row = i * kKeysPerCopy + lane / kLanesPerKey, chunk = lane % kLanesPerKey;
                copy16(cache + s.at[i] + 16 * (chunk ^ (values ? swz_v<D>(row) : swz_k<D>(row))),
                       lds + i * 16 * kWave);
            }
        };

        typedef typename Tile<NARROW>::V V;  // scores and outputs of one MFMA: 4 or 16 per lane
        constexpr int kScores = NARROW ? 2 : 1, kOut = NARROW ? D / 16 : D / 32, kRegs = NARROW ? 4 : 16;
        V o[kOut] = {};
        float m = kNegInf, l = 0.0f;  // l: this lane's part of the sum
        const auto key_of = [&](int u, int i) { return NARROW ? 16 * u + 4 * (lane >> 4) + i : score_key(i, lane); };
        if (have(0)) {
            if constexpr (SPARSE) {
                copy_column(0);
                copy_column(1);
                wait_copies();
            }
            Token k0 = token(0), next = token(1);
            copy_entry(0, k0);
            wait_copies();
            // q is waited for here: the compiler would wait for it, and with it for
            // every copy, in the loop
#pragma unroll
            for (int c = 0; c < kQ; ++c) asm volatile("" : "+v"(q[c]));
            Step cur = locate(0, k0), ahead = cur;
            copy_rows(a.kcache, cur, false);
            copy_entry(1, next);
            if constexpr (SPARSE) copy_column(2);
            copy_rows(a.vcache, cur, true);
            for (int j = 0; have(j); ++j) {
                const bool more = have(j + 1);
                const int s = token_step<WINDOW>(span, t0 + wave + j * WAVES);
                wait_all_but<kCopies>();
                V z[kScores];
                if constexpr (NARROW) score_narrow<DT, D>(mine, q, z, lane);
                else z[0] = score_tile<DT, D>(mine, q, lane);
                if (more) {
                    ahead = locate(j + 1, next);
                    wait_reads();
                    copy_rows(a.kcache, ahead, false);
                }
                if (cur.bad) {
#pragma unroll
                    for (int u = 0; u < kScores; ++u)
#pragma unroll
                        for (int i = 0; i < kRegs; ++i)
                            z[u][i] = (cur.bad >> key_of(u, i)) & 1 ? __builtin_nanf("") : z[u][i];
                }
                if (SPARSE) {
                    if (cur.seen != 0xFFFFFFFFu) {
#pragma unroll
                        for (int u = 0; u < kScores; ++u)
#pragma unroll
                            for (int i = 0; i < kRegs; ++i)
                                z[u][i] = (cur.seen >> key_of(u, i)) & 1 ? z[u][i] : kNegInf;
                    }
                } else if (partly_seen<WINDOW, kStreamKeys>(a, s * kStreamKeys, least, keys)) {
#pragma unroll
                    for (int i = 0; i < kRegs; ++i)
                        z[0][i] = sees<WINDOW>(a, ctx, s * kStreamKeys + key_of(0, i)) ? z[0][i] : kNegInf;
                }
                softmax_step<DT>(z, a.scale_log2, m, l, o);
                if (more) wait_all_but<kCopies>();
                else wait_copies();
                // a step without tokens holds the values of block 0, whatever they are
                if (!SPARSE || cur.seen != 0) {
                    if constexpr (NARROW) output_narrow<DT, D>(mine + kTileBytes, z, o, lane);
                    else output_tile<DT, D>(mine + kTileBytes, z[0], o, lane);
                }
                if (more) {
                    next = token(j + 2);
                    wait_reads();
                    copy_entry(j + 2, next);
                    if constexpr (SPARSE) copy_column(j + 3);
                    copy_rows(a.vcache, ahead, true);
                    cur = ahead;
                }
            }
            wait_copies();
        }
        l = xor32_sum(l);
        if (NARROW) l = xor16_sum(l);

        // join the waves' states: each leaves its output in its own buffers
        float *left = reinterpret_cast<float *>(mine);
        const int pair_at = NARROW ? lane & 15 : lane & 31;
#pragma unroll
        for (int c = 0; c < kOut; ++c)
#pragma unroll
            for (int g = 0; g < kRegs / 4; ++g) {
                const f32x4 v = {o[c][4 * g], o[c][4 * g + 1], o[c][4 * g + 2], o[c][4 * g + 3]};
                const int d = NARROW ? 16 * c + 4 * (lane >> 4) : out_element<D>(c, 4 * g, lane);
                *reinterpret_cast<f32x4 *>(left + left_at(pair_at, d / 4)) = v;
            }
        if (lane == pair_at) {
            sh.top_of[wave][lane] = m;
            sh.sum_of[wave][lane] = l;
        }
        __syncthreads();
        constexpr int kThreadsPer = kThreads / kAttnTile, kPer = D / kThreadsPer;  // outputs per thread
        const int pm = t / kThreadsPer, d0 = (t % kThreadsPer) * kPer;
        float top = kNegInf, total = 0.0f, r[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) r[i] = 0.0f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) top = fmaxf(top, sh.top_of[i][pm]);
        const float ref = top == kNegInf ? 0.0f : top;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
            const float f = __builtin_amdgcn_exp2f(sh.top_of[i][pm] - ref);
            total += sh.sum_of[i][pm] * f;
            const float *src = reinterpret_cast<const float *>(sh.ring[i]);
#pragma unroll
            for (int j = 0; j < kPer; j += 4) {
                const f32x4 v = *reinterpret_cast<const f32x4 *>(src + left_at(pm, (d0 + j) / 4));
#pragma unroll
                for (int e = 0; e < 4; ++e) r[j + e] += v[e] * f;
            }
        }
        const Pair pp = pair_of(a, w, pm);
        // a NaN output whose own sum is a number is mended (a pair whose own scores are
        // NaN has a NaN sum)
        bool nan = false;
#pragma unroll
        for (int i = 0; i < kPer; ++i) nan |= r[i] != r[i];
        const bool mend = ballot(nan && pp.live && total == total) != 0;
        if (pp.live && dest) {
#pragma unroll
            for (int i = 0; i < kPer; i += 4)
                *reinterpret_cast<f32x4 *>(dest + pm * D + d0 + i) = f32x4{r[i], r[i + 1], r[i + 2], r[i + 3]};
            if (d0 == 0) {
                dest[kAttnTile * D + pm] = top;
                dest[kAttnTile * (D + 1) + pm] = total;
            }
        } else if (pp.live) {
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
            typedef typename Half<DT>::T T;
            typedef T V4 __attribute__((ext_vector_type(4)));
            T *out = static_cast<T *>(a.out) + pp.row * a.o_row + pp.head * a.o_head + d0;
#pragma unroll
            for (int i = 0; i < kPer; i += 4) {
                V4 v;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = (T)(r[i + j] * inv);
                *reinterpret_cast<V4 *>(out + i) = v;
            }
            if (a.lse && d0 == 0)
                a.lse[(int64_t)pp.row * (a.num_kv_heads * a.group) + pp.head] =
                    (top + __builtin_amdgcn_logf(total)) * kLn2;
        }
        if (mend) {
            __threadfence_block();  // what this wave wrote is read back
            mend_pairs(launch_args(), w, wave, span, t0, t1, total, dest);
        }
    }

    // The wave's pairs of the join over steps [t0, t1) (see mend_pair); sums: that of
    // its i-th pair in lanes 16 i on.
    static __device__ __attribute__((noinline)) void mend_pairs(const AttnArgs &a, TileWork w, int wave, KeySpan span,
                                                                int t0, int t1, float sums, float *dest) {
        const int k0 = t0 * kStreamKeys, k1 = min(t1 * kStreamKeys, span.keys);
        constexpr int kMine = kAttnTile / WAVES;
        const int32_t *idx = SPARSE ? a.idx + (int64_t)w.row0 * a.k : nullptr;
        const int limit = !SPARSE || !a.ctx_lens ? a.cap : visible(a, w.row0), req = max(w.req, 0);
        FirstPlaces<D> f;
        if constexpr (!WINDOW) f = first_places<DT, D, SPARSE>(a, req, w.hk, idx, limit, k0, k1);
        int f_row = -1;  // WINDOW: the row whose tokens f is of
        for (int i = 0; i < kMine; ++i) {
            const int p = wave * kMine + i;
            const Pair x = pair_of(a, w, p);
            const float sum = readlane_f(sums, kWave / kMine * i);
            if (!x.live || sum != sum) continue;
            PairPlace at = {static_cast<const uint16_t *>(a.q) + x.row * a.q_row + x.head * a.q_head,
                            static_cast<typename Half<DT>::T *>(a.out) + x.row * a.o_row + x.head * a.o_head,
                            a.lse ? a.lse + (int64_t)x.row * (a.num_kv_heads * a.group) + x.head : nullptr, nullptr,
                            nullptr, nullptr};
            if (dest) {
                at.state = dest + p * D;
                at.top = dest + kAttnTile * D + p;
                at.total = dest + kAttnTile * (D + 1) + p;
            }
            OwnPlaces own = {k0, SPARSE ? k1 : min(k1, visible(a, x.row)), 0, 0};
            if constexpr (WINDOW) {
                own = window_places<kStreamKeys>(a, span, visible(a, x.row), t0, t1);
                if (f_row != x.row) f = own_first_places<DT, D>(a, req, w.hk, own);
                f_row = x.row;
            }
            mend_pair<DT, D, SPARSE>(a, req, w.hk, own, f, false, at);
        }
    }
};

// one workgroup per tile
template <int DT, int D, bool SPARSE, bool NARROW>
__global__ __launch_bounds__(kStreamThreads, 2) void attn_stream_kernel(AttnArgs a) {
    typedef Stream<DT, D, SPARSE, NARROW, false> S;
    __shared__ typename S::Shared sh;
    TileWork w;
    if (!tile_work<SPARSE>(a, blockIdx.x, blockIdx.y, w)) return;
    const KeySpan span = tile_keys<SPARSE>(a, w.row0, w.rows);
    S::run(a, sh, w, span, 0, span_steps<kStreamKeys>(span), nullptr);
}

// Work in units of a step of every wave: a tile with rows has one at
// least, so that rows that see nothing are written too.
__device__ __forceinline__ int units_of(int steps) { return max((steps + kStreamWaves - 1) / kStreamWaves, 1); }

// the workgroups that the line of `total` units is cut for: each has one at least
__device__ __forceinline__ int groups_of(int64_t total) { return (int)min(total, (int64_t)kStreamGroups); }
// the first unit of workgroup g, and the workgroup that has unit u: the last g with
// first_unit(g) <= u
__device__ __forceinline__ int64_t first_unit(int g, int64_t total) { return g * total / groups_of(total); }
__device__ __forceinline__ int group_of(int64_t u, int64_t total) {
    return (int)(((u + 1) * groups_of(total) + total - 1) / total) - 1;
}

// the workgroups with parts of a tile, its head part and its rows
struct TileSpan {
    int16_t first, last;
    int hs, row0, rows;
};

// Which slots have rows: bit l of word kPer w + i is that of slot kPer (64 w + l) + i,
// the i-th of lane l of wave w.
struct LiveSlots {
    static constexpr int kPer = kMaxSlots / kStreamThreads, kWords = kStreamWaves * kPer;
    uint64_t words[kWords];

    // how many slots before `slot` have rows, in word n
    __device__ __forceinline__ int count(int n, int slot) const {
        const int thread = slot / kPer - kWave * (n / kPer);  // `slot` is its slot % kPer
        const int lanes = thread + (n % kPer < slot % kPer);   // lanes whose slot of the word lies before
        const uint64_t below = lanes <= 0 ? 0 : lanes >= kWave ? ~(uint64_t)0 : ((uint64_t)1 << lanes) - 1;
        return __builtin_popcountll(words[n] & below);
    }
    // all words, by one wave
    __device__ __forceinline__ int before(int slot) const {
        static_assert(kWords <= kWave, "a word per lane");
        const int n = lane_id();
        return wave_total_sum(n < kWords ? count(n, slot) : 0);
    }
    // the same by one thread
    __device__ __forceinline__ int before_alone(int slot) const {
        int sum = 0;
        for (int n = 0; n < kWords; ++n) sum += count(n, slot);
        return sum;
    }
};

// Equal parts of all tiles' keys, one per workgroup.  Tile hs * slots + slot; the
// units of a slot are the same for every hs.
template <int DT, int D, bool SPARSE, bool NARROW>
__global__ __launch_bounds__(kStreamThreads, 2) void attn_cut_kernel(AttnArgs a) {
    typedef Stream<DT, D, SPARSE, NARROW, false> S;
    __shared__ typename S::Shared sh;
    __shared__ int32_t before[kMaxSlots + 1];  // units of the slots before
    __shared__ int32_t wave_sums[kStreamWaves];
    const int t = threadIdx.x, g = blockIdx.x;
    const int hss = a.num_kv_heads * a.num_subs, slots = a.slots;
    __shared__ Requests requests;  // dense only, as is `live`
    __shared__ LiveSlots live;
    if constexpr (SPARSE) {
        const int u = units_of((a.k * a.ratio + kStreamKeys - 1) / kStreamKeys);
        for (int i = t; i <= slots; i += kStreamThreads) before[i] = i * u;
        __syncthreads();
    } else {
        slot_counts<kStreamThreads, false>(a, requests, before, nullptr);
        constexpr int kPer = LiveSlots::kPer;
        int u[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int slot = t * kPer + i, keys = slot < slots ? before[slot] : -1;
            u[i] = keys < 0 ? 0 : units_of((keys + kStreamKeys - 1) / kStreamKeys);
            const uint64_t with_rows = ballot(keys >= 0);
            if ((t & 63) == 0) live.words[kPer * (t >> 6) + i] = with_rows;
        }
        __syncthreads();
        slot_sums<kStreamThreads>(before, slots, u, wave_sums);
    }
    const int per_head = before[slots];
    const int tiles = SPARSE ? slots : live.before(slots);  // of a head part
    const int64_t total = (int64_t)per_head * hss;
    if (g > 0 && g >= groups_of(total)) return;
    if (g == 0) {  // which workgroups have parts of each tile
        TileSpan *spans = reinterpret_cast<TileSpan *>(part_of<D>(a, kStreamGroups, a.tiles));
        for (int i = tiles * hss + t; i < a.tiles; i += kStreamThreads) spans[i] = {};
        for (int i = t; i < slots * hss; i += kStreamThreads) {
            const int hs = i / slots, slot = i - hs * slots;
            const int64_t u0 = (int64_t)hs * per_head + before[slot], u1 = (int64_t)hs * per_head + before[slot + 1];
            if (u1 == u0) continue;
            TileSpan s = {(int16_t)group_of(u0, total), (int16_t)group_of(u1 - 1, total), hs, slot, 1};
            if constexpr (!SPARSE) {
                const RowTile w = find_tile(a, requests, slot);
                s.row0 = w.row0;
                s.rows = w.rows;
            }
            const int tile = hs * tiles + (SPARSE ? slot : live.before_alone(slot));
            if (tile < a.tiles) spans[tile] = s;
        }
    }
    if (total == 0) return;
    int64_t u = first_unit(g, total);
    const int64_t end = first_unit(g + 1, total);
    while (u < end) {
        const int hs = __builtin_amdgcn_readfirstlane((int)(u / per_head));
        const int in_head = (int)(u - (int64_t)hs * per_head);
        int slot = 0, hi = slots;  // the slot with before[slot] <= in_head < before[slot + 1]
        while (hi - slot > 1) {
            const int mid = (slot + hi) >> 1;
            if (before[mid] <= in_head) slot = mid;
            else hi = mid;
        }
        slot = __builtin_amdgcn_readfirstlane(slot);
        const int64_t tile0 = (int64_t)hs * per_head + before[slot], tile1 = (int64_t)hs * per_head + before[slot + 1];
        const int64_t stop = min(end, tile1);
        TileWork w;
        if constexpr (SPARSE) {
            tile_work<SPARSE>(a, slot, hs, w);
        } else {
            part_heads(a, hs, w);
            const RowTile r = find_tile(a, requests, slot);
            w.req = __builtin_amdgcn_readfirstlane(r.req);
            w.row0 = __builtin_amdgcn_readfirstlane(r.row0);
            w.rows = __builtin_amdgcn_readfirstlane(r.rows);
        }
        const KeySpan span = tile_keys<SPARSE>(a, w.row0, w.rows);
        const int steps = span_steps<kStreamKeys>(span);
        const int t0 = __builtin_amdgcn_readfirstlane((int)(u - tile0) * kStreamWaves);
        const int t1 = __builtin_amdgcn_readfirstlane(min((int)(stop - tile0) * kStreamWaves, steps));
        float *dest = nullptr;
        if (u > tile0 || stop < tile1) {
            // q_starts that decrease could make more tiles than there are places for
            const int tile = hs * tiles + (SPARSE ? slot : live.before(slot));
            if (tile < a.tiles) dest = part_of<D>(a, g, tile);
        }
        S::run(a, sh, w, span, t0, t1, dest);
        u = stop;
        __syncthreads();  // the joined states have been read before the next copies land
    }
}

template <int DT, int D>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(AttnArgs a) {
    const int tile = blockIdx.x;
    const TileSpan s = reinterpret_cast<const TileSpan *>(part_of<D>(a, kStreamGroups, a.tiles))[tile];
    if (s.last <= s.first) return;
    constexpr int kPairs = kJoinThreads / (D / 4);
    const int m = blockIdx.y * kPairs + threadIdx.x / (D / 4);
    TileWork w;
    part_heads(a, s.hs, w);
    w.row0 = s.row0;
    w.rows = s.rows;
    const Pair pp = pair_of(a, w, m);
    if (!pp.live) return;
    const float *p = part_of<D>(a, s.first, tile);
    constexpr int kPart = kAttnTile * (D + 2);
    join_parts<DT, D, kAttnTile>(
        p, kPart, s.last - s.first + 1, m, 4 * (threadIdx.x % (D / 4)),
        static_cast<typename Half<DT>::T *>(a.out) + pp.row * a.o_row + pp.head * a.o_head,
        a.lse ? a.lse + (int64_t)pp.row * (a.num_kv_heads * a.group) + pp.head : nullptr);
}

template <int DT, int D, bool SPARSE, bool NARROW>
hipError_t run_stream(const AttnArgs &a, hipStream_t s) {
    const unsigned heads = (unsigned)(a.num_kv_heads * a.num_subs);
    if (!a.part) {
        hipLaunchKernelGGL((attn_stream_kernel<DT, D, SPARSE, NARROW>), dim3((unsigned)a.slots, heads), dim3(kStreamThreads),
                           0, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((attn_cut_kernel<DT, D, SPARSE, NARROW>), dim3(kStreamGroups), dim3(kStreamThreads), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attn_join_kernel<DT, D>),
                       dim3((unsigned)a.tiles, kAttnTile * (D / 4) / kJoinThreads), dim3(kJoinThreads), 0, s, a);
    return hipGetLastError();
}

// Windows: a tile's keys are bounded by the window, the first tokens and its rows, so the
// host knows into how many parts it is worth cutting tiles, and a workgroup finds its part
// without looking at the other tiles' rows.  Head part hs of tile `tile` has place
// tile * heads + hs; the first `whole` places have a workgroup each, the others one for
// each of their parts.  There are a.tiles places: those of tiles without rows hold CUs, take a
// state in the workspace and count against the most parts.  (With one for each of 128 requests of
// which 4 have a row, 23.1 us for 8 kv heads and windows of 4,096 where 4 requests take 19.7; of
// 256, too many to be cut, 41.6.)
//
// The tile with number `tile`, by a wave: false where there is none.  Of up to 1,024
// requests the tiles with rows are numbered without gaps, of more as slots.  (Slots without
// rows hold CUs before others can start: 64 requests of a row with windows of 4,096, 80 slots,
// 129 us, 98 without gaps.)
__device__ __forceinline__ int tiles_of(const AttnArgs &a, int s, int e) { return (max(e - s, 0) + a.tile_rows - 1) / a.tile_rows; }
__device__ __forceinline__ bool window_tile(const AttnArgs &a, int tile, RowTile &t) {
    const int n = a.num_reqs, lane = lane_id(), T = a.tile_rows;
    if (n > kCountedReqs) {
        // slots without rows come at a fixed pace, and workgroups go to the 8 XCDs in turn:
        // they are rotated among the 8 of a round, by another amount each round
        const int round = tile / 8, slot = 8 * round + (tile + round + round / 8) % 8;
        return slot < a.slots && find_tile(a, slot, t);
    }
    // a lane's requests, and the lane whose requests have the tile
    const int per = (n + kWave - 1) / kWave;
    int s = request_start(a, min(lane * per, n)), e = s, sum = 0;
    for (int k = 1; k <= per; ++k) {
        const int from = e;
        e = request_start(a, min(lane * per + k, n));
        sum += tiles_of(a, from, e);
    }
    int inc = wave_incl_sum(sum);
    uint64_t b = ballot(inc > tile);
    if (b == 0) return false;
    int at = __builtin_ctzll(b), before = readlane(inc - sum, at), req = at;
    if (per > 1) {  // its requests, one to a lane
        req = at * per + lane;
        s = request_start(a, min(req, n));
        e = request_start(a, min(req + 1, n));
        sum = lane < per ? tiles_of(a, s, e) : 0;
        inc = wave_incl_sum(sum) + before;
        b = ballot(inc > tile);
        at = __builtin_ctzll(b);
        req = readlane(req, at);
        before = readlane(inc - sum, at);
    }
    const int row0 = readlane(s, at) + (tile - before) * T;
    t = {req, row0, min(T, readlane(e, at) - row0)};
    return true;
}

// the rows of a tile whose parts are joined (0: none)
struct TileRows {
    int row0, rows;
};
template <int D>
__device__ __forceinline__ float *window_state(const AttnArgs &a, int64_t number) {
    return a.part + number * (kAttnTile * (D + 2));
}
template <int D>
__device__ __forceinline__ TileRows *window_rows(const AttnArgs &a) {
    return reinterpret_cast<TileRows *>(window_state<D>(a, (int64_t)(a.tiles - a.whole) * a.parts));
}

template <int DT, int D>
__global__ __launch_bounds__(kWave * kWindowWaves, 2) void window_stream_kernel(AttnArgs a) {
    typedef Stream<DT, D, false, false, true, kWindowWaves> S;
    __shared__ typename S::Shared sh;
    const int heads = a.num_kv_heads * a.num_subs, id = (int)(blockIdx.y * gridDim.x + blockIdx.x);
    const bool cut = id >= a.whole && a.parts > 1;
    const int parts = cut ? a.parts : 1, cut_at = cut ? (id - a.whole) / parts : 0;  // among those that are cut
    const int j = cut ? id - a.whole - cut_at * parts : 0, at = cut ? a.whole + cut_at : id;
    if (at >= a.tiles) return;  // behind the last one in the grid's last row
    const int tile = at / heads, hs = at - tile * heads;
    RowTile r;
    const bool have = window_tile(a, tile, r);
    if (cut && j == 0 && threadIdx.x == 0) window_rows<D>(a)[cut_at] = {r.row0, have ? r.rows : 0};
    if (!have) return;
    TileWork w = {__builtin_amdgcn_readfirstlane(r.req), __builtin_amdgcn_readfirstlane(r.row0),
                  __builtin_amdgcn_readfirstlane(r.rows), 0, 0, 0};
    part_heads(a, hs, w);
    const KeySpan span = window_keys(a, w.row0, w.rows);
    const int steps = span_steps<kStreamKeys>(span);
    const int t0 = __builtin_amdgcn_readfirstlane((int)((int64_t)steps * j / parts));
    const int t1 = __builtin_amdgcn_readfirstlane((int)((int64_t)steps * (j + 1) / parts));
    S::run(a, sh, w, span, t0, t1, cut ? window_state<D>(a, id - a.whole) : nullptr);
}

template <int DT, int D>
__global__ __launch_bounds__(kJoinThreads) void window_join_kernel(AttnArgs a) {
    const int cut_at = blockIdx.x, heads = a.num_kv_heads * a.num_subs;
    const TileRows r = window_rows<D>(a)[cut_at];
    constexpr int kPairs = kJoinThreads / (D / 4);
    const int m = blockIdx.y * kPairs + threadIdx.x / (D / 4);
    TileWork w;
    part_heads(a, (a.whole + cut_at) % heads, w);
    w.row0 = r.row0;
    w.rows = r.rows;
    const Pair pp = pair_of(a, w, m);
    if (!pp.live) return;
    join_parts<DT, D, kAttnTile>(
        window_state<D>(a, (int64_t)cut_at * a.parts), kAttnTile * (D + 2), a.parts, m, 4 * (threadIdx.x % (D / 4)),
        static_cast<typename Half<DT>::T *>(a.out) + pp.row * a.o_row + pp.head * a.o_head,
        a.lse ? a.lse + (int64_t)pp.row * (a.num_kv_heads * a.group) + pp.head : nullptr);
}

template <int DT, int D>
hipError_t run_window(const AttnArgs &a, hipStream_t s) {
    const int64_t cut = a.tiles - a.whole;
    // in rows of 2^16 workgroups: a dimension of a grid has less than 2^32 lanes (the places
    // behind the last tile have none)
    const int64_t groups = a.whole + cut * a.parts, row = 1 << 16;
    const dim3 grid((unsigned)(groups < row ? groups : row), (unsigned)((groups + row - 1) / row));
    hipLaunchKernelGGL((window_stream_kernel<DT, D>), grid, dim3(kWave * kWindowWaves), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.parts == 1) return e;
    hipLaunchKernelGGL((window_join_kernel<DT, D>), dim3((unsigned)cut, kAttnTile * (D / 4) / kJoinThreads),
                       dim3(kJoinThreads), 0, s, a);
    return hipGetLastError();
}

enum class Keys { kAll, kSelected, kWindow };

template <int DT, int D>
hipError_t run_kind(const AttnArgs &a, Keys keys, hipStream_t s) {
    if (keys == Keys::kAll) return run_stream<DT, D, false, false>(a, s);
    if (keys == Keys::kWindow) return run_window<DT, D>(a, s);
    return a.sub_heads <= 16 ? run_stream<DT, D, true, true>(a, s) : run_stream<DT, D, true, false>(a, s);
}

template <int DT>
hipError_t run_dim(const AttnArgs &a, Keys keys, hipStream_t s) {
    return a.head_dim == 128 ? run_kind<DT, 128>(a, keys, s) : run_kind<DT, 64>(a, keys, s);
}

hipError_t run_type(const AttnArgs &a, Keys keys, hipStream_t s) {
    return a.dtype == kBF16 ? run_dim<kBF16>(a, keys, s) : run_dim<kFP16>(a, keys, s);
}

}  // namespace

hipError_t launch_attn_stream(const AttnArgs &a, bool sparse, hipStream_t s) {
    return run_type(a, sparse ? Keys::kSelected : Keys::kAll, s);
}
hipError_t launch_window_stream(const AttnArgs &a, hipStream_t s) { return run_type(a, Keys::kWindow, s); }

int64_t attn_workspace_bytes(int head_dim, int64_t tiles) {
    return (kStreamGroups + tiles) * (kAttnTile * (head_dim + 2) * 4) + (int64_t)sizeof(TileSpan) * tiles;
}

int64_t window_workspace_bytes(int head_dim, int64_t tiles, int parts) {
    return tiles * parts * ((int64_t)kAttnTile * (head_dim + 2) * 4) + (int64_t)sizeof(TileRows) * tiles;
}

}  // namespace qsa
