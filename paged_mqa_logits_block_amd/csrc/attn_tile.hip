// Attention of a chunk of new tokens over the paged cache: requests with many
// stacked (row, head) pairs.
//
// One workgroup takes 256 pairs that share a kv head, 32 per wave, and walks the
// keys in steps of 64 that all waves share.  What bounds it is the matrix cores
// and, close behind, the vector unit (the exponentials) and LDS (a wave reads
// every key and value of the step, 32 KB at D = 128, for 32 MFMAs).  So the two
// waves of a SIMD take turns: while waves 0..3 multiply, waves 4..7 are in their
// softmax, and the other way round, with a barrier at each turn:
//
//   multiply s:  output += V(s - 1) weights(s - 1); scores = K(s) q
//   softmax s:   weights(s); copies of K(s + 2) and V(s + 1) started
//
// Keys and values have three buffers each, filled straight from global memory by
// all waves; the copies started in softmax s are waited for at the end of multiply
// s + 1, two turns later, and used from multiply s + 2 on.  The buffers they fill
// were last read in multiply s - 1, which all waves have left by then.
//
// Measured: 2,048 rows at the end of 16,384 tokens, 32 over 4 heads, D = 128, bf16:
// 471 us, 1,095 TFLOP/s, where a library product of 8192^3 reaches 1,390 on the same
// card (459 to 516 us by card; fp16 takes 8% more).  On the way there: 931 us with the
// arguments in scratch, 731 without, 674 with a lagging softmax reference, 569 with the
// turns and scalar table entries, 552 with heads dealt to the XCDs.  The clock drops
// from 2.3 to 1.9 GHz while the matrix cores work, so the card's power is part of the
// bound.

#include "attn_device.h"

namespace qsa {
namespace {

constexpr int kTileWaves = 8;
constexpr int kTileThreads = 64 * kTileWaves;
constexpr int kTileKeys = 64;
static_assert(kTilePairs == kAttnTile * kTileWaves, "32 pairs to a wave");

// A cut tile's state: the outputs of its 256 pairs relative to their references,
// the references, the sums.
template <int D>
constexpr int kTilePart = kTilePairs * (D + 2);

// The wave's pairs over keys [k0, k1), mended or done anew (see mend_pair); sums: that
// of pair p in lane p.
template <int DT, int D>
__device__ __attribute__((noinline)) void mend_pairs(const AttnArgs &a, int req, int row0, int rows, int wave, int hk,
                                                     int k0, int k1, int most, bool anew, float sums, float *dest) {
    FirstPlaces<D> f;
    if (!anew) f = first_places<DT, D, false>(a, req, hk, nullptr, 0, k0, min(k1, most));
    for (int p = 0; p < kAttnTile; ++p) {
        const int m = wave * kAttnTile + p, r = m / a.group;
        if (r >= rows) break;
        const float sum = readlane_f(sums, p);
        if (!anew && sum != sum) continue;
        const int row = row0 + r, head = hk * a.group + (m - r * a.group);
        PairPlace at = {static_cast<const uint16_t *>(a.q) + row * a.q_row + head * a.q_head,
                        static_cast<typename Half<DT>::T *>(a.out) + row * a.o_row + head * a.o_head,
                        a.lse ? a.lse + (int64_t)row * (a.num_kv_heads * a.group) + head : nullptr, nullptr, nullptr,
                        nullptr};
        if (dest) {
            at.state = dest + m * D;
            at.top = dest + kTilePairs * D + m;
            at.total = dest + kTilePairs * (D + 1) + m;
        }
        mend_pair<DT, D, false>(a, req, hk, k0, min(k1, visible(a, row)), f, anew, at);
    }
}

// s_barrier alone: what each wave has to wait for first stands before the calls
__device__ __forceinline__ void turn() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// The products of a turn: PV adds the values (LDS rows at vb) times the packed
// weights p to o, QK makes the scores z of the keys at kb.  They run in groups of
// four MFMAs; operands are read kAhead groups before their products (1 and 2 take the
// same time).
template <int DT, int D, bool PV, bool QK>
__device__ __forceinline__ void multiply(const uint8_t *vb, const uint8_t *kb, const i32x4 (&p)[4],
                                         const i32x4 (&q)[D / 16], f32x16 (&o)[D / 32], f32x16 (&z)[2], int lane) {
    constexpr int kAhead = 1, kM = D / 32, kV = PV ? kM : 0, kK = QK ? D / 32 : 0;
    i32x4 f[kAhead + 1][4];
    const int row = lane & 31, h = lane >> 5;
    const auto read = [&](int g) {
        i32x4 *x = f[g % (kAhead + 1)];
        if (g < kV) {  // 4 / kM blocks of 16 keys, all output tiles
#pragma unroll
            for (int i = 0; i < 4; i += kM) {
                i32x4 v[kM];
                read_values<D>(vb, 16 * (4 / kM * g + i / kM), v, lane);
#pragma unroll
                for (int m = 0; m < kM; ++m) x[i + m] = v[m];
            }
        } else {  // two chunks of both score tiles, whose chains of products take turns
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = *reinterpret_cast<const i32x4 *>(
                    kb + (32 * (i & 1) + row) * 2 * D + (((2 * (2 * (g - kV) + (i >> 1)) + h) ^ swz_k<D>(row)) << 4));
        }
    };
    if (QK) z[0] = z[1] = f32x16{};
#pragma unroll
    for (int g = 0; g < kAhead; ++g) read(g);
#pragma unroll
    for (int g = 0; g < kV + kK; ++g) {
        if (g + kAhead < kV + kK) read(g + kAhead);
        __builtin_amdgcn_sched_barrier(0);
        const i32x4 *x = f[g % (kAhead + 1)];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (g < kV) o[i % kM] = mfma32<DT>(x[i], p[4 / kM * g + i / kM], o[i % kM]);
            else z[i & 1] = mfma32<DT>(x[i], q[2 * (g - kV) + (i >> 1)], z[i & 1]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Workgroups go to the 8 XCDs in turn, and each XCD has an L2 of its own: the kv
// heads are dealt to the XCDs (as far as their number shares a factor with 8), so
// that an L2 sees the keys of few heads.  Within a head the tiles are taken from
// the last on: a chunk's last rows see the most keys.
constexpr int kXcds = 8;
__host__ __device__ __forceinline__ int head_classes(int heads) {
    return heads % 8 == 0 ? 8 : heads % 4 == 0 ? 4 : heads % 2 == 0 ? 2 : 1;
}
// workgroup `id` of a launch with per_head workgroups for each kv head: its head and
// its place among the head's
__device__ __forceinline__ bool place_of(const AttnArgs &a, int per_head, int id, int &hk, int &at) {
    const int classes = head_classes(a.num_kv_heads), x = id % kXcds, j = id / kXcds * (kXcds / classes) + x / classes;
    const int i = j / per_head;
    hk = x % classes + classes * i;
    at = per_head - 1 - (j - i * per_head);
    return hk < a.num_kv_heads;
}
inline unsigned place_grid(int num_kv_heads, int64_t per_head) {
    const int classes = head_classes(num_kv_heads), share = kXcds / classes;  // XCDs per class of heads
    return (unsigned)((per_head * (num_kv_heads / classes) + share - 1) / share * kXcds);
}

// WHOLE: the block size is a multiple of 8, so that the 8 keys that a wave copies in
// a step lie in one block: its table entry is read by a scalar load and the copies
// take a scalar base, with offsets that stay the same from step to step.  (With a
// table load and address per lane the copies' part of a turn took as long as the
// softmax: 1,100 cycles against 1,000.)
template <int D>
struct TileShared {
    __align__(16) uint8_t kring[3][kTileKeys * D * 2], vring[3][kTileKeys * D * 2];
    int most_of[kTileWaves], any_bad;
};

// steps [s0, min(s1, the tile's steps)) of tile w and kv head hk; dest: the place of
// the state, or null to write the outputs
template <int DT, int D, bool WHOLE>
__device__ __forceinline__ void run_steps(const AttnArgs &a, TileShared<D> &sh, const RowTile &w, int hk, int s0, int s1,
                                          float *dest) {
    constexpr int kStepBytes = kTileKeys * D * 2;  // keys (or values) of one step
    constexpr int kLanesPerKey = D / 8, kKeysPerCopy = kWave / kLanesPerKey;
    constexpr int kCopies = kTileKeys / kKeysPerCopy / kTileWaves;  // copies of each kind per wave
    auto &kring = sh.kring;
    auto &vring = sh.vring;
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));  // addresses are made anew for each range, not kept live across them
    const int lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int m = wave * kAttnTile + (lane & 31), r = m / a.group;
    const bool live = r < w.rows;
    const int row = w.row0 + r, head = hk * a.group + (m - r * a.group);

    // visible counts: of this pair, the wave's largest and smallest, the tile's largest
    const int ctx = live ? min(max(a.ctx_lens[row], 0), a.cap) : 0;
    const int wave_most = __builtin_amdgcn_readfirstlane(wave_max_i(ctx));
    const int wave_least = -__builtin_amdgcn_readfirstlane(wave_max_i(live ? -ctx : -0x7FFFFFFF));
    if (lane == 0) sh.most_of[wave] = wave_most;
    if (t == 0) sh.any_bad = 0;

    i32x4 q[D / 16];
    const uint16_t *qrow = static_cast<const uint16_t *>(a.q) + row * a.q_row + head * a.q_head;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        q[c] = i32x4{0, 0, 0, 0};
        if (live) q[c] = *reinterpret_cast<const i32x4 *>(qrow + 16 * c + 8 * (lane >> 5));
    }
    __syncthreads();
    int keys = 0;
#pragma unroll
    for (int i = 0; i < kTileWaves; ++i) keys = max(keys, sh.most_of[i]);
    keys = __builtin_amdgcn_readfirstlane(keys);
    const int steps = min(s1, (keys + kTileKeys - 1) / kTileKeys);
    const bool active = wave_most > s0 * kTileKeys;

    const uint32_t kring_lds = lds_offset(kring), vring_lds = lds_offset(vring);
    const int32_t *table = a.block_table + (int64_t)w.req * a.max_blocks;
    // This lane's keys of a step: rows kKeysPerCopy * (kCopies * wave + i) + lane /
    // kLanesPerKey.  Behind the last visible key the copies take that key again.
    const auto key_row = [&](int i) { return kKeysPerCopy * (kCopies * wave + i) + lane / kLanesPerKey; };
    const int chunk = lane % kLanesPerKey;
    bool met_bad = false;
    // loaded a step ahead of the copies: this lane's table entries, or the wave's
    int32_t entry[kCopies], whole_entry = 0;
    // where the copies of a step come from
    int64_t at[kCopies];
    const uint8_t *kbase = nullptr, *vbase = nullptr;
    uint32_t lane_at[kCopies];
    const uint32_t slot_bytes = a.kv_slot * 16;  // WHOLE: 8 slots are below 2^32 bytes
#pragma unroll
    for (int i = 0; i < kCopies; ++i) lane_at[i] = (uint32_t)(key_row(i) - 8 * wave) * slot_bytes;
    const auto load_entries = [&](int s) {
        if constexpr (WHOLE) {
            const uint32_t e = block_index(a, (uint32_t)min(s * kTileKeys + 8 * wave, keys - 1));
            whole_entry = ((const __attribute__((address_space(4))) int32_t *)(uintptr_t)table)[e];
        } else {
#pragma unroll
            for (int i = 0; i < kCopies; ++i)
                entry[i] = table[block_index(a, (uint32_t)min(s * kTileKeys + key_row(i), keys - 1))];
        }
    };
    // All entries count as waited for here, where the copies are waited for too:
    // waiting for one between two copies would wait for the copies before it.
    const auto pin_entries = [&]() {
        if constexpr (!WHOLE) {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) asm volatile("" : "+v"(entry[i]));
        }
    };
    const auto locate = [&](int s) {
        if constexpr (WHOLE) {
            const int first = min(s * kTileKeys + 8 * wave, keys - 1);
            const uint32_t e = block_index(a, (uint32_t)first);
            const bool bad = whole_entry < 0 || whole_entry >= a.num_blocks;
            met_bad |= bad;
            const int64_t off = kv_offset(a, bad ? 0 : whole_entry, (uint32_t)first - e * (uint32_t)a.block_size, hk);
            kbase = a.kcache + off;
            vbase = a.vcache + off;
            if (s * kTileKeys + 8 * wave + 8 > keys) {  // the last keys
#pragma unroll
                for (int i = 0; i < kCopies; ++i)
                    lane_at[i] = (uint32_t)min(key_row(i) - 8 * wave, keys - 1 - first) * slot_bytes;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                const uint32_t tok = (uint32_t)min(s * kTileKeys + key_row(i), keys - 1), e = block_index(a, tok);
                const bool bad = entry[i] < 0 || entry[i] >= a.num_blocks;
                met_bad |= bad;
                at[i] = kv_offset(a, bad ? 0 : entry[i], tok - e * (uint32_t)a.block_size, hk);
            }
        }
    };
    const auto copy_keys = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const uint32_t lds = kring_lds + buf * kStepBytes + (kCopies * wave + i) * 16 * kWave;
            const uint32_t piece = 16 * (chunk ^ swz_k<D>(key_row(i)));
            if constexpr (WHOLE) copy16(kbase, lane_at[i] + piece, lds);
            else copy16(a.kcache + at[i] + piece, lds);
        }
    };
    const auto copy_values = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const uint32_t lds = vring_lds + buf * kStepBytes + (kCopies * wave + i) * 16 * kWave;
            const uint32_t piece = 16 * (chunk ^ swz_v<D>(key_row(i)));
            if constexpr (WHOLE) copy16(vbase, lane_at[i] + piece, lds);
            else copy16(a.vcache + at[i] + piece, lds);
        }
    };

    f32x16 o[D / 32] = {};
    float ref = kNegInf, total = 0.0f;  // total: this lane's half of the sum
    if (steps > s0) {
        load_entries(s0);
        pin_entries();
        locate(s0);
        copy_keys(0);
        copy_values(0);
        load_entries(s0 + 1);
        pin_entries();
        locate(s0 + 1);  // past the end: the last key once more, never used
        copy_keys(1);
        load_entries(s0 + 2);
        wait_copies();
        pin_entries();
#pragma unroll
        for (int c = 0; c < D / 16; ++c) asm volatile("" : "+v"(q[c]));
        __syncthreads();
        if (wave >= kTileWaves / 2) turn();
        f32x16 z[2];
        i32x4 p[4];
        int b0 = 0, b1 = 1, b2 = 2;  // buffers of steps s, s + 1, s + 2 (and s - 1)
        const auto softmax_turn = [&](int s) {
            wait_copies();
            pin_entries();
            turn();
            if (s + 1 < steps) {
                copy_values(b1);
                if (s + 2 < steps) {
                    locate(s + 2);
                    copy_keys(b2);
                    load_entries(s + 3);
                }
            }
            if (active) {
                if ((s + 1) * kTileKeys > wave_least) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            z[u][i] = s * kTileKeys + 32 * u + score_key(i, lane) < ctx ? z[u][i] : kNegInf;
                }
                softmax_step<DT>(z, a.scale_log2, ref, total, o);
#pragma unroll
                for (int g = 0; g < 4; ++g) p[g] = pack8<DT>(z[g >> 1], 8 * (g & 1));
            }
            // a scalar load on its way would make the products wait for all LDS reads
            if constexpr (WHOLE) asm volatile("s_waitcnt lgkmcnt(0)" : "+s"(whole_entry));
            turn();
            const int b = b0;
            b0 = b1;
            b1 = b2;
            b2 = b;
        };
        if (active) multiply<DT, D, false, true>(vring[0], kring[0], p, q, o, z, lane);
        softmax_turn(s0);
        for (int s = s0 + 1; s < steps; ++s) {
            if (active) multiply<DT, D, true, true>(vring[b2], kring[b0], p, q, o, z, lane);
            softmax_turn(s);
        }
        if (active) multiply<DT, D, true, false>(vring[b2], kring[b0], p, q, o, z, lane);
        if (wave < kTileWaves / 2) turn();
        wait_copies();
    }
    total = xor32_sum(total);

    // Where the tile met a table entry outside the pool the wave's pairs are done anew,
    // each over its own keys; a NaN output whose own sum is a number is mended (a pair
    // whose own scores are NaN has a NaN sum).
    if (ballot(met_bad) && lane == 0) sh.any_bad = 1;
    __syncthreads();
    const bool anew = sh.any_bad != 0;
    bool nan = false;
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) nan |= o[c][i] != o[c][i];
    const bool mend = ballot(nan && live && total == total) != 0;
    if (live && !anew) {
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        typedef typename Half<DT>::T T;
        typedef T V4 __attribute__((ext_vector_type(4)));
        T *out = static_cast<T *>(a.out) + row * a.o_row + head * a.o_head;
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int at = out_element<D>(c, 4 * g, lane);
                const f32x4 v = {o[c][4 * g], o[c][4 * g + 1], o[c][4 * g + 2], o[c][4 * g + 3]};
                if (dest) {
                    *reinterpret_cast<f32x4 *>(dest + m * D + at) = v;
                    continue;
                }
                V4 x;
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = (T)(v[j] * inv);
                *reinterpret_cast<V4 *>(out + at) = x;
            }
        if (lane < kAttnTile) {
            if (dest) {
                dest[kTilePairs * D + m] = ref;
                dest[kTilePairs * (D + 1) + m] = total;
            } else if (a.lse) {
                a.lse[(int64_t)row * (a.num_kv_heads * a.group) + head] = (ref + __builtin_amdgcn_logf(total)) * kLn2;
            }
        }
    }
    if (anew || mend) {
        __threadfence_block();  // what this wave wrote is read back
        mend_pairs<DT, D>(launch_args(), w.req, w.row0, w.rows, wave, hk, s0 * kTileKeys, steps * kTileKeys, wave_most,
                          anew, total, dest);
    }
}

// one workgroup per tile
template <int DT, int D, bool WHOLE>
__global__ __launch_bounds__(kTileThreads, 2) void attn_tile_kernel(AttnArgs a) {
    __shared__ TileShared<D> sh;
    int hk, slot;
    RowTile w;
    if (!place_of(a, a.slots, blockIdx.x, hk, slot) || !find_tile(a, slot, w)) return;
    w.req = __builtin_amdgcn_readfirstlane(w.req);
    run_steps<DT, D, WHOLE>(a, sh, w, hk, 0, 0x7FFFFFFF, nullptr);
}

// Cut launch: every tile's steps are cut into pieces of about `piece` steps, one per
// workgroup, with `piece` chosen from the tiles' total so that there are about as
// many pieces as CUs; a tile of up to that many steps stays whole.  (Equal parts of
// the whole line, as in the streaming kernel, would give most workgroups two
// tiles here, each with the start and the end of a tile's work.)  Pieces of cut
// tiles leave their states in the workspace, at most 2 kStreamGroups of them: a cut
// tile's pieces are more than half of `piece` long.
constexpr int kLeastSteps = 4;

struct TileSpan {
    int first, pieces;  // places of a cut tile's states
    int row0, rows;
};

template <int DT, int D, bool WHOLE>
__global__ __launch_bounds__(kTileThreads, 2) void attn_tile_cut_kernel(AttnArgs a) {
    __shared__ TileShared<D> sh;
    // pieces of the slots before (at most 1,280), and, shifted by 16, those of cut tiles
    // among them (at most 512)
    __shared__ int32_t before[kMaxSlots + 1];
    __shared__ int32_t steps_of[kMaxSlots + 1];  // steps of the slot; first its largest visible count
    __shared__ int32_t wave_sums[kTileWaves], sums[2];
    __shared__ Requests requests;
    const int t = threadIdx.x, slots = a.slots;
    constexpr int kPer = kMaxSlots / kTileThreads;
    if (t < 2) sums[t] = 0;
    slot_counts<kTileThreads>(a, requests, steps_of);
    int u[kPer], steps = 0, tiles = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int slot = t * kPer + i, keys = slot < slots ? steps_of[slot] : -1;
        u[i] = keys < 0 ? 0 : max((keys + kTileKeys - 1) / kTileKeys, 1);  // rows that see nothing are written too
        steps += u[i];
        tiles += keys >= 0;
    }
    steps = wave_total_sum(steps);
    tiles = wave_total_sum(tiles);
    if ((t & 63) == 0) {
        atomicAdd(&sums[0], steps);
        atomicAdd(&sums[1], tiles);
    }
    __syncthreads();
    // pieces are total / piece and about half a piece more per tile; rounded up, so
    // that total / piece is below `room` also where the quotient is off by a rounding
    const float total = (float)sums[0] * (float)a.num_kv_heads;
    const int half = (int)min((int64_t)sums[1] * a.num_kv_heads / 2, (int64_t)kStreamGroups);
    const int room = max(kStreamGroups - half, kStreamGroups / 4);
    const int piece = max((int)(total / (float)room * 1.000001f) + 1, kLeastSteps);
    int c[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int slot = t * kPer + i;
        if (slot < slots) steps_of[slot] = u[i];
        c[i] = (u[i] + piece - 1) / piece;
        c[i] |= c[i] > 1 ? c[i] << 16 : 0;
    }
    slot_sums<kTileThreads>(before, slots, c, wave_sums);
    const auto pieces_before = [&](int slot) { return before[slot] & 0xFFFF; };
    const auto cut_before = [&](int slot) { return before[slot] >> 16; };
    const int per_head = pieces_before(slots), cut_per_head = cut_before(slots);

    TileSpan *spans = reinterpret_cast<TileSpan *>(a.part + (int64_t)2 * kStreamGroups * kTilePart<D>);
    for (int i = (int)blockIdx.x * kTileThreads + t; i < slots * a.num_kv_heads; i += (int)gridDim.x * kTileThreads) {
        const int hk = i / slots, slot = i - hk * slots;
        TileSpan s = {hk * cut_per_head + cut_before(slot), cut_before(slot + 1) - cut_before(slot), 0, 0};
        if (s.pieces > 0) {
            const RowTile w = find_tile(a, requests, slot);
            s.row0 = w.row0;
            s.rows = w.rows;
        }
        spans[i] = s;
    }
    int hk, at;
    if (per_head == 0 || !place_of(a, per_head, blockIdx.x, hk, at)) return;
    int slot = 0, hi = slots;  // the last slot with at most `at` pieces before it
    while (hi - slot > 1) {
        const int mid = (slot + hi) >> 1;
        if (pieces_before(mid) <= at) slot = mid;
        else hi = mid;
    }
    slot = __builtin_amdgcn_readfirstlane(slot);
    const int n = pieces_before(slot + 1) - pieces_before(slot), j = at - pieces_before(slot), all = steps_of[slot];
    RowTile w = find_tile(a, requests, slot);
    w.req = __builtin_amdgcn_readfirstlane(w.req);
    w.row0 = __builtin_amdgcn_readfirstlane(w.row0);
    w.rows = __builtin_amdgcn_readfirstlane(w.rows);
    float *dest = n > 1 ? a.part + (int64_t)(hk * cut_per_head + cut_before(slot) + j) * kTilePart<D> : nullptr;
    run_steps<DT, D, WHOLE>(a, sh, w, hk, __builtin_amdgcn_readfirstlane((int)((int64_t)all * j / n)),
                            __builtin_amdgcn_readfirstlane((int)((int64_t)all * (j + 1) / n)), dest);
}

template <int DT, int D>
__global__ __launch_bounds__(kJoinThreads) void attn_tile_join_kernel(AttnArgs a) {
    const TileSpan s = reinterpret_cast<const TileSpan *>(a.part + (int64_t)2 * kStreamGroups * kTilePart<D>)[blockIdx.x];
    if (s.pieces <= 1) return;
    constexpr int kPairs = kJoinThreads / (D / 4);
    const int hk = blockIdx.x / a.slots, m = blockIdx.y * kPairs + threadIdx.x / (D / 4), r = m / a.group;
    if (r >= s.rows) return;
    const int row = s.row0 + r, head = hk * a.group + (m - r * a.group);
    join_parts<DT, D, kTilePairs>(
        a.part + (int64_t)s.first * kTilePart<D>, kTilePart<D>, s.pieces, m, 4 * (threadIdx.x % (D / 4)),
        static_cast<typename Half<DT>::T *>(a.out) + row * a.o_row + head * a.o_head,
        a.lse ? a.lse + (int64_t)row * (a.num_kv_heads * a.group) + head : nullptr);
}

template <int DT, int D, bool WHOLE>
hipError_t run_tile(const AttnArgs &a, hipStream_t s) {
    if (!a.part) {
        hipLaunchKernelGGL((attn_tile_kernel<DT, D, WHOLE>), dim3(place_grid(a.num_kv_heads, a.slots)),
                           dim3(kTileThreads), 0, s, a);
        return hipGetLastError();
    }
    // at most kStreamGroups pieces and one more per tile
    const int64_t per_head = a.slots + kStreamGroups / a.num_kv_heads + 1;
    hipLaunchKernelGGL((attn_tile_cut_kernel<DT, D, WHOLE>), dim3(place_grid(a.num_kv_heads, per_head)),
                       dim3(kTileThreads), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attn_tile_join_kernel<DT, D>),
                       dim3((unsigned)(a.slots * a.num_kv_heads), kTilePairs * (D / 4) / kJoinThreads),
                       dim3(kJoinThreads), 0, s, a);
    return hipGetLastError();
}

template <int DT>
hipError_t run_dim(const AttnArgs &a, hipStream_t s) {
    const bool whole = a.block_size % 8 == 0 && a.kv_slot < (1u << 25);
    if (a.head_dim == 128) return whole ? run_tile<DT, 128, true>(a, s) : run_tile<DT, 128, false>(a, s);
    return whole ? run_tile<DT, 64, true>(a, s) : run_tile<DT, 64, false>(a, s);
}

}  // namespace

hipError_t launch_attn_tile(const AttnArgs &a, hipStream_t s) {
    return a.dtype == kBF16 ? run_dim<kBF16>(a, s) : run_dim<kFP16>(a, s);
}

int64_t attn_tile_workspace_bytes(int head_dim, int64_t tiles) {
    return (int64_t)2 * kStreamGroups * kTilePairs * (head_dim + 2) * 4 + (int64_t)sizeof(TileSpan) * tiles;
}

}  // namespace qsa
