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

#include "attn_device.h"

namespace qsa {
namespace {

constexpr int kTileWaves = 8;
constexpr int kTileThreads = 64 * kTileWaves;
constexpr int kTileKeys = 64;

// The wave's pairs, each over its own visible keys (see own_range).
template <int DT, int D>
__device__ __attribute__((noinline)) void own_pairs(const AttnArgs &a, int req, int row0, int rows, int wave,
                                                    int hk) {
    typedef typename Half<DT>::T T;
    const int lane = lane_id();
    for (int p = 0; p < kAttnTile; ++p) {
        const int m = wave * kAttnTile + p, r = m / a.group;
        if (r >= rows) break;
        const int row = row0 + r, head = hk * a.group + (m - r * a.group);
        float top, total, o[D / 64];
        own_range<DT, D>(a, req, static_cast<const uint16_t *>(a.q) + row * a.q_row + head * a.q_head, hk, 0,
                         min(max(a.ctx_lens[row], 0), a.cap), top, total, o);
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        T *out = static_cast<T *>(a.out) + row * a.o_row + head * a.o_head;
        for (int i = 0; i < D / 64; ++i) out[lane * (D / 64) + i] = (T)(o[i] * inv);
        if (a.lse && lane == 0)
            a.lse[(int64_t)row * (a.num_kv_heads * a.group) + head] = (top + __builtin_amdgcn_logf(total)) * kLn2;
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
// four MFMAs; operands are read kAhead groups before their products, as four
// waves read at once and a read takes longer than one group's products.
template <int DT, int D, bool PV, bool QK>
__device__ __forceinline__ void multiply(const uint8_t *vb, const uint8_t *kb, const i32x4 (&p)[4],
                                         const i32x4 (&q)[D / 16], f32x16 (&o)[D / 32], f32x16 (&z)[2], int lane) {
    constexpr int kAhead = 2, kM = D / 32, kV = PV ? kM : 0, kK = QK ? D / 32 : 0;
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

// WHOLE: the block size is a multiple of 8, so that the 8 keys that a wave copies in
// a step lie in one block: its table entry is read by a scalar load and the copies
// take a scalar base, with offsets that stay the same from step to step.  (With a
// table load and address per lane the copies' part of a turn took as long as the
// softmax: 1,100 cycles against 1,000.)
template <int DT, int D, bool WHOLE>
__global__ __launch_bounds__(kTileThreads, 2) void attn_tile_kernel(AttnArgs a) {
    constexpr int kStepBytes = kTileKeys * D * 2;  // keys (or values) of one step
    constexpr int kLanesPerKey = D / 8, kKeysPerCopy = kWave / kLanesPerKey;
    constexpr int kCopies = kTileKeys / kKeysPerCopy / kTileWaves;  // copies of each kind per wave
    __shared__ __align__(16) uint8_t kring[3][kStepBytes], vring[3][kStepBytes];
    __shared__ int most_of[kTileWaves], any_bad;

    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int hk = blockIdx.y;
    RowTile w;
    if (!find_tile(a, blockIdx.x, w)) return;
    w.req = __builtin_amdgcn_readfirstlane(w.req);
    const int m = wave * kAttnTile + (lane & 31), r = m / a.group;
    const bool live = r < w.rows;
    const int row = w.row0 + r, head = hk * a.group + (m - r * a.group);

    // visible counts: of this pair, the wave's largest and smallest, the tile's largest
    const int ctx = live ? min(max(a.ctx_lens[row], 0), a.cap) : 0;
    const int wave_most = __builtin_amdgcn_readfirstlane(wave_max_i(ctx));
    const int wave_least = -__builtin_amdgcn_readfirstlane(wave_max_i(live ? -ctx : -0x7FFFFFFF));
    if (lane == 0) most_of[wave] = wave_most;
    if (t == 0) any_bad = 0;

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
    for (int i = 0; i < kTileWaves; ++i) keys = max(keys, most_of[i]);
    keys = __builtin_amdgcn_readfirstlane(keys);
    const int steps = (keys + kTileKeys - 1) / kTileKeys;
    const bool active = wave_most > 0;

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
    if (steps > 0) {
        load_entries(0);
        pin_entries();
        locate(0);
        copy_keys(0);
        copy_values(0);
        load_entries(1);
        pin_entries();
        locate(1);  // past the end: the last key once more, never used
        copy_keys(1);
        load_entries(2);
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
                softmax_step(z, a.scale_log2, ref, total, o);
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
        softmax_turn(0);
        for (int s = 1; s < steps; ++s) {
            if (active) multiply<DT, D, true, true>(vring[b2], kring[b0], p, q, o, z, lane);
            softmax_turn(s);
        }
        if (active) multiply<DT, D, true, false>(vring[b2], kring[b0], p, q, o, z, lane);
        if (wave < kTileWaves / 2) turn();
        wait_copies();
    }
    total = xor32_sum(total);

    // The wave's pairs are done again, each over its own keys, where the tile met a
    // table entry outside the pool, or where a NaN can come from a value that only
    // other rows of the wave see (zero weight times a value that is not finite).
    if (ballot(met_bad) && lane == 0) any_bad = 1;
    __syncthreads();
    bool again = any_bad != 0;
    if (wave_least < wave_most) {
        bool nan = false;
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) nan |= o[c][i] != o[c][i];
        again |= ballot(nan && live) != 0;
    }
    if (again) {
        own_pairs<DT, D>(launch_args(), w.req, w.row0, w.rows, wave, hk);
        return;
    }
    if (!live) return;
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    typedef typename Half<DT>::T T;
    typedef T V4 __attribute__((ext_vector_type(4)));
    T *out = static_cast<T *>(a.out) + row * a.o_row + head * a.o_head;
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            V4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = (T)(o[c][4 * g + j] * inv);
            *reinterpret_cast<V4 *>(out + out_element<D>(c, 4 * g, lane)) = v;
        }
    if (a.lse && lane < kAttnTile)
        a.lse[(int64_t)row * (a.num_kv_heads * a.group) + head] = (ref + __builtin_amdgcn_logf(total)) * kLn2;
}

template <int DT, int D>
hipError_t run_tile(const AttnArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)a.slots, (unsigned)a.num_kv_heads);
    if (a.block_size % 8 == 0 && a.kv_slot < (1u << 25))
        hipLaunchKernelGGL((attn_tile_kernel<DT, D, true>), grid, dim3(kTileThreads), 0, s, a);
    else
        hipLaunchKernelGGL((attn_tile_kernel<DT, D, false>), grid, dim3(kTileThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_tile(const AttnArgs &a, hipStream_t s) {
    if (a.dtype == kBF16) return a.head_dim == 128 ? run_tile<kBF16, 128>(a, s) : run_tile<kBF16, 64>(a, s);
    return a.head_dim == 128 ? run_tile<kFP16, 128>(a, s) : run_tile<kFP16, 64>(a, s);
}

}  // namespace qsa
