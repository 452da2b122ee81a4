// Attention of a chunk of new tokens over the paged cache: requests with many
// stacked (row, head) pairs.
//
// One workgroup takes 256 pairs that share a kv head, 32 per wave, and walks the
// keys in steps of 64 that all waves share.  What bounds it is the matrix
// cores and, beside them, LDS: a wave reads every key and value of the step
// (32 KB at D = 128) for 32 MFMAs.  A step's keys and values are copied to LDS by
// all waves, straight from global memory, while the step before is worked on;
// one barrier a step.

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

template <int DT, int D>
__global__ __launch_bounds__(kTileThreads, 2) void attn_tile_kernel(AttnArgs a) {
    constexpr int kStepBytes = kTileKeys * D * 2;  // keys (or values) of one step
    constexpr int kLanesPerKey = D / 8, kKeysPerCopy = kWave / kLanesPerKey;
    constexpr int kCopies = kTileKeys / kKeysPerCopy / kTileWaves;  // copies of each kind per wave
    __shared__ __align__(16) uint8_t ring[2 * 2 * kStepBytes];

    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int hk = blockIdx.y;
    RowTile w;
    if (!find_tile(a, blockIdx.x, w)) return;
    const int m = wave * kAttnTile + (lane & 31), r = m / a.group;
    const bool live = r < w.rows;
    const int row = w.row0 + r, head = hk * a.group + (m - r * a.group);
    const auto visible = [&](int at) { return min(max(a.ctx_lens[at], 0), a.cap); };

    // visible counts: of this pair, the wave's largest and smallest, the tile's largest
    const int ctx = live ? visible(row) : 0;
    const int wave_most = __builtin_amdgcn_readfirstlane(wave_max_i(ctx));
    const int wave_least = -__builtin_amdgcn_readfirstlane(wave_max_i(live ? -ctx : -0x7FFFFFFF));
    __shared__ int most_of[kTileWaves];
    if (lane == 0) most_of[wave] = wave_most;
    __syncthreads();
    int keys = 0;
#pragma unroll
    for (int i = 0; i < kTileWaves; ++i) keys = max(keys, most_of[i]);
    keys = __builtin_amdgcn_readfirstlane(keys);
    const int steps = (keys + kTileKeys - 1) / kTileKeys;

    i32x4 q[D / 16];
    const uint16_t *qrow = static_cast<const uint16_t *>(a.q) + row * a.q_row + head * a.q_head;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        q[c] = i32x4{0, 0, 0, 0};
        if (live) q[c] = *reinterpret_cast<const i32x4 *>(qrow + 16 * c + 8 * (lane >> 5));
    }

    const uint32_t ring_lds = lds_offset(ring);
    const int32_t *table = a.block_table + (int64_t)w.req * a.max_blocks;
    // this lane's keys of a step: row kKeysPerCopy * (kCopies * wave + i) + lane / kLanesPerKey
    struct Places {
        int32_t entry[kCopies], in[kCopies];
    };
    const auto key_row = [&](int i) { return kKeysPerCopy * (kCopies * wave + i) + lane / kLanesPerKey; };
    const auto load_entries = [&](int s) {
        Places p;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            // behind the last visible key the copies take that key again
            const uint32_t tok = (uint32_t)min(s * kTileKeys + key_row(i), keys - 1);
            const uint32_t e = tok / (uint32_t)a.block_size;
            p.in[i] = (int32_t)(tok - e * (uint32_t)a.block_size);
            p.entry[i] = table[e];
        }
        return p;
    };
    __shared__ uint32_t bad_of[2][2 * kTileWaves];  // keys behind table entries outside the pool
    const auto start_copies = [&](const Places &p, int buf) {
        const uint32_t lds = ring_lds + buf * 2 * kStepBytes;
        const int chunk = lane % kLanesPerKey;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) {
            const bool bad = p.entry[i] < 0 || p.entry[i] >= a.num_blocks;
            const int at = key_row(i), first = kCopies * wave + i;
            const int64_t off = (bad ? 0 : (int64_t)p.entry[i] * a.kv_block) + (int64_t)p.in[i] * a.kv_slot +
                                (int64_t)hk * a.kv_head;
            copy16(a.kcache + 2 * (off + 8 * (chunk ^ swz_k<D>(at))), lds + first * 16 * kWave);
            copy16(a.vcache + 2 * (off + 8 * (chunk ^ swz_v<D>(at))), lds + kStepBytes + first * 16 * kWave);
            // one bit per key of the copy, from the first lane of each key
            const uint64_t b = ballot(bad);
            uint32_t bits = 0;
#pragma unroll
            for (int k = 0; k < kKeysPerCopy; ++k) bits |= (uint32_t)((b >> (k * kLanesPerKey)) & 1) << k;
            if (lane == 0) bad_of[buf][first] = bits;
        }
    };

    f32x16 o[D / 32] = {};
    float top = kNegInf, total = 0.0f;  // total: this lane's half of the sum
    Places next;
    if (steps > 0) {
        next = load_entries(0);
        start_copies(next, 0);
        if (steps > 1) next = load_entries(1);
    }
    for (int s = 0; s < steps; ++s) {
        wait_copies();
        __syncthreads();
        if (s + 1 < steps) {
            start_copies(next, (s + 1) & 1);
            if (s + 2 < steps) next = load_entries(s + 2);
        }
        if (s * kTileKeys >= wave_most) continue;
        const uint8_t *kb = ring + (s & 1) * 2 * kStepBytes;
        f32x16 z[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) z[u] = score_tile<DT, D>(kb + u * kStepBytes / 2, q, lane);
        uint64_t bad = 0;
#pragma unroll
        for (int i = 0; i < kTileKeys / kKeysPerCopy; ++i)
            bad |= (uint64_t)bad_of[s & 1][i] << (i * kKeysPerCopy);
        if (bad) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    z[u][i] = (bad >> (32 * u + score_key(i, lane))) & 1 ? __builtin_nanf("") : z[u][i];
        }
        if ((s + 1) * kTileKeys > wave_least) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    z[u][i] = s * kTileKeys + 32 * u + score_key(i, lane) < ctx ? z[u][i] : kNegInf;
        }
        softmax_step(z, a.scale_log2, top, total, o);
#pragma unroll
        for (int u = 0; u < 2; ++u)
            output_tile<DT, D>(kb + kStepBytes + u * kStepBytes / 2, z[u], o, lane);
    }
    total = xor32_sum(total);

    // A NaN can come from a value that only other rows of the wave see (zero weight
    // times a value that is not finite): then the wave's pairs are done again, each
    // over its own keys.
    if (wave_least < wave_most) {
        bool nan = false;
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) nan |= o[c][i] != o[c][i];
        if (ballot(nan && live)) {
            own_pairs<DT, D>(launch_args(), w.req, w.row0, w.rows, wave, hk);
            return;
        }
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
            *reinterpret_cast<V4 *>(out + 32 * c + 8 * g + 4 * (lane >> 5)) = v;
        }
    if (a.lse && lane < kAttnTile)
        a.lse[(int64_t)row * (a.num_kv_heads * a.group) + head] = (top + __builtin_amdgcn_logf(total)) * kLn2;
}

template <int DT, int D>
hipError_t run_tile(const AttnArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((attn_tile_kernel<DT, D>), dim3((unsigned)a.slots, (unsigned)a.num_kv_heads),
                       dim3(kTileThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_tile(const AttnArgs &a, hipStream_t s) {
    if (a.dtype == kBF16) return a.head_dim == 128 ? run_tile<kBF16, 128>(a, s) : run_tile<kBF16, 64>(a, s);
    return a.head_dim == 128 ? run_tile<kFP16, 128>(a, s) : run_tile<kFP16, 64>(a, s);
}

}  // namespace qsa
