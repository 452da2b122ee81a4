// Norms of query and key heads with their rotary positions, keys and values going
// straight into the paged caches:
//
//   y = x w / sqrt(mean(x^2) + eps)                      (heads with a weight)
//   (a, b) -> factor (a cos t - b sin t, b cos t + a sin t),  t = position inv_freq[i]
//
// over the pairs i of a head's rotated part, in 32 bits from the loaded values to the
// one rounding at the end.
//
// A lane holds 16 elements of a head: two chunks of 8 that lie half the rotated part
// apart, so that both elements of a pair are in it in either layout; the elements that
// are not rotated are dealt to the lanes behind.  A head is D / 16 lanes, and its mean
// square a sum over these.
//
// Angles: t in turns is position * (inv_freq / 2 pi) in 64 bits, less the nearest whole
// number, which is then rounded to 32 (a product in 32 bits would be off by 2^-24 of
// the whole angle, 0.06 rad at a position of one million).  A workgroup takes the sines
// and cosines of its row once, into LDS, for all heads.
//
// What bounds it is the bytes, read once and written once.  Measured: 16,384 rows of 32
// query, 4 key and 4 value heads at D = 128 (335 MB) 56 us, 6.0 TB/s, where a library copy
// that moves 539 MB reaches 5.3; 79 us with workgroups of 256 lanes for a row's 320, 84 to 98
// with a wave per row that keeps angles and weights in 135 registers (3 waves to a SIMD
// have too few loads on their way).  One row 2.6 us in the trace, where an empty kernel
// takes 1.9: the position, its angle and the store follow one another.
#include "attn_internal.h"
#include "qsa_device.h"
#include "qsa_internal.h"
#include "step_internal.h"

namespace qsa {
namespace {

constexpr int kRopeThreads = 1024;  // the most of a workgroup

template <int DT>
__device__ __forceinline__ float half_to_f32(uint32_t u) {
    if constexpr (DT == kBF16) return __uint_as_float(u << 16);
    else return (float)__builtin_bit_cast(_Float16, (uint16_t)u);
}

template <int DT>
__device__ __forceinline__ void unpack8(i32x4 v, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = (uint32_t)v[i];
        x[2 * i] = half_to_f32<DT>(u & 0xFFFF);
        x[2 * i + 1] = half_to_f32<DT>(u >> 16);
    }
}

template <int DT>
__device__ __forceinline__ i32x4 round8(const float (&x)[8]) {
    if constexpr (DT == kBF16) {
        bf16x8 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (__bf16)x[j];
        return __builtin_bit_cast(i32x4, v);
    } else {
        typedef _Float16 h8 __attribute__((ext_vector_type(8)));
        h8 v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (_Float16)x[j];
        return __builtin_bit_cast(i32x4, v);
    }
}

// sum over the 8 or 4 neighbouring lanes of a head
template <int LANES>
__device__ __forceinline__ float head_sum(float v) {
    v += __uint_as_float(dpp_u32<kDppXor1>(__float_as_uint(v)));
    v += __uint_as_float(dpp_u32<kDppXor2>(__float_as_uint(v)));
    if constexpr (LANES == 8) v += __uint_as_float(dpp_u32<kDppHalfMirror>(__float_as_uint(v)));
    return v;
}

// (a, b) turned by the angle of (cos, sin)
__device__ __forceinline__ void turn_pair(float &a, float &b, float c, float s) {
    const float x = a * c - b * s;
    b = b * c + a * s;
    a = x;
}

// a row's position, and the sine and cosine of pair f there
__device__ __forceinline__ int64_t position_of(const NormRopeArgs &a, int64_t row) {
    return (int64_t)a.positions[row] + a.position_offset;
}
__device__ __forceinline__ void turn_of(const NormRopeArgs &a, int64_t pos, int f, float &c, float &s) {
    const double turns = (double)pos * (a.inv_freq[f] * 0.15915494309189533577);
    sincospif(2.0f * (float)(turns - __builtin_rint(turns)), &s, &c);
    c *= a.factor;
    s *= a.factor;
}
// a row's place in the caches in elements, -1: none
__device__ __forceinline__ int64_t place_of(const NormRopeArgs &a, int64_t row) {
    if (!a.kcache) return -1;
    const int64_t slot = a.slots[row];
    if (slot < 0 || slot >= a.num_blocks * a.block_size) return -1;
    const int64_t blk = slot / a.block_size;
    return blk * a.kv_block + (slot - blk * a.block_size) * a.kv_slot;
}

// A lane's two chunks, the same for every head.
struct Chunks {
    int c0, c1;
    bool turns;
};
__device__ __forceinline__ Chunks chunks_of(const NormRopeArgs &a, int l) {
    const int turned = a.rot_dim / 8, first = a.rot_offset / 8;
    Chunks k = {first + l, first + l + turned / 2, l < turned / 2};
    if (!k.turns) {
        k.c0 = 2 * l - turned;
        k.c1 = k.c0 + 1;
        if (k.c0 >= first) k.c0 += turned;
        if (k.c1 >= first) k.c1 += turned;
    }
    return k;
}

// The head of a row that a lane works on: query heads, then key heads, then value heads.
struct Head {
    int h;
    bool is_q, is_v;
};
__device__ __forceinline__ Head head_of(const NormRopeArgs &a, int head) {
    Head x = {head, head < a.num_heads, head >= a.num_heads + a.num_kv_heads};
    x.h -= x.is_q ? 0 : x.is_v ? a.num_heads + a.num_kv_heads : a.num_heads;
    return x;
}
__device__ __forceinline__ const uint16_t *source_of(const NormRopeArgs &a, int64_t row, const Head &x) {
    return x.is_q ? a.q + row * a.q_row + x.h * a.q_head
                  : x.is_v ? a.v + row * a.v_row + x.h * a.v_head : a.k + row * a.k_row + x.h * a.k_head;
}

// the norm of a head of which this lane has the chunks x and y, with their weights w
template <int D>
__device__ __forceinline__ void norm_chunks(float (&x)[8], float (&y)[8], const float (&w)[16], float eps) {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += x[j] * x[j] + y[j] * y[j];
    const float inv = 1.0f / sqrtf(head_sum<D / 16>(sum) * (1.0f / D) + eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        x[j] *= inv * w[j];
        y[j] *= inv * w[8 + j];
    }
}
// the rotation by cosines c and sines s of their pairs: those that x and y make, or
// interleaved x's four, then y's
template <bool HALF>
__device__ __forceinline__ void turn_chunks(float (&x)[8], float (&y)[8], const float (&c)[8], const float (&s)[8]) {
    if constexpr (HALF) {
#pragma unroll
        for (int j = 0; j < 8; ++j) turn_pair(x[j], y[j], c[j], s[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            turn_pair(x[2 * j], x[2 * j + 1], c[j], s[j]);
            turn_pair(y[2 * j], y[2 * j + 1], c[4 + j], s[4 + j]);
        }
    }
}
template <bool ONCE>
__device__ __forceinline__ i32x4 load_chunk(const uint16_t *p) {
    if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const i32x4 *>(p));
    else return *reinterpret_cast<const i32x4 *>(p);
}
template <bool ONCE>
__device__ __forceinline__ void store_chunks(uint16_t *dst, const Chunks &k, i32x4 a, i32x4 b) {
    i32x4 *p0 = reinterpret_cast<i32x4 *>(dst + 8 * k.c0), *p1 = reinterpret_cast<i32x4 *>(dst + 8 * k.c1);
    if constexpr (ONCE) {
        __builtin_nontemporal_store(a, p0);
        __builtin_nontemporal_store(b, p1);
    } else {
        *p0 = a;
        *p1 = b;
    }
}

// A workgroup per row, with a lane for each two chunks of its heads (or of a part of them).
// ONCE: rows that pass through the caches without staying there.
template <int DT, int D, bool HALF, bool ONCE>
__global__ __launch_bounds__(kRopeThreads) void norm_rope_kernel(NormRopeArgs a) {
    constexpr int kLanes = D / 16;
    __shared__ float cosines[D / 2], sines[D / 2];
    const int t = threadIdx.x, pairs = a.rot_dim / 2, l = t % kLanes;
    const int64_t row = blockIdx.x;
    const int head = ((int)blockIdx.y * (int)blockDim.x + t) / kLanes;
    const bool have = head < a.heads;
    const Head x = head_of(a, have ? head : 0);
    const Chunks k = chunks_of(a, l);
    // all loads on their way before the angles
    const uint16_t *src = source_of(a, row, x);
    const i32x4 raw0 = load_chunk<ONCE>(src + 8 * k.c0), raw1 = load_chunk<ONCE>(src + 8 * k.c1);
    const float *weight = x.is_q ? a.q_weight : x.is_v ? nullptr : a.k_weight;
    float w[16];
    if (weight) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = weight[8 * k.c0 + j];
            w[8 + j] = weight[8 * k.c1 + j];
        }
    }
    const int64_t at = place_of(a, row), pos = position_of(a, row);
    for (int f = t; f < pairs; f += (int)blockDim.x) turn_of(a, pos, f, cosines[f], sines[f]);
    __syncthreads();
    if (pos < 0 || !have) return;
    float u[8], v[8];
    unpack8<DT>(raw0, u);
    unpack8<DT>(raw1, v);
    if (weight) norm_chunks<D>(u, v, w, a.eps);
    if (k.turns && !x.is_v) {
        float c[8], s[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int f = HALF ? 8 * l + j : j < 4 ? 4 * l + j : pairs / 2 + 4 * l + j - 4;
            c[j] = cosines[f];
            s[j] = sines[f];
        }
        turn_chunks<HALF>(u, v, c, s);
    }
    const i32x4 out0 = x.is_v ? raw0 : round8<DT>(u), out1 = x.is_v ? raw1 : round8<DT>(v);
    if (x.is_q) {
        store_chunks<ONCE>(a.q_out + row * a.qo_row + x.h * a.qo_head, k, out0, out1);
        return;
    }
    if (!x.is_v && a.k_out) store_chunks<ONCE>(a.k_out + row * a.ko_row + x.h * a.ko_head, k, out0, out1);
    if (at >= 0) store_chunks<ONCE>((x.is_v ? a.vcache : a.kcache) + at + x.h * a.kv_head, k, out0, out1);
}

// Bytes read and written from which they are streamed: more than the 8 L2s hold (4 MB each).
// 16,384 rows of 32 + 4 heads and their values (335 MB) 62 us plain, 56 streamed (loads or
// stores alone: 67 and 61); 1,001 rows (4 MB) 4.3 and 4.4.
constexpr int64_t kOnceBytes = 32 << 20;

template <int DT, int D, bool HALF>
hipError_t run_rope(const NormRopeArgs &a, hipStream_t s) {
    const int lanes = a.heads * (D / 16), parts = (lanes + kRopeThreads - 1) / kRopeThreads;
    const int threads = ((lanes + parts - 1) / parts + kWave - 1) / kWave * kWave;
    const dim3 grid((unsigned)a.num_rows, (unsigned)parts), block((unsigned)threads);
    if ((int64_t)a.num_rows * a.heads * D * 4 > kOnceBytes)
        hipLaunchKernelGGL((norm_rope_kernel<DT, D, HALF, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((norm_rope_kernel<DT, D, HALF, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <int DT>
hipError_t run_dim(const NormRopeArgs &a, hipStream_t s) {
    if (a.head_dim == 128) return a.layout == 0 ? run_rope<DT, 128, true>(a, s) : run_rope<DT, 128, false>(a, s);
    return a.layout == 0 ? run_rope<DT, 64, true>(a, s) : run_rope<DT, 64, false>(a, s);
}

}  // namespace

hipError_t launch_norm_rope(const NormRopeArgs &a, hipStream_t s) {
    return a.dtype == kBF16 ? run_dim<kBF16>(a, s) : run_dim<kFP16>(a, s);
}

}  // namespace qsa
