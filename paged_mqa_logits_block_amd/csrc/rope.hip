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
// and cosines of its rows once, into LDS, for all their heads.
#include "attn_internal.h"
#include "qsa_device.h"
#include "qsa_internal.h"
#include "step_internal.h"

namespace qsa {
namespace {

constexpr int kRopeThreads = 256;

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

// ROWS rows per workgroup, and every gridDim.y-th kRopeThreads lanes of their heads.
template <int DT, int D, bool HALF, int ROWS>
__global__ __launch_bounds__(kRopeThreads) void norm_rope_kernel(NormRopeArgs a) {
    constexpr int kLanes = D / 16;
    __shared__ float cosines[ROWS][D / 2], sines[ROWS][D / 2];
    __shared__ int64_t cache_at[ROWS];  // the row's place in the caches in elements, -1: none
    __shared__ int32_t live[ROWS];
    const int t = threadIdx.x, row0 = (int)blockIdx.x * ROWS, rows = min(ROWS, a.num_rows - row0);
    const int pairs = a.rot_dim / 2;
    for (int i = t; i < rows * pairs; i += kRopeThreads) {
        const int r = i / pairs, f = i - r * pairs;
        const int64_t pos = (int64_t)a.positions[row0 + r] + a.position_offset;
        const double turns = (double)pos * (a.inv_freq[f] * 0.15915494309189533577);
        float s, c;
        sincospif(2.0f * (float)(turns - __builtin_rint(turns)), &s, &c);
        cosines[r][f] = c * a.factor;
        sines[r][f] = s * a.factor;
    }
    if (t < rows) {
        live[t] = (int64_t)a.positions[row0 + t] + a.position_offset >= 0;
        int64_t at = -1;
        if (a.kcache) {
            const int64_t slot = a.slots[row0 + t];
            if (slot >= 0 && slot < a.num_blocks * a.block_size) {
                const int64_t blk = slot / a.block_size;
                at = blk * a.kv_block + (slot - blk * a.block_size) * a.kv_slot;
            }
        }
        cache_at[t] = at;
    }
    __syncthreads();

    // this lane's chunks, the same for every head
    const int l = t % kLanes, turned = a.rot_dim / 8, first = a.rot_offset / 8;
    const bool turns = l < turned / 2;
    int c0 = first + l, c1 = c0 + turned / 2;
    if (!turns) {
        c0 = 2 * l - turned;
        c1 = c0 + 1;
        if (c0 >= first) c0 += turned;
        if (c1 >= first) c1 += turned;
    }
    const int per_row = a.heads * kLanes, items = rows * per_row;
    for (int i = (int)blockIdx.y * kRopeThreads + t; i < items; i += (int)gridDim.y * kRopeThreads) {
        const int r = i / per_row, head = (i - r * per_row) / kLanes;
        const int64_t row = row0 + r;
        const bool is_q = head < a.num_heads, is_v = head >= a.num_heads + a.num_kv_heads;
        const int h = head - (is_q ? 0 : is_v ? a.num_heads + a.num_kv_heads : a.num_heads);
        const uint16_t *src = is_q ? a.q + row * a.q_row + h * a.q_head
                                   : is_v ? a.v + row * a.v_row + h * a.v_head : a.k + row * a.k_row + h * a.k_head;
        const i32x4 raw0 = *reinterpret_cast<const i32x4 *>(src + 8 * c0);
        const i32x4 raw1 = *reinterpret_cast<const i32x4 *>(src + 8 * c1);
        float x[8], y[8];
        unpack8<DT>(raw0, x);
        unpack8<DT>(raw1, y);
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += x[j] * x[j] + y[j] * y[j];
        sum = head_sum<kLanes>(sum);
        const float *w = is_q ? a.q_weight : is_v ? nullptr : a.k_weight;
        if (w) {
            const float inv = 1.0f / sqrtf(sum * (1.0f / D) + a.eps);
            const float *w0 = w + 8 * c0, *w1 = w + 8 * c1;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] *= inv * w0[j];
                y[j] *= inv * w1[j];
            }
        }
        if (turns && !is_v) {
            const float *c = cosines[r], *s = sines[r];
            if constexpr (HALF) {
#pragma unroll
                for (int j = 0; j < 8; ++j) turn_pair(x[j], y[j], c[8 * l + j], s[8 * l + j]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    turn_pair(x[2 * j], x[2 * j + 1], c[4 * l + j], s[4 * l + j]);
                    turn_pair(y[2 * j], y[2 * j + 1], c[4 * l + pairs / 2 + j], s[4 * l + pairs / 2 + j]);
                }
            }
        }
        if (!live[r]) continue;
        const i32x4 out0 = is_v ? raw0 : round8<DT>(x), out1 = is_v ? raw1 : round8<DT>(y);
        const auto store = [&](uint16_t *dst) {
            *reinterpret_cast<i32x4 *>(dst + 8 * c0) = out0;
            *reinterpret_cast<i32x4 *>(dst + 8 * c1) = out1;
        };
        if (is_q) {
            store(a.q_out + row * a.qo_row + h * a.qo_head);
        } else {
            if (!is_v && a.k_out) store(a.k_out + row * a.ko_row + h * a.ko_head);
            if (cache_at[r] >= 0) store((is_v ? a.vcache : a.kcache) + cache_at[r] + h * a.kv_head);
        }
    }
}

template <int DT, int D, bool HALF>
hipError_t run_rope(const NormRopeArgs &a, hipStream_t s) {
    const unsigned parts = (unsigned)((a.heads * (D / 16) + kRopeThreads - 1) / kRopeThreads);
    hipLaunchKernelGGL((norm_rope_kernel<DT, D, HALF, 1>), dim3((unsigned)a.num_rows, parts), dim3(kRopeThreads), 0, s, a);
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
