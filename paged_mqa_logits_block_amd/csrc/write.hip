// Cache writes through a slot map: slot s is slot s % B of pool block s / B, and
// rows whose slot is negative or past the pool write nothing.
//
// write_kv copies 16-bit keys and values; both are bound by the bytes of the
// rows, read once and written once, 16 bytes per thread and step.
//
// write_keys stores the indexer's keys: 16-bit keys as they are, or as e4m3 with
// the f32 scale s = amax / 448 of each key (1 for a key of zeros, and for a
// paged cache that keeps no scales) and codes rne(x / s), the largest magnitude landing on the format's largest value.  A
// key is held by D / 8 lanes, 16 bytes of it each, so its maximum is a
// reduction over 8 or 16 neighbouring lanes and each lane packs 8 codes: the
// key is read once, and its codes and scale are written once.
//
// Measured (kernel traces): keys and values of 16,384 rows, 4 heads of 128 (67 MB moved):
// 12.8 us, 5.3 TB/s, where a library copy of as many bytes takes 10.7; 36 rows 2.7 us, a
// launch.  16,384 index keys: 16-bit 3.3 us, fp8 4.2 (5.1 where each call's inputs are
// not in the caches: 6.5 MB); 36 keys 1.9 and 2.4 us.

#include "attn_internal.h"
#include "qsa_device.h"
#include "qsa_internal.h"

namespace qsa {
namespace {

constexpr int kWriteThreads = 256;
typedef int i32x2_a4 __attribute__((ext_vector_type(2), aligned(4)));

__global__ __launch_bounds__(kWriteThreads) void write_kv_kernel(WriteKvArgs a) {
    const uint32_t per_head = (uint32_t)a.head_dim / 8, per_row = per_head * (uint32_t)a.num_kv_heads;
    const int64_t total = (int64_t)a.num_rows * per_row;
    const int64_t last = a.num_blocks * a.block_size;
    const uint8_t *src = blockIdx.y ? a.v : a.k;
    uint8_t *dst = blockIdx.y ? a.vcache : a.kcache;
    for (int64_t o = (int64_t)blockIdx.x * kWriteThreads + threadIdx.x; o < total;
         o += (int64_t)gridDim.x * kWriteThreads) {
        const int64_t r = o / per_row;
        const uint32_t in = (uint32_t)(o - r * per_row), h = in / per_head, c = in - h * per_head;
        const int64_t slot = a.slots[r];
        if (slot < 0 || slot >= last) continue;
        const int64_t blk = slot / a.block_size, pos = slot - blk * a.block_size;
        const i32x4 x = *reinterpret_cast<const i32x4 *>(src + 2 * (r * a.src_row + h * a.src_head + 8 * c));
        *reinterpret_cast<i32x4 *>(dst + 2 * (blk * a.kv_block + pos * a.kv_slot + h * a.kv_head + 8 * c)) = x;
    }
}

// max over the 16-lane row's lanes that differ in the low bits of the lane
// index only: 8 lanes (D = 64) or 16 (D = 128)
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
    v = fmaxf(v, xor_lane_f(v, 1));
    v = fmaxf(v, xor_lane_f(v, 2));
    v = fmaxf(v, xor_lane_f(v, 4));
    if constexpr (LANES == 16) v = fmaxf(v, xor_lane_f(v, 8));
    return v;
}

template <int D, int SRC, bool FP8>
__global__ __launch_bounds__(kWriteThreads) void write_keys_kernel(WriteKeysArgs a) {
    constexpr int kLanes = D / 8;
    const int c = threadIdx.x % kLanes;
    const int64_t r = (int64_t)blockIdx.x * (kWriteThreads / kLanes) + threadIdx.x / kLanes;
    const int64_t rr = r < a.num_rows ? r : a.num_rows - 1;  // whole waves reach the reduction
    const int64_t slot = a.slots[rr];
    const i32x4 x = *reinterpret_cast<const i32x4 *>(a.src + 2 * (rr * a.src_stride + 8 * c));
    const bool live = r < a.num_rows && slot >= 0 && slot < a.num_blocks * a.block_size;
    const int64_t blk = live ? slot / a.block_size : 0;
    const int pos = live ? (int)(slot - blk * a.block_size) : 0;
    uint8_t *block = a.kcache + blk * a.block_bytes;
    if constexpr (!FP8) {
        if (live) *reinterpret_cast<i32x4 *>(block + (int64_t)pos * 2 * D + 16 * c) = x;
    } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (SRC == kBF16) {
                f[2 * i] = __int_as_float(x[i] << 16);
                f[2 * i + 1] = __int_as_float(x[i] & 0xFFFF0000);
            } else {
                f[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)x[i]);
                f[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)((uint32_t)x[i] >> 16));
            }
        }
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
        top = lanes_max<kLanes>(top);
        // a paged cache without scales holds the values themselves, saturated
        const bool scaled = a.layout != 0 || a.kscale;
        const float scale = scaled && top > 0.0f ? top / 448.0f : 1.0f;
        int32_t code[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float v[4];
            // the quotient can pass 448 by a rounding: clamp before the conversion
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float u = f[4 * i + j] / scale;
                v[j] = u != u ? u : fminf(fmaxf(u, -448.0f), 448.0f);
            }
            int32_t p = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
            code[i] = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], p, true);
        }
        if (live) {
            const int64_t at = a.layout == 2 ? (int64_t)(pos >> 4) * 16 * D + (c >> 1) * 256 + (pos & 15) * 16 + 8 * (c & 1)
                                             : (int64_t)pos * D + 8 * c;
            // co-packed blocks of an odd number of keys start on 4-byte boundaries
            *reinterpret_cast<i32x2_a4 *>(block + at) = i32x2_a4{code[0], code[1]};
            if (c == 0) {
                float *sc = a.layout == 0 ? (scaled ? a.kscale + slot : nullptr)
                                          : reinterpret_cast<float *>(block + (int64_t)a.block_size * D) + pos;
                if (sc) *sc = scale;
            }
        }
    }
}

template <int D, int SRC, bool FP8>
hipError_t run_keys(const WriteKeysArgs &a, hipStream_t s) {
    const int rows = kWriteThreads / (D / 8);
    const unsigned groups = (unsigned)(((int64_t)a.num_rows + rows - 1) / rows);
    hipLaunchKernelGGL((write_keys_kernel<D, SRC, FP8>), dim3(groups), dim3(kWriteThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_write_kv(const WriteKvArgs &a, hipStream_t s) {
    const int64_t total = (int64_t)a.num_rows * a.num_kv_heads * (a.head_dim / 8);
    int64_t groups = (total + kWriteThreads - 1) / kWriteThreads;
    if (groups > 8192) groups = 8192;  // grid-stride beyond that
    hipLaunchKernelGGL(write_kv_kernel, dim3((unsigned)groups, 2), dim3(kWriteThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_write_keys(const WriteKeysArgs &a, hipStream_t s) {
    const bool fp8 = a.k_dtype == kFP8;
    if (!fp8) return a.head_dim == 128 ? run_keys<128, kBF16, false>(a, s) : run_keys<64, kBF16, false>(a, s);
    if (a.src_dtype == kBF16)
        return a.head_dim == 128 ? run_keys<128, kBF16, true>(a, s) : run_keys<64, kBF16, true>(a, s);
    return a.head_dim == 128 ? run_keys<128, kFP16, true>(a, s) : run_keys<64, kFP16, true>(a, s);
}

}  // namespace qsa
