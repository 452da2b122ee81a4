// Host/device interface of the attention kernels (paged chunk attention and
// attention over selected tokens) and of the kernels that fill their inputs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qsa {

// Stacked (row, head) pairs of one wave's MFMA tile.
constexpr int kAttnTile = 32;
// Keys per step of a streaming wave, and waves per streaming workgroup.
constexpr int kStreamKeys = 32;
constexpr int kStreamWaves = 8;
// Workgroups that a cut launch aims at (one per CU), and the most row tiles of one.
constexpr int kStreamGroups = 256;
constexpr int kMaxSlots = 1024;

// Stacked pairs of a workgroup of the tile kernel.
constexpr int kTilePairs = 256;

struct AttnArgs {
    const void *q;
    const uint8_t *kcache;
    const uint8_t *vcache;
    const int32_t *block_table;
    const int32_t *ctx_lens;    // dense: visible keys per row; sparse: token limit per row, or null
    const int32_t *q_starts;    // dense: [num_reqs + 1]
    const int32_t *row_to_req;  // sparse
    const int32_t *idx;         // sparse: [num_rows][k]
    void *out;
    float *lse;                 // or null
    float *part;                // workspace of a cut launch, or null
    int32_t num_rows;
    int32_t num_kv_heads;
    int32_t group;              // query heads per kv head
    int32_t head_dim;
    int32_t block_size;
    int32_t num_reqs;
    int32_t max_blocks;
    int32_t cap;                // tokens a table row can hold
    int32_t k, ratio;           // sparse: selected columns per row, tokens per column
    int32_t dtype;
    float scale_log2;           // softmax scale * log2(e)
    int64_t num_blocks;
    int64_t q_row, q_head;      // strides in elements
    int64_t o_row, o_head;
    uint32_t kv_block, kv_slot, kv_head;  // strides in 16 bytes
    // tok / block_size = high word of (2 tok) div_mul, shifted right by div_shift: with
    // l = ceil(log2 block_size), div_shift = max(l - 1, 0) and
    // div_mul = ceil(2^(31 + div_shift) / block_size), exact for tok < 2^30
    uint32_t div_mul;
    int32_t div_shift;
    // launch shape
    int32_t slots;              // row tiles of the grid
    int32_t tiles;              // the most tiles with rows, of all head parts (a cut launch)
    int32_t sub_heads;          // query heads per workgroup of one kv head
    int32_t num_subs;           // workgroups per kv head
    int32_t tile_rows;          // query rows per tile
};

hipError_t launch_attn_stream(const AttnArgs &a, bool sparse, hipStream_t s);
// bytes of a cut launch's workspace, of the streaming and of the tile kernel
int64_t attn_workspace_bytes(int head_dim, int64_t tiles);
int64_t attn_tile_workspace_bytes(int head_dim, int64_t tiles);
hipError_t launch_attn_tile(const AttnArgs &a, hipStream_t s);

struct PlanArgs {
    const int32_t *past_lens, *new_lens, *free_blocks;
    int32_t *block_table, *q_starts, *row_to_req, *ctx_lens;
    int64_t *slots;
    int32_t *col_lens;
    int64_t *col_slots;
    int32_t *blocks_used;
    int32_t num_reqs, max_blocks, block_size, ratio, num_rows, num_free;
    int64_t num_blocks;
};

constexpr int kPlanMaxReqs = 4096;
hipError_t launch_plan(const PlanArgs &a, hipStream_t s);

struct WriteKvArgs {
    const uint8_t *k, *v;
    const int64_t *slots;
    uint8_t *kcache, *vcache;
    int32_t num_rows, num_kv_heads, head_dim, block_size;
    int64_t num_blocks;
    int64_t src_row, src_head;  // strides in elements
    int64_t kv_block, kv_slot, kv_head;
};

hipError_t launch_write_kv(const WriteKvArgs &a, hipStream_t s);

struct WriteKeysArgs {
    const uint8_t *src;
    const int64_t *slots;
    uint8_t *kcache;
    float *kscale;
    int32_t num_rows, head_dim, block_size, src_dtype, k_dtype, layout;
    int64_t num_blocks, src_stride, block_bytes;
};

hipError_t launch_write_keys(const WriteKeysArgs &a, hipStream_t s);

}  // namespace qsa
