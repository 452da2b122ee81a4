// Host/device interface of the kernels at the two ends of a serving step: head
// norms with rotary positions, and the verification of drafted tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qsa {

struct NormRopeArgs {
    const uint16_t *q, *k, *v;         // null: no such heads
    const float *q_weight, *k_weight;  // null: no norm
    const int32_t *positions;
    const double *inv_freq;            // [rot_dim / 2]
    const int64_t *slots;              // with kcache
    uint16_t *q_out, *k_out, *kcache, *vcache;
    int32_t num_rows, num_heads, num_kv_heads, head_dim, rot_dim, rot_offset, layout, dtype, position_offset, block_size;
    float eps, factor;
    int64_t num_blocks;
    // strides in elements
    int64_t q_row, q_head, k_row, k_head, v_row, v_head, qo_row, qo_head, ko_row, ko_head;
    int64_t kv_block, kv_slot, kv_head;
    // launch shape
    int32_t heads;       // of a row: query heads, key heads, value heads
};

hipError_t launch_norm_rope(const NormRopeArgs &a, hipStream_t s);

// Vocabulary entries whose weights one wave adds up.
constexpr int kVerifySpan = 2048;
constexpr int kVerifyMaxVocab = 1 << 20;

struct VerifyArgs {
    const float *probs, *draft_probs;  // draft_probs null: each draft was certain
    const int32_t *tokens, *q_starts;
    const float *uniforms, *sample_uniforms;
    int32_t *out_tokens, *num_tokens;
    double *part;                      // workspace of a split launch, or null
    int32_t num_rows, num_reqs, vocab, max_tokens, spans;
    int64_t prob_row, draft_row;
};

hipError_t launch_verify(const VerifyArgs &a, hipStream_t s);
// bytes of a split launch's workspace
int64_t verify_workspace_bytes(int64_t num_reqs, int64_t spans);

}  // namespace qsa
