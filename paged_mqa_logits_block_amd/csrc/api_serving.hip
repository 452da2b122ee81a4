// C-ABI entry points around the scorer: the batch plan, the cache writes, and
// attention over the paged cache (all visible tokens, or the selected ones).
// As in api.hip, validation reads host scalars only and every call can be
// captured.
#include "api_common.h"
#include "attn_internal.h"
#include "qsa_internal.h"
#include "qsaidx.h"

namespace {

using qsa::aligned16;
using qsa::fail;
using qsa::ok;

qsa_status launched(hipError_t e) {
    return e == hipSuccess ? ok() : fail(QSA_E_HIP, "launch failed: %s", hipGetErrorString(e));
}

qsa_status check_plan(const int32_t *past_lens, const int32_t *new_lens, const int32_t *free_blocks,
                      const int32_t *block_table, const int32_t *q_starts, const int32_t *row_to_req,
                      const int32_t *ctx_lens, const int64_t *slots, const qsa_plan_shape *s) {
    if (!s) return fail(QSA_E_INVALID, "shape is NULL");
    if (s->num_rows < 0 || s->num_free < 0)
        return fail(QSA_E_INVALID, "num_rows = %d and num_free = %d must be >= 0", s->num_rows, s->num_free);
    if (s->num_reqs < 1 || s->max_blocks < 1 || s->block_size < 1 || s->num_blocks < 1 || s->ratio < 1)
        return fail(QSA_E_INVALID, "num_reqs, max_blocks, block_size, num_blocks and ratio must be >= 1");
    if (s->block_size % s->ratio != 0)
        return fail(QSA_E_INVALID, "ratio = %d does not divide block_size = %d", s->ratio, s->block_size);
    if (!past_lens || !new_lens || !block_table || !q_starts || (s->num_free > 0 && !free_blocks) ||
        (s->num_rows > 0 && (!row_to_req || !ctx_lens || !slots)))
        return fail(QSA_E_INVALID, "past_lens, new_lens, free_blocks, block_table, q_starts, row_to_req, ctx_lens "
                                   "and slots must be non-NULL");
    if (s->num_reqs > qsa::kPlanMaxReqs)
        return fail(QSA_E_UNSUPPORTED, "num_reqs = %d (built: up to %d)", s->num_reqs, qsa::kPlanMaxReqs);
    if ((int64_t)s->max_blocks * s->block_size > (1 << 30))
        return fail(QSA_E_RANGE, "max_blocks * block_size = %lld > 2^30", (long long)s->max_blocks * s->block_size);
    if (s->num_rows > (1 << 30)) return fail(QSA_E_RANGE, "num_rows = %d > 2^30", s->num_rows);
    if (s->num_blocks > ((int64_t)1 << 50)) return fail(QSA_E_RANGE, "num_blocks too large");
    return ok();
}

qsa_status check_write_kv(const void *k, const void *v, const int64_t *slots, const void *kcache, const void *vcache,
                          const qsa_kv_shape *s) {
    if (!s) return fail(QSA_E_INVALID, "shape is NULL");
    if (s->num_rows < 0) return fail(QSA_E_INVALID, "num_rows = %d < 0", s->num_rows);
    if (s->num_kv_heads < 1 || s->head_dim < 1 || s->block_size < 1 || s->num_blocks < 1)
        return fail(QSA_E_INVALID, "num_kv_heads, head_dim, block_size and num_blocks must be >= 1");
    if (s->src_row_stride < 0 || s->src_head_stride < 0 || s->kv_block_stride < 0 || s->kv_slot_stride < 0 ||
        s->kv_head_stride < 0)
        return fail(QSA_E_INVALID, "strides must be >= 0");
    if (s->num_rows > 0 && (!k || !v || !slots || !kcache || !vcache))
        return fail(QSA_E_INVALID, "k, v, slots, kcache and vcache must be non-NULL");
    if (s->dtype != QSA_BF16 && s->dtype != QSA_FP16) return fail(QSA_E_DTYPE, "dtype = %d (built: bf16, fp16)", s->dtype);
    if (s->head_dim != 64 && s->head_dim != 128)
        return fail(QSA_E_UNSUPPORTED, "head_dim = %d (built: 64, 128)", s->head_dim);
    if (s->block_size > 1024) return fail(QSA_E_UNSUPPORTED, "block_size = %d (built: 1 to 1024)", s->block_size);
    if (s->num_kv_heads > 1024) return fail(QSA_E_UNSUPPORTED, "num_kv_heads = %d (built: 1 to 1024)", s->num_kv_heads);
    if (s->kv_head_stride < (s->num_kv_heads > 1 ? s->head_dim : 0) ||
        s->kv_slot_stride < (s->block_size > 1 ? s->head_dim : 0) ||
        s->kv_block_stride < (s->num_blocks > 1 ? s->head_dim : 0))
        return fail(QSA_E_INVALID, "cache strides must be at least head_dim");
    if (s->num_blocks > ((int64_t)1 << 50) || s->kv_block_stride > ((int64_t)1 << 50) / s->num_blocks ||
        s->kv_slot_stride > ((int64_t)1 << 40) || s->kv_head_stride > ((int64_t)1 << 40) ||
        s->src_row_stride > ((int64_t)1 << 30) || s->src_head_stride > ((int64_t)1 << 30))
        return fail(QSA_E_RANGE, "cache or source too large");
    if (s->num_rows > 0 && (!aligned16(k) || !aligned16(v) || !aligned16(kcache) || !aligned16(vcache)))
        return fail(QSA_E_ALIGN, "k, v, kcache and vcache must be 16-byte aligned");
    if (s->num_rows > 0 && ((s->src_row_stride | s->src_head_stride | s->kv_block_stride | s->kv_slot_stride |
                             s->kv_head_stride) & 7) != 0)
        return fail(QSA_E_ALIGN, "strides must be multiples of 8 elements");
    return ok();
}

qsa_status check_write_keys(const void *keys, const int64_t *slots, const void *kcache, const float *kscale,
                            const qsa_keys_shape *s) {
    if (!s) return fail(QSA_E_INVALID, "shape is NULL");
    if (s->num_rows < 0) return fail(QSA_E_INVALID, "num_rows = %d < 0", s->num_rows);
    if (s->head_dim < 1 || s->block_size < 1 || s->num_blocks < 1)
        return fail(QSA_E_INVALID, "head_dim, block_size and num_blocks must be >= 1");
    if (s->src_stride < s->head_dim && s->num_rows > 1)
        return fail(QSA_E_INVALID, "src_stride = %lld < head_dim = %d", (long long)s->src_stride, s->head_dim);
    if (s->num_rows > 0 && (!keys || !slots || !kcache))
        return fail(QSA_E_INVALID, "keys, slots and kcache must be non-NULL");
    if (s->src_dtype != QSA_BF16 && s->src_dtype != QSA_FP16)
        return fail(QSA_E_DTYPE, "src_dtype = %d (built: bf16, fp16)", s->src_dtype);
    if (s->k_dtype != QSA_FP8_E4M3FN && s->k_dtype != s->src_dtype)
        return fail(QSA_E_DTYPE, "k_dtype = %d: e4m3 or the source's type", s->k_dtype);
    if (s->kv_layout < QSA_KV_PAGED || s->kv_layout > QSA_KV_COPACKED_SHUFFLED)
        return fail(QSA_E_INVALID, "kv_layout = %d", s->kv_layout);
    const bool fp8 = s->k_dtype == QSA_FP8_E4M3FN, copacked = s->kv_layout != QSA_KV_PAGED;
    if (copacked && !fp8) return fail(QSA_E_UNSUPPORTED, "co-packed layouts hold fp8 keys only");
    if (kscale && (!fp8 || copacked))
        return fail(QSA_E_INVALID, "kscale applies to fp8 keys in the paged layout only");
    if (s->head_dim != 64 && s->head_dim != 128)
        return fail(QSA_E_UNSUPPORTED, "head_dim = %d (built: 64, 128)", s->head_dim);
    if (s->block_size > 1024) return fail(QSA_E_UNSUPPORTED, "block_size = %d (built: 1 to 1024)", s->block_size);
    if (s->kv_layout == QSA_KV_COPACKED_SHUFFLED && s->block_size % 16 != 0)
        return fail(QSA_E_UNSUPPORTED, "the preshuffled layout needs block_size %% 16 == 0");
    if (s->num_rows > (1 << 27)) return fail(QSA_E_RANGE, "num_rows = %d > 2^27", s->num_rows);
    if (s->num_blocks > ((int64_t)1 << 40) || s->src_stride > ((int64_t)1 << 30))
        return fail(QSA_E_RANGE, "cache or source too large");
    if (s->num_rows > 0 && (!aligned16(keys) || !aligned16(kcache)))
        return fail(QSA_E_ALIGN, "keys and kcache must be 16-byte aligned");
    if (s->num_rows > 1 && s->src_stride % 8 != 0)
        return fail(QSA_E_ALIGN, "src_stride must be a multiple of 8 elements");
    return ok();
}

// Calls with up to this many stacked pairs per kv head and request on average are
// streamed, small ones at least (the lengths are on the device).  One request, 4 kv
// heads of 8 query heads at D = 128, us streamed / by the tile kernel: 16 rows of
// 2,048 tokens 14.9 / 19.5, of 16,384 22.1 / 26.6, of 65,536 48.8 / 43.5; 12 rows
// 14.7 / 18.3, 31.2 / 25.2, 70.3 / 39.7; 8 rows 14.3 / 17.1, 20.8 / 24.0, 38.0 /
// 38.0.
constexpr int kStreamPairs = 64, kSmallPairs = 512;
// Tiles up to which tiles of uneven length are cut, and the rows up to which the
// workgroups find their parts (each reads every row's visible count).  (1,024 decode
// tiles of 1,000 to 4,000 tokens: 222 us cut, 212 whole; 256 of 8,000 to 16,000 run
// at 5.6 TB/s cut, where whole ones wait for the longest.)
constexpr int kCutTiles = 1024, kCutRows = 8192;

// Tiles of one length are cut only where whole ones would leave more than 15% of
// the CUs' time unused.  (Selected tokens of 1,024 tiles: 97 us cut, 78 whole; 256
// tiles of a 2,048-row chunk 555 + 28 cut, 515 whole; 104 uneven tiles of 17
// requests 39 + 8 cut, 92 whole.)
bool fills_badly(int64_t tiles) {
    const int64_t rounds = (tiles + qsa::kStreamGroups - 1) / qsa::kStreamGroups;
    return tiles * 100 < rounds * qsa::kStreamGroups * 85;
}

struct AttnPlan {
    bool stream;               // streaming kernel, else the tile kernel
    int sub_heads, num_subs;   // streaming: heads per workgroup, workgroups per kv head
    int tile_rows;             // query rows per tile
    int64_t slots;             // row tiles
    int64_t tiles;             // a cut launch of the streaming kernel: the most tiles with rows
    int64_t bytes;             // workspace of a cut launch, 0: not cut
};

AttnPlan plan_attn(const qsa_attn_shape *s, bool sparse, int64_t keys) {
    AttnPlan p = {};
    const int group = s->num_heads / s->num_kv_heads;
    const int64_t R = s->num_rows, n = s->num_reqs;
    p.num_subs = (group + qsa::kAttnTile - 1) / qsa::kAttnTile;
    p.sub_heads = (group + p.num_subs - 1) / p.num_subs;
    p.num_subs = (group + p.sub_heads - 1) / p.sub_heads;
    const int64_t heads = (int64_t)s->num_kv_heads * p.num_subs;
    const bool long_keys = keys > qsa::kStreamKeys * qsa::kStreamWaves;
    if (sparse) {
        p.stream = true;
        p.tile_rows = 1;
        p.slots = R;
        p.tiles = R * heads;
        if (R <= qsa::kMaxSlots && R * heads <= kCutTiles && fills_badly(R * heads) && long_keys)
            p.bytes = qsa::attn_workspace_bytes(s->head_dim, p.tiles);
        return p;
    }
    // With at most four rows per request on average (a verify step), what one long
    // request adds to a batch streamed whole stays below the others' part.  us streamed
    // / by the tile kernel, 4 kv heads of 8 heads at D = 128: 64 requests of 4 rows,
    // 8,000 to 16,000 tokens 279 / 323; 63 requests of one row and one of 32, 64, 192,
    // 8,000 tokens each 209 / 200, 221 / 324, 280 / 313; 199 and one of 100, 300, 600,
    // 4,000 tokens 315 / 363, 353 / 355, 393 / 356; 7 and one of 8, 24, 8,000 tokens
    // 34 / 32, 44 / 39.  2 of 16 at D = 64: 63 and one of 32, 192, 8,000 tokens 58 / 121,
    // 83 / 122; 64 of 4 rows 89 / 72.  1 of 32: 63 and one of 96, 8,000 tokens 78 / 77.
    // The lengths, which decide it, are on the device: over 130 such batches the choice
    // costs at most 27% (8 requests of 4 rows, 1 of 32: 21 / 27).
    const int64_t few = group >= kStreamPairs ? 1 : kStreamPairs / group;
    p.stream = R <= few * n && (R <= 4 * n || R * group <= kSmallPairs);
    const int64_t T = p.tile_rows = p.stream ? qsa::kAttnTile / p.sub_heads : qsa::kTilePairs / group;
    p.slots = R / T + n;
    const int64_t tile_heads = p.stream ? heads : s->num_kv_heads;
    // tiles with rows: as many as requests or as full tiles, or some more
    const int64_t least = n < R ? n : R, full = (R + T - 1) / T, tiles = (full > least ? full : least) * tile_heads;
    if (p.slots > qsa::kMaxSlots || n > qsa::kMaxSlots || R > kCutRows || tiles > kCutTiles) return p;
    // the workgroups add up the slots' steps of 64 keys in 32 bits
    if (p.slots * (keys / 64 + 1) > 0x7FFFFFFF) return p;
    p.tiles = (R / T + least) * heads;
    if (p.stream && long_keys) p.bytes = qsa::attn_workspace_bytes(s->head_dim, p.tiles);
    if (!p.stream && (n > 1 || fills_badly(tiles)))
        p.bytes = qsa::attn_tile_workspace_bytes(s->head_dim, p.slots * s->num_kv_heads);
    return p;
}

// the sizes that plan_attn and the launches take
qsa_status check_attn_sizes(const qsa_attn_shape *s, bool sparse, int32_t k, int32_t ratio) {
    if (!s) return fail(QSA_E_INVALID, "shape is NULL");
    if (s->num_rows < 0) return fail(QSA_E_INVALID, "num_rows = %d < 0", s->num_rows);
    if (s->num_heads < 1 || s->num_kv_heads < 1 || s->head_dim < 1 || s->block_size < 1 || s->num_reqs < 1 ||
        s->max_blocks < 1 || s->num_blocks < 1)
        return fail(QSA_E_INVALID, "num_heads, num_kv_heads, head_dim, block_size, num_reqs, max_blocks and "
                                   "num_blocks must be >= 1");
    if (s->num_heads % s->num_kv_heads != 0)
        return fail(QSA_E_INVALID, "num_heads = %d is not a multiple of num_kv_heads = %d", s->num_heads, s->num_kv_heads);
    if (sparse) {
        if (k < 1) return fail(QSA_E_INVALID, "k = %d < 1", k);
        if (ratio < 1) return fail(QSA_E_INVALID, "ratio = %d < 1", ratio);
    }
    if (s->head_dim != 64 && s->head_dim != 128)
        return fail(QSA_E_UNSUPPORTED, "head_dim = %d (built: 64, 128)", s->head_dim);
    if (s->block_size > 1024) return fail(QSA_E_UNSUPPORTED, "block_size = %d (built: 1 to 1024)", s->block_size);
    const int group = s->num_heads / s->num_kv_heads;
    if (group > 128) return fail(QSA_E_UNSUPPORTED, "%d heads per kv head (built: 1 to 128)", group);
    if (s->num_heads > 8192) return fail(QSA_E_UNSUPPORTED, "num_heads = %d (built: up to 8192)", s->num_heads);
    if (s->num_rows > (1 << 21) || s->num_reqs > (1 << 21))
        return fail(QSA_E_RANGE, "num_rows = %d or num_reqs = %d > 2^21", s->num_rows, s->num_reqs);
    if ((int64_t)s->max_blocks * s->block_size > (1 << 30))
        return fail(QSA_E_RANGE, "max_blocks * block_size = %lld > 2^30", (long long)s->max_blocks * s->block_size);
    if (sparse && (int64_t)k * ratio > (1 << 24))
        return fail(QSA_E_RANGE, "k * ratio = %lld > 2^24", (long long)k * ratio);
    // workgroups of the tile kernel
    const int64_t tiles = ((int64_t)s->num_rows / (qsa::kTilePairs / group) + s->num_reqs) * s->num_kv_heads;
    if (!sparse && tiles > (1 << 22))
        return fail(QSA_E_RANGE, "too many tiles (%lld > 2^22) of rows, requests and kv heads", (long long)tiles);
    return ok();
}

qsa_status check_attn(const void *q, const void *kcache, const void *vcache, const int32_t *block_table,
                      const int32_t *per_row, const int32_t *starts_or_idx, const void *out,
                      const qsa_attn_shape *s, bool sparse, int32_t k, int32_t ratio) {
    qsa_status st = check_attn_sizes(s, sparse, k, ratio);
    if (st != QSA_OK) return st;
    // the kernels work with scale * log2(e)
    if (!(s->scale > 0.0f) || s->scale > 1e38f) return fail(QSA_E_INVALID, "scale must be in (0, 1e38]");
    if (s->q_row_stride < 0 || s->q_head_stride < 0 || s->out_row_stride < 0 || s->out_head_stride < 0 ||
        s->kv_block_stride < 0 || s->kv_slot_stride < 0 || s->kv_head_stride < 0)
        return fail(QSA_E_INVALID, "strides must be >= 0");
    if ((s->num_rows > 1 && s->out_row_stride < s->head_dim) || (s->num_heads > 1 && s->out_head_stride < s->head_dim))
        return fail(QSA_E_INVALID, "the strides of out must be at least head_dim");
    if (s->num_rows > 0 && (!q || !kcache || !vcache || !block_table || !per_row || !starts_or_idx || !out))
        return fail(QSA_E_INVALID, "q, kcache, vcache, block_table, %s and out must be non-NULL",
                    sparse ? "row_to_req, idx" : "ctx_lens, q_starts");
    if (s->dtype != QSA_BF16 && s->dtype != QSA_FP16) return fail(QSA_E_DTYPE, "dtype = %d (built: bf16, fp16)", s->dtype);
    const int64_t most = (int64_t)1 << 34;
    if (s->num_blocks > ((int64_t)1 << 50) || s->kv_block_stride > ((int64_t)1 << 50) / s->num_blocks ||
        s->kv_block_stride > most || s->kv_slot_stride > most || s->kv_head_stride > most || s->q_row_stride > most || s->q_head_stride > most ||
        s->out_row_stride > most || s->out_head_stride > most)
        return fail(QSA_E_RANGE, "a stride or the cache is too large");
    if (s->num_rows > 0 && (!aligned16(q) || !aligned16(kcache) || !aligned16(vcache) || !aligned16(out)))
        return fail(QSA_E_ALIGN, "q, kcache, vcache and out must be 16-byte aligned");
    if (s->num_rows > 0 && ((s->q_row_stride | s->q_head_stride | s->out_row_stride | s->out_head_stride |
                             s->kv_block_stride | s->kv_slot_stride | s->kv_head_stride) & 7) != 0)
        return fail(QSA_E_ALIGN, "strides must be multiples of 8 elements");
    return ok();
}

qsa_status check_workspace(const void *workspace, int64_t bytes, int64_t need) {
    if (!workspace) return ok();
    if (bytes < need)
        return fail(QSA_E_INVALID, "workspace_bytes = %lld < %lld", (long long)bytes, (long long)need);
    if (need > 0 && !aligned16(workspace)) return fail(QSA_E_ALIGN, "workspace must be 16-byte aligned");
    return ok();
}

qsa::AttnArgs attn_args(const void *q, const void *kcache, const void *vcache, const int32_t *block_table, void *out,
                        float *lse, const qsa_attn_shape *s) {
    qsa::AttnArgs a = {};
    a.q = q;
    a.kcache = static_cast<const uint8_t *>(kcache);
    a.vcache = static_cast<const uint8_t *>(vcache);
    a.block_table = block_table;
    a.out = out;
    a.lse = lse;
    a.num_rows = s->num_rows;
    a.num_kv_heads = s->num_kv_heads;
    a.group = s->num_heads / s->num_kv_heads;
    a.head_dim = s->head_dim;
    a.block_size = s->block_size;
    a.num_reqs = s->num_reqs;
    a.max_blocks = s->max_blocks;
    a.cap = s->max_blocks * s->block_size;
    a.dtype = s->dtype;
    a.scale_log2 = s->scale * 1.44269504088896340736f;
    a.num_blocks = s->num_blocks;
    a.q_row = s->q_row_stride;
    a.q_head = s->q_head_stride;
    a.o_row = s->out_row_stride;
    a.o_head = s->out_head_stride;
    a.kv_block = (uint32_t)(s->kv_block_stride / 8);
    a.kv_slot = (uint32_t)(s->kv_slot_stride / 8);
    a.kv_head = (uint32_t)(s->kv_head_stride / 8);
    int bits = 0;
    while ((1 << bits) < s->block_size) ++bits;
    a.div_shift = bits > 0 ? bits - 1 : 0;
    a.div_mul = (uint32_t)((((uint64_t)1 << (31 + a.div_shift)) + s->block_size - 1) / s->block_size);
    return a;
}

void launch_shape(qsa::AttnArgs &a, const AttnPlan &p, void *workspace) {
    a.sub_heads = p.sub_heads;
    a.num_subs = p.num_subs;
    a.tile_rows = p.tile_rows;
    a.slots = (int32_t)p.slots;
    a.tiles = (int32_t)p.tiles;
    a.part = p.bytes > 0 ? static_cast<float *>(workspace) : nullptr;
}

}  // namespace

extern "C" {

qsa_status qsa_plan_batch_check(const int32_t *past_lens, const int32_t *new_lens, const int32_t *free_blocks,
                                const int32_t *block_table, const int32_t *q_starts, const int32_t *row_to_req,
                                const int32_t *ctx_lens, const int64_t *slots, const qsa_plan_shape *shape) {
    return check_plan(past_lens, new_lens, free_blocks, block_table, q_starts, row_to_req, ctx_lens, slots, shape);
}

qsa_status qsa_plan_batch(const int32_t *past_lens, const int32_t *new_lens, const int32_t *free_blocks,
                          int32_t *block_table, int32_t *q_starts, int32_t *row_to_req, int32_t *ctx_lens,
                          int64_t *slots, int32_t *col_lens, int64_t *col_slots, int32_t *blocks_used,
                          const qsa_plan_shape *s, void *stream) {
    qsa_status st = check_plan(past_lens, new_lens, free_blocks, block_table, q_starts, row_to_req, ctx_lens, slots, s);
    if (st != QSA_OK) return st;
    qsa::PlanArgs a = {past_lens, new_lens, free_blocks, block_table, q_starts, row_to_req, ctx_lens, slots, col_lens,
                       col_slots, blocks_used, s->num_reqs, s->max_blocks, s->block_size, s->ratio, s->num_rows,
                       s->num_free, s->num_blocks};
    return launched(qsa::launch_plan(a, static_cast<hipStream_t>(stream)));
}

qsa_status qsa_write_kv_check(const void *k, const void *v, const int64_t *slots, const void *kcache,
                              const void *vcache, const qsa_kv_shape *shape) {
    return check_write_kv(k, v, slots, kcache, vcache, shape);
}

qsa_status qsa_write_kv(const void *k, const void *v, const int64_t *slots, void *kcache, void *vcache,
                        const qsa_kv_shape *s, void *stream) {
    qsa_status st = check_write_kv(k, v, slots, kcache, vcache, s);
    if (st != QSA_OK) return st;
    if (s->num_rows == 0) return ok();
    qsa::WriteKvArgs a = {static_cast<const uint8_t *>(k), static_cast<const uint8_t *>(v), slots,
                          static_cast<uint8_t *>(kcache), static_cast<uint8_t *>(vcache), s->num_rows,
                          s->num_kv_heads, s->head_dim, s->block_size, s->num_blocks, s->src_row_stride,
                          s->src_head_stride, s->kv_block_stride, s->kv_slot_stride, s->kv_head_stride};
    return launched(qsa::launch_write_kv(a, static_cast<hipStream_t>(stream)));
}

qsa_status qsa_write_keys_check(const void *keys, const int64_t *slots, const void *kcache, const float *kscale,
                                const qsa_keys_shape *shape) {
    return check_write_keys(keys, slots, kcache, kscale, shape);
}

qsa_status qsa_write_keys(const void *keys, const int64_t *slots, void *kcache, float *kscale,
                          const qsa_keys_shape *s, void *stream) {
    qsa_status st = check_write_keys(keys, slots, kcache, kscale, s);
    if (st != QSA_OK) return st;
    if (s->num_rows == 0) return ok();
    const int64_t elt = s->k_dtype == QSA_FP8_E4M3FN ? 1 : 2;
    const int64_t block = (int64_t)s->block_size * (s->head_dim * elt + (s->kv_layout != QSA_KV_PAGED ? 4 : 0));
    qsa::WriteKeysArgs a = {static_cast<const uint8_t *>(keys), slots, static_cast<uint8_t *>(kcache), kscale,
                            s->num_rows, s->head_dim, s->block_size, s->src_dtype, s->k_dtype, s->kv_layout,
                            s->num_blocks, s->src_stride, block};
    return launched(qsa::launch_write_keys(a, static_cast<hipStream_t>(stream)));
}

int64_t qsa_paged_attention_workspace_bytes(const qsa_attn_shape *s) {
    if (check_attn_sizes(s, false, 0, 0) != QSA_OK || s->num_rows == 0) return 0;
    return plan_attn(s, false, (int64_t)s->max_blocks * s->block_size).bytes;
}

qsa_status qsa_paged_attention_check(const void *q, const void *kcache, const void *vcache,
                                     const int32_t *block_table, const int32_t *ctx_lens, const int32_t *q_starts,
                                     const void *out, const qsa_attn_shape *s, const void *workspace,
                                     int64_t workspace_bytes) {
    qsa_status st = check_attn(q, kcache, vcache, block_table, ctx_lens, q_starts, out, s, false, 0, 0);
    if (st != QSA_OK) return st;
    return check_workspace(workspace, workspace_bytes, qsa_paged_attention_workspace_bytes(s));
}

qsa_status qsa_paged_attention(const void *q, const void *kcache, const void *vcache, const int32_t *block_table,
                               const int32_t *ctx_lens, const int32_t *q_starts, void *out, float *lse,
                               const qsa_attn_shape *s, void *workspace, int64_t workspace_bytes, void *stream) {
    qsa_status st = qsa_paged_attention_check(q, kcache, vcache, block_table, ctx_lens, q_starts, out, s, workspace,
                                              workspace_bytes);
    if (st != QSA_OK) return st;
    if (s->num_rows == 0) return ok();
    const AttnPlan p = plan_attn(s, false, (int64_t)s->max_blocks * s->block_size);
    qsa::AttnArgs a = attn_args(q, kcache, vcache, block_table, out, lse, s);
    a.ctx_lens = ctx_lens;
    a.q_starts = q_starts;
    launch_shape(a, p, workspace);
    return launched(p.stream ? qsa::launch_attn_stream(a, false, static_cast<hipStream_t>(stream))
                             : qsa::launch_attn_tile(a, static_cast<hipStream_t>(stream)));
}

int64_t qsa_sparse_attention_workspace_bytes(const qsa_attn_shape *s, int32_t k, int32_t ratio) {
    if (check_attn_sizes(s, true, k, ratio) != QSA_OK || s->num_rows == 0) return 0;
    return plan_attn(s, true, (int64_t)k * ratio).bytes;
}

qsa_status qsa_sparse_attention_check(const void *q, const void *kcache, const void *vcache,
                                      const int32_t *block_table, const int32_t *row_to_req, const int32_t *idx,
                                      int32_t k, int32_t ratio, const void *out, const qsa_attn_shape *s,
                                      const void *workspace, int64_t workspace_bytes) {
    qsa_status st = check_attn(q, kcache, vcache, block_table, row_to_req, idx, out, s, true, k, ratio);
    if (st != QSA_OK) return st;
    return check_workspace(workspace, workspace_bytes, qsa_sparse_attention_workspace_bytes(s, k, ratio));
}

qsa_status qsa_sparse_attention(const void *q, const void *kcache, const void *vcache, const int32_t *block_table,
                                const int32_t *row_to_req, const int32_t *idx, int32_t k, int32_t ratio,
                                const int32_t *token_lens, void *out, float *lse, const qsa_attn_shape *s,
                                void *workspace, int64_t workspace_bytes, void *stream) {
    qsa_status st = qsa_sparse_attention_check(q, kcache, vcache, block_table, row_to_req, idx, k, ratio, out, s,
                                               workspace, workspace_bytes);
    if (st != QSA_OK) return st;
    if (s->num_rows == 0) return ok();
    const AttnPlan p = plan_attn(s, true, (int64_t)k * ratio);
    qsa::AttnArgs a = attn_args(q, kcache, vcache, block_table, out, lse, s);
    a.ctx_lens = token_lens;
    a.row_to_req = row_to_req;
    a.idx = idx;
    a.k = k;
    a.ratio = ratio;
    launch_shape(a, p, workspace);
    return launched(qsa::launch_attn_stream(a, true, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
