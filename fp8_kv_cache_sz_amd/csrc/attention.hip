// Causal attention over the paged KV cache (attention.hpp), and the workspace
// that both kinds of attention take.
#include "attention.hpp"

using namespace sz;

// A size is asked for before any call has looked at the fields, and the plan's
// divisions and products hold within what the calls take: nothing else has one.
static bool has_plan(const sz_cache *c, const sz_batch *b, uint32_t q_heads)
{
    return c && b && check_rows_type(c->dtype, c->head_dim) == SZ_OK && c->kv_heads > 0 && c->kv_heads <= kMaxHeads &&
           q_heads > 0 && q_heads <= kMaxQueryHeads && q_heads % c->kv_heads == 0 && check_counts(b) == SZ_OK;
}

extern "C" uint64_t sz_paged_attention_workspace_size(const sz_cache *cache, const sz_batch *batch, uint32_t q_heads)
{
    if (!has_plan(cache, batch, q_heads)) return 0;
    PagedBatch b{};
    b.seqs = batch->seqs;
    b.tokens = batch->tokens;
    b.max_new = std::min(batch->max_new, batch->tokens);
    b.max_kv = batch->max_kv;
    if (b.seqs == 0 || b.tokens == 0) return attn_ws_bytes(1, 0, 0);
    // the most chunks that any window gives
    const AttnPlan p = attn_plan(cache, b, q_heads / cache->kv_heads, 0, false);
    uint64_t splits = 1;
    if (p.rows)
        splits = std::max(splits, most_splits(b.max_kv, rows_wanted(b.max_kv, (uint64_t)b.seqs * cache->kv_heads)));
    if (p.tiles)
        splits = std::max(splits, most_splits(b.max_kv, tiles_wanted(b.max_kv, (uint64_t)p.slots * cache->kv_heads, p.tile_waves,
                                                                     (uint64_t)b.tokens * q_heads * cache->head_dim)));
    const AttnPlan t = attn_plan(cache, b, q_heads / cache->kv_heads, 0, true);
    if (t.tiles)
        splits = std::max(splits, most_splits(b.max_kv, tiles_wanted(b.max_kv, (uint64_t)t.grid_slots * cache->kv_heads, t.tile_waves,
                                                                     (uint64_t)b.tokens * q_heads * cache->head_dim)));
    if (rows_in_blocks(cache, b, q_heads / cache->kv_heads))             // trees
        splits = std::max(splits, most_splits(b.max_kv, rows_wanted(b.max_kv, (uint64_t)b.seqs * cache->kv_heads *
                                                                                  row_blocks(b, q_heads / cache->kv_heads))));
    return attn_ws_bytes(splits, (uint64_t)b.tokens * q_heads, cache->head_dim);
}

extern "C" int sz_paged_attention(const sz_cache *cache, const sz_batch *batch, const void *d_q, uint32_t q_heads,
                                  uint64_t q_token_stride, uint64_t q_head_stride, float scale, uint32_t window,
                                  void *d_out, float *d_lse, void *d_ws, uint64_t ws_bytes, int32_t *d_status,
                                  void *stream)
{
    return attend(AttnArgs{}, cache, batch, d_q, q_heads, q_token_stride, q_head_stride, scale, window, d_out, d_lse, d_ws,
                  ws_bytes, d_status, stream);
}
