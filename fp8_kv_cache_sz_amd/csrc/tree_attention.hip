// Attention of trees of drafted tokens over the paged KV cache: the kernels of
// attention.hpp with masks among the new tokens.  A source of its own, so that the
// causal kernels' code does not depend on these.
#include "attention.hpp"

using namespace sz;

extern "C" int sz_tree_attention(const sz_cache *cache, const sz_batch *batch, const uint64_t *d_masks, uint32_t words,
                                 const void *d_q, uint32_t q_heads, uint64_t q_token_stride, uint64_t q_head_stride,
                                 float scale, uint32_t window, void *d_out, float *d_lse, void *d_ws, uint64_t ws_bytes,
                                 int32_t *d_status, void *stream)
{
    if (!batch || words == 0 || words > SZ_TREE_WORDS || std::min(batch->max_new, batch->tokens) > 64ull * words) return SZ_E_ARG;
    if (batch->tokens && batch->seqs && !d_masks) return SZ_E_ARG;
    if (reinterpret_cast<uintptr_t>(d_masks) & 7u) return SZ_E_ALIGN;
    TreeArgs a{};
    a.masks = d_masks;
    a.words = words;
    return attend(a, cache, batch, d_q, q_heads, q_token_stride, q_head_stride, scale, window, d_out, d_lse, d_ws, ws_bytes,
                  d_status, stream);
}
