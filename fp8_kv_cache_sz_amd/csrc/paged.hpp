// Shared parts of the paged KV cache (cache.hip, attention.hip): the views of
// an sz_cache and an sz_batch that kernels take, their host checks, and the
// device steps that every kernel of the cache needs (a packed token's
// sequence, a page's address, FP8 rows to BF16).
//
// Everything a batch says lies in device memory, so the kernels check it as
// they read it: a sequence whose lengths contradict each other or the host's
// bounds is skipped, a page number outside the cache is read as page 0 and
// never written, and either puts SZ_E_FORMAT into the status word.  No
// address is formed from an unchecked value.
#pragma once

#include "common.hpp"
#include "keys.hpp"

namespace sz {

struct PagedCache {
    uint8_t *data;            // [pages][2][heads][1 << lg_page][D]
    uint8_t *scales;          // [pages][2][heads][1 << lg_page], FP8 only
    uint32_t pages;
    uint32_t heads;
    uint32_t lg_page;
};

struct PagedBatch {
    const int32_t *table;     // [seqs][width]
    const int32_t *lens;      // [seqs]
    const int32_t *starts;    // [seqs + 1]
    uint32_t seqs, width;
    uint32_t tokens, max_new, max_kv;
    int32_t *status;
};

// One sequence as its kernel sees it: new tokens [start, start + n) of the
// packed axis at positions [len - n, len).
struct Sequence {
    int32_t start, n, len;
};

constexpr uint32_t kMinPage = 16, kMaxPage = 1024;
constexpr uint32_t kMaxHeads = 1024;

// Host checks of a cache and a batch (no device memory is touched).
inline int check_paged(const sz_cache *c, const sz_batch *b, const int32_t *d_status, PagedCache &pc, PagedBatch &pb)
{
    if (!c || !b) return SZ_E_ARG;
    if (c->dtype != SZ_BF16 && c->dtype != SZ_FP8_E5M2 && c->dtype != SZ_FP8_E4M3) return SZ_E_DTYPE;
    if (c->head_dim != 64 && c->head_dim != 128) return SZ_E_ARG;
    if (c->page_tokens < kMinPage || c->page_tokens > kMaxPage || (c->page_tokens & (c->page_tokens - 1)))
        return SZ_E_ARG;
    if (c->kv_heads == 0 || c->kv_heads > kMaxHeads || c->pages == 0 || c->pages > 0x7FFFFFFFull || !c->data)
        return SZ_E_ARG;
    if (c->dtype != SZ_BF16 && !c->scales) return SZ_E_ARG;
    if (!aligned16(c->data) || !aligned16(c->scales)) return SZ_E_ALIGN;
    if (b->seqs > (1u << 24) || b->tokens > kMaxTokens || b->max_kv > kMaxTokens) return SZ_E_ARG;
    if (b->seqs && (!b->starts || !b->kv_lens || (b->table_width && !b->page_table))) return SZ_E_ARG;
    if ((uint64_t)b->max_kv > (uint64_t)b->table_width * c->page_tokens) return SZ_E_ARG;
    for (const void *p : {(const void *)b->page_table, (const void *)b->kv_lens, (const void *)b->starts,
                          (const void *)d_status})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return SZ_E_ALIGN;
    if (!d_status) return SZ_E_ARG;
    uint32_t lg = 0;
    while ((1u << lg) < c->page_tokens) ++lg;
    pc = PagedCache{static_cast<uint8_t *>(c->data), static_cast<uint8_t *>(c->scales), (uint32_t)c->pages,
                    c->kv_heads, lg};
    pb = PagedBatch{b->page_table, b->kv_lens, b->starts, b->seqs, b->table_width, b->tokens,
                    std::min(b->max_new, b->tokens), b->max_kv, const_cast<int32_t *>(d_status)};
    return SZ_OK;
}

// A [tokens][heads][head_dim] BF16 tensor whose rows are contiguous: strides
// in elements, each row 16-byte aligned.
inline int check_rows(const void *p, uint64_t token_stride, uint64_t head_stride, uint64_t tokens, uint32_t heads)
{
    if (tokens && !p) return SZ_E_ARG;
    if (!aligned16(p)) return SZ_E_ALIGN;
    if ((tokens > 1 && token_stride % 8) || (heads > 1 && head_stride % 8)) return SZ_E_ALIGN;
    if (token_stride >= (1ull << 40) || head_stride >= (1ull << 40)) return SZ_E_ARG;
    return SZ_OK;
}

// ---------------------------------------------------------------------------
// Device steps
// ---------------------------------------------------------------------------
__device__ __forceinline__ void flag_batch(const PagedBatch &b) { *b.status = SZ_E_FORMAT; }

__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

// A sequence's lengths, checked against the host's bounds; a sequence that
// contradicts them has no tokens.
__device__ __forceinline__ Sequence checked(const PagedBatch &b, int32_t start, int32_t next, int32_t len)
{
    const bool good = start >= 0 && next >= start && next <= (int32_t)b.tokens && next - start <= (int32_t)b.max_new &&
                      len >= 0 && len <= (int32_t)b.max_kv;
    if (!good) {
        flag_batch(b);
        return Sequence{0, 0, 0};
    }
    return Sequence{start, next - start, len};
}
__device__ __forceinline__ Sequence sequence(const PagedBatch &b, uint32_t i)
{
    return checked(b, b.starts[i], b.starts[i + 1], b.lens[i]);
}

// Largest i in [0, count) with key(i) <= x for ascending keys, or -1; one
// wave, 64 keys a step (one step up to 64 keys, two up to 4,096).
template <typename Key>
__device__ __forceinline__ int32_t wave_last_not_above(uint32_t count, int64_t x, Key key)
{
    uint32_t lo = 0, span = count;                       // the answer is in [lo, lo + span) or lo - 1
    while (span > 0) {
        const uint32_t step = (span + 63) / 64;
        const uint32_t off = lane_id() * step;
        const bool in = off < span;
        const int64_t v = key(lo + (in ? off : 0));
        const uint32_t hits = (uint32_t)__popcll(__ballot(in && v <= x));
        if (hits == 0) return (int32_t)lo - 1;
        const uint32_t first = (hits - 1) * step;
        if (step == 1) return (int32_t)(lo + first);
        lo += first + 1;                                 // lo - 1 is not above x
        span = min(step - 1, span - first - 1);
    }
    return (int32_t)lo - 1;
}

// The page that holds position p of sequence i, 0 (flagged) where the table
// names none of the cache's.  p < len.
__device__ __forceinline__ uint32_t page_of(const PagedCache &c, const PagedBatch &b, uint32_t i, uint32_t p)
{
    const uint32_t page = (uint32_t)b.table[(uint64_t)i * b.width + (p >> c.lg_page)];
    if (page >= c.pages) {
        flag_batch(b);
        return 0;
    }
    return page;
}

// Row (page, K or V, head, row in page) of the cache, counted in rows.
__device__ __forceinline__ uint64_t row_index(const PagedCache &c, uint32_t page, uint32_t kv, uint32_t head,
                                              uint32_t row)
{
    return ((((uint64_t)page * 2 + kv) * c.heads + head) << c.lg_page) + row;
}

// Two FP8 values (the low or high half of w) times 2^(byte - 127), as a BF16
// pair; scale_bits = byte << 23, of which the instruction takes the exponent:
// byte 0 is 2^-127, 255 a NaN.  One instruction, exact: an FP8 value has at
// most four significant bits and BF16 keeps eight, so the product rounds only
// where it leaves BF16's range.
template <int DT, bool HI>
__device__ __forceinline__ uint32_t fp8_pair_to_bf16(uint32_t w, uint32_t scale_bits)
{
    const float s = __builtin_bit_cast(float, scale_bits);
    if constexpr (DT == SZ_FP8_E4M3)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, HI));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, s, HI));
}

}  // namespace sz
