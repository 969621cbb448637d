// Shared parts of the paged KV cache (cache.hip, attention.hip, rotary.hip,
// tree.hip, pool.hip): the views of an sz_cache and an sz_batch that kernels
// take, their host checks, and the device steps that several kernels need (a
// packed token's sequence, a page's address, FP8 rows to BF16 and back).
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
constexpr uint32_t kMaxHeads = 1024, kMaxQueryHeads = 0xFFFF;

// Host checks of single fields, which sizes of workspaces share.
inline int check_rows_type(uint32_t dtype, uint32_t head_dim)
{
    if (dtype != SZ_BF16 && dtype != SZ_FP8_E5M2 && dtype != SZ_FP8_E4M3) return SZ_E_DTYPE;
    return head_dim == 64 || head_dim == 128 ? SZ_OK : SZ_E_ARG;
}
inline int check_counts(const sz_batch *b)
{
    return b->seqs > (1u << 24) || b->tokens > kMaxTokens || b->max_kv > kMaxTokens ? SZ_E_ARG : SZ_OK;
}

// Host checks of a batch by itself, and of its pages' size (no device memory
// is touched).
inline int check_batch(const sz_batch *b, const int32_t *d_status, PagedBatch &pb)
{
    if (check_counts(b) != SZ_OK) return SZ_E_ARG;
    if (b->seqs && (!b->starts || !b->kv_lens || (b->table_width && !b->page_table))) return SZ_E_ARG;
    for (const void *p : {(const void *)b->page_table, (const void *)b->kv_lens, (const void *)b->starts,
                          (const void *)d_status})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return SZ_E_ALIGN;
    pb = PagedBatch{b->page_table, b->kv_lens, b->starts, b->seqs, b->table_width, b->tokens,
                    std::min(b->max_new, b->tokens), b->max_kv, const_cast<int32_t *>(d_status)};
    return SZ_OK;
}
inline int page_size(uint32_t page_tokens, uint32_t &lg)
{
    if (page_tokens < kMinPage || page_tokens > kMaxPage || (page_tokens & (page_tokens - 1))) return SZ_E_ARG;
    for (lg = 0; (1u << lg) < page_tokens;) ++lg;
    return SZ_OK;
}

// Host checks of a cache and a batch.
inline int check_paged(const sz_cache *c, const sz_batch *b, const int32_t *d_status, PagedCache &pc, PagedBatch &pb)
{
    if (!c || !b) return SZ_E_ARG;
    const int type = check_rows_type(c->dtype, c->head_dim);
    if (type != SZ_OK) return type;
    uint32_t lg = 0;
    if (page_size(c->page_tokens, lg) != SZ_OK) return SZ_E_ARG;
    if (c->kv_heads == 0 || c->kv_heads > kMaxHeads || c->pages == 0 || c->pages > 0x7FFFFFFFull || !c->data)
        return SZ_E_ARG;
    if (c->dtype != SZ_BF16 && !c->scales) return SZ_E_ARG;
    if (!aligned16(c->data) || !aligned16(c->scales)) return SZ_E_ALIGN;
    if ((uint64_t)b->max_kv > (uint64_t)b->table_width * c->page_tokens) return SZ_E_ARG;
    const int rc = check_batch(b, d_status, pb);
    if (rc != SZ_OK) return rc;
    if (!d_status) return SZ_E_ARG;
    pc = PagedCache{static_cast<uint8_t *>(c->data), static_cast<uint8_t *>(c->scales), (uint32_t)c->pages,
                    c->kv_heads, lg};
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
__device__ __forceinline__ bool consistent(const PagedBatch &b, int32_t start, int32_t next, int32_t len)
{
    return start >= 0 && next >= start && next <= (int32_t)b.tokens && next - start <= (int32_t)b.max_new && len >= 0 &&
           len <= (int32_t)b.max_kv;
}
__device__ __forceinline__ Sequence checked(const PagedBatch &b, int32_t start, int32_t next, int32_t len)
{
    if (!consistent(b, start, next, len)) {
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

// Lanes per row of the calls that move rows: each moves 8 values (16 bytes of BF16).
template <int D>
constexpr uint32_t kRowLanes = D / 8;

// Maximum over the LANES (8 or 16) lanes of a row, DPP within 16 lanes:
// quad_perm swaps of 1 and 2, then mirrors of 8 and 16.
template <uint32_t LANES>
__device__ __forceinline__ uint32_t row_max(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
    if (LANES == 16) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
    return v;
}

template <int DT>
__device__ __forceinline__ uint32_t fp8_pair(float lo, float hi, uint32_t into, bool high)
{
    if constexpr (DT == SZ_FP8_E4M3)
        return high ? __builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, into, true)
                    : __builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, into, false);
    else
        return high ? __builtin_amdgcn_cvt_pk_bf8_f32(lo, hi, into, true)
                    : __builtin_amdgcn_cvt_pk_bf8_f32(lo, hi, into, false);
}

// One 16-byte chunk of a row, BF16 -> cache.
template <int DT, int D>
__device__ __forceinline__ void put_chunk(const PagedCache &c, uint64_t at, uint32_t off, uint4 v)
{
    if constexpr (DT == SZ_BF16) {
        *reinterpret_cast<uint4 *>(c.data + (at * D + off) * 2) = v;
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t a = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t lo = w[e] & 0x7FFFu, hi = (w[e] >> 16) & 0x7FFFu;
            a = max(a, lo < 0x7F80u ? lo : 0u);
            a = max(a, hi < 0x7F80u ? hi : 0u);
        }
        a = row_max<kRowLanes<D>>(a);
        // a = 1.m 2^(E-127): a <= 1.75 2^(EMAX+k) from k = E - 127 - EMAX, one more where 1.m > 1.75
        constexpr int32_t EMAX = DT == SZ_FP8_E4M3 ? 8 : 15;
        const int32_t byte = max(1, (int32_t)(a >> 7) - EMAX + ((a & 0x7Fu) > 0x60u ? 1 : 0));
        const float inv = __builtin_bit_cast(float, (uint32_t)(254 - byte) << 23);
        uint32_t q[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float lo = __builtin_bit_cast(float, w[e] << 16) * inv;
            const float hi = __builtin_bit_cast(float, w[e] & 0xFFFF0000u) * inv;
            q[e / 2] = fp8_pair<DT>(lo, hi, q[e / 2], e % 2 == 1);
        }
        *reinterpret_cast<uint2 *>(c.data + at * D + off) = make_uint2(q[0], q[1]);
        if (off == 0) c.scales[at] = (uint8_t)byte;
    }
}

// The sequence and position of token t0 + lane, for the wave's lanes below
// TOKENS (others, and tokens without a place: false).  Loads that wait for one
// another are most of a small call's time, so the starts and lengths of the 64
// sequences from t0's on come in one (up to 63 sequences: the first), and each
// token counts its own from there.  `edges`: this wave also looks at what no
// token's own sequence shows.
template <uint32_t TOKENS>
__device__ __forceinline__ bool token_position(const PagedBatch &b, uint32_t t0, bool edges, uint32_t &seq, int32_t &pos)
{
    const uint32_t lane = lane_id();
    uint32_t base = 0;
    for (uint32_t span = b.seqs + 1; span > 64;) {
        const uint32_t step = (span + 63) / 64, at = lane * step;
        const uint32_t hits = (uint32_t)__popcll(__ballot(at < span && (int64_t)b.starts[base + min(at, span - 1)] <= t0));
        const uint32_t skip = hits > 0 ? (hits - 1) * step : 0;
        base += skip;
        span = min(step, span - skip);
    }
    const bool there = base + lane < b.seqs;
    const int32_t start = base + lane <= b.seqs ? b.starts[base + lane] : INT32_MAX;
    const int32_t len = there ? b.lens[base + lane] : 0;
    // Starts that descend, and an axis that begins or ends outside [0, tokens].
    const int32_t after = __shfl_down(start, 1, 64);
    bool wrong = lane < 63 && there && after < start;
    if (edges && lane < 2) {
        const int32_t edge = b.starts[lane * b.seqs];
        wrong |= edge < 0 || edge > (int32_t)b.tokens;
    }
    if (wrong) flag_batch(b);
    uint32_t count = 0;                              // of the starts up to this lane's token
#pragma unroll
    for (uint32_t j = 0; j < TOKENS; ++j) {
        const uint64_t passed = __ballot(start <= (int32_t)(t0 + j));
        if (lane == j) count = (uint32_t)__popcll(passed);
    }
    const int32_t my_start = __shfl(start, (int)max(count, 1u) - 1, 64), my_next = __shfl(start, (int)min(count, 63u), 64);
    const int32_t my_len = __shfl(len, (int)max(count, 1u) - 1, 64);
    if (lane >= TOKENS || t0 + lane >= b.tokens || count == 0) return false;
    const uint32_t t = t0 + lane;
    uint32_t i = base + count - 1;
    Sequence s{0, 0, 0};
    if (count < 64) {
        if (i < b.seqs) s = checked(b, my_start, my_next, my_len);
    } else {                                         // 64 sequences on, or more
        for (uint32_t past = b.seqs; past - i > 1;) {
            const uint32_t mid = i + (past - i) / 2;
            (b.starts[mid] <= (int32_t)t ? i : past) = mid;
        }
        if (i < b.seqs) s = sequence(b, i);
    }
    seq = i;
    pos = s.len - s.n + ((int32_t)t - s.start);
    return (int32_t)t >= s.start && (int32_t)t < s.start + s.n && pos >= 0;
}

}  // namespace sz
