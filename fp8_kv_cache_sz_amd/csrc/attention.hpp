// Attention of new tokens over the paged KV cache: the kernels and their plans,
// for causal attention (attention.hip) and for trees of drafted tokens
// (tree_attention.hip).
//
// For a new token at position p of its sequence and query head h (KV head
// h / G), over the visible keys j, max(0, p - window + 1) <= j <= p:
//   s_j = scale q . K_j      m = max s_j      l = sum exp(s_j - m)
//   o   = sum exp(s_j - m) V_j / l            lse = m + ln l
// computed in one pass over the keys with a running m and l, in powers of two:
// exp(s - m) = 2^(c (x - m')), x = q . K_j, c = scale log2 e.  m' need not be
// the maximum itself, only near enough that no power overflows: it is raised,
// and the sums scaled, only when a score exceeds it by more than 2^kSlack,
// which is rare after the first keys.  Scores, m', l and o are 32 bits, and K
// and V enter as the exact BF16 values that sz_cache_read returns.  The matrix
// instructions take BF16 probabilities: sz_attn_rows, which waits for memory,
// gives them what the rounding left as a second product; sz_attn_tiles, bound
// by those products, rounds (at most 2^-8 of each, of either sign, as much as
// the result's own rounding: 0.0020 to 0.0024 of a result's size from the
// 64-bit one where 32-bit probabilities leave 0.0016 to 0.0017).  A second
// product would be half as many products again.  l adds the powers before the
// rounding, so that lse keeps 32 bits.
//
// Rows are (token, head of the KV head's group), so one K/V row read serves
// the G query heads of its KV head.  Both kernels compute S^T = K Q^T, whose
// result layout gives each lane one row's scores (maxima and sums stay in
// the lane) and is, keys renumbered, the operand layout of O^T = V^T P^T: P
// never leaves its registers.
//   sz_attn_rows  sequences with at most 16 (or 32) rows per KV head (single
//                 tokens, drafts): bound by reading K and V.
//   sz_attn_tiles the others: 128 rows a workgroup, bound by the matrix and
//                 vector units.
// Where there are few rows the keys are split into chunks whose partial
// (m, l, o) sz_attn_join joins, always in the order of the chunks.
//
// Trees (TreeArgs) differ in what hides a score: cached keys j < len - n are seen
// as by a causal token, of the n new ones those that the row's mask names.  So
// only the blocks and tiles that reach the new tokens (or a window's start) look at
// masks, 64 keys at a time, as one shifted 64-bit word of the row; all others run
// the causal code.  A row's causal order is gone, which leaves equal work to all
// tiles of a sequence, and room for other plans: equal slots (tiles_each), long
// sequences first (fold_of), fewer and longer chunks (kTreeFill), small batches in
// blocks of 16 rows (rows_in_blocks).  Measured (MI355X, 8 KV heads of 128, four
// query heads each, calls one after another; a launch by itself, traced, takes 4 to
// 8 % more): 64 trees of 8 tokens over up to 4,000 keys, E5M2 58 us, 5.3 TB/s; 32 of
// 61 over up to 8,192, E4M3 200 us, 738 TFLOP/s (32 over 8,192 each 291 to 309 us,
// 902 to 849, on two cards); 13 tokens over 1,000 in BF16 12.7 us, which is a chain
// of launch, lengths, masks, page, K and V, join.
// Which kernel a batch gets, and with it whether probabilities are held to 2^-15
// or rounded to BF16, follows the host's bounds (attn_plan) and not the lengths.
#pragma once

#include "paged.hpp"

#include <cmath>
#include <type_traits>

namespace sz {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// A lambda whose captures are registers: a call would put them in memory.
#define SZ_INLINE __attribute__((always_inline))

constexpr uint32_t kAttnThreads = 256;
constexpr uint32_t kRowsTokens = 256;    // of a tree in sz_attn_rows
constexpr uint32_t kRowsMax = 16;        // rows of sz_attn_rows, or twice as many: its products have 16
constexpr uint32_t kTileKeys = 64;
constexpr uint32_t kKeyAlign = 64;       // chunks start at multiples of this
constexpr float kSlack = 8.0f;
constexpr float kNone = -__builtin_huge_valf();

struct AttnArgs {
    PagedCache c;
    PagedBatch b;
    const uint16_t *q;
    uint64_t q_token, q_head;
    uint16_t *out;            // [tokens][q_heads][D]
    float *lse;               // [tokens][q_heads] or null
    float *part;              // [splits][tokens][q_heads][D], o before the division by l
    float2 *part_ml;          // [splits][tokens][q_heads] (m', l)
    uint32_t *arrived;        // [seqs][kv heads] chunks done, 0 between calls; null: sz_attn_join joins
    float scale, c2;          // c2: scale log2 e
    uint32_t group, q_heads;
    int32_t window;           // 0: none; window_keys()
    uint32_t rows_limit;      // sequences of up to so many rows are sz_attn_rows's
    uint32_t rows_chunk, rows_splits;      // keys of a chunk, chunks (sz_attn_rows)
    uint32_t tile_chunk, tile_splits;      // (sz_attn_tiles)
    static constexpr bool kTree = false, kOrdered = false;
};

// Of trees of drafted tokens: the kernels are the same, told apart by their
// arguments' type.
struct TreeArgs : AttnArgs {
    const uint64_t *masks;    // [tokens][words], the new tokens that a token sees
    uint32_t words;
    uint32_t tiles_each;      // slots of a sequence, 0: as many as its tokens need, and one
    uint32_t fold;            // sequences in the order of their lengths (by_length), 0: in their own
    uint32_t row_blocks;      // of a sequence's rows in sz_attn_rows
    uint32_t rows_fold;       // as fold, where sz_attn_rows takes OrderedArgs
    static constexpr bool kTree = true;
};
// sz_attn_rows with its sequences in the order of their lengths.  A kernel of its
// own: finding the order costs a small call 1.6 us of 14.
struct OrderedArgs : TreeArgs {
    static constexpr bool kOrdered = true;
};

// First key of sequence s that any of its new tokens sees, rounded down.
__device__ __forceinline__ int32_t first_key(const Sequence &s, int32_t window)
{
    return first_seen(s.len - s.n, window) & ~(int32_t)(kKeyAlign - 1);
}

// The visible keys [lo, hi] of position p; none (hi < lo) for p < 0.
__device__ __forceinline__ void visible(int32_t p, int32_t window, int32_t &lo, int32_t &hi)
{
    hi = p;
    lo = first_seen(p, window);
}

// What a token of a tree sees: of the cached keys, which end before `past` =
// len - n, those from lo on, and of the new ones those that its mask names.
// Bits of new tokens that have no place are not looked at, nor is the mask of
// a token without one (p < 0).
struct Sight {
    int32_t lo;
    bool blind;               // sees nothing
};
// Bits 0..63: new tokens from..from + 63 that token tok of sequence s sees.
__device__ __forceinline__ uint64_t new_seen(const TreeArgs &a, const Sequence &s, int32_t tok, int32_t from)
{
    const int32_t past = s.len - s.n, none = max(0, -past);          // the first new token with a place
    if (tok < none || from >= s.n || from + 63 < none) return 0;
    const uint64_t *row = a.masks + (uint64_t)(s.start + tok) * a.words;
    const int32_t w = from >> 6, shift = from & 63;                  // w = -1: before the first
    uint64_t bits = w >= 0 ? row[w] >> shift : 0;
    if (shift && w + 1 < (int32_t)a.words) bits |= row[w + 1] << (64 - shift);
    if (from < none) bits &= ~0ull << (none - from);
    if (s.n - from < 64) bits &= ~(~0ull << (s.n - from));
    return bits;
}
__device__ __forceinline__ uint32_t row_blocks(const TreeArgs &a) { return a.row_blocks; }
__device__ __forceinline__ uint32_t row_blocks(const AttnArgs &) { return 1; }
__device__ __forceinline__ Sight tree_sight(const TreeArgs &a, const Sequence &s, int32_t tok)
{
    const int32_t past = s.len - s.n;
    if (a.window == 0 && past > 0) return Sight{0, false};           // whatever the mask says
    int32_t count = 0;
    for (int32_t from = 0; from < s.n; from += 64) count += (int32_t)__popcll(new_seen(a, s, tok, from));
    Sight v;
    v.lo = first_seen(past + max(count, 1) - 1, a.window);
    v.blind = count == 0 && v.lo >= past;
    return v;
}
// Bits 0..63: keys kb..kb + 63 that are cached before the new ones and seen.
__device__ __forceinline__ uint64_t old_seen(int32_t lo, int32_t past, int32_t kb)
{
    const int32_t first = max(lo - kb, 0), end = min(past - kb, 64);
    if (first >= end) return 0;
    return (~0ull >> (64 - (end - first))) << first;
}

// A value that the compiler takes for a new one: what follows from it is worked
// out here, not kept in registers from before.
__device__ __forceinline__ uint32_t opaque(uint32_t x)
{
    asm volatile("" : "+v"(x));
    return x;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// A factor of sums, 2^x.  Never 0, so that an infinite sum stays infinite: at
// 2^-149 it is as much below the powers themselves, which end at 2^-126.
__device__ __forceinline__ float scaling(float x) { return fmaxf(exp2_fast(x), 0x1p-149f); }

// A row's running reference.  The powers are 2^(c x - base) with base = c m'
// rounded: one fused multiply each.  delta = c m' - base is what the rounding
// left; it keeps the reference exact where it changes.  Where |c m'| is over
// kFar the rounding could be a power of its own, so there (far, of the whole
// wave: rare) the scores are made differences x - m' first, and base = -delta.
constexpr float kFar = 1048576.f;
struct Reference {
    float top = kNone, delta = 0.f;                    // m' and delta
    __device__ __forceinline__ bool below(float x, float c) const { return (x - top) * c > kSlack; }
    // Raises m' to x at least; what the sums so far are to be scaled by.
    __device__ __forceinline__ float raise(float x, float c)
    {
        const float raised = fmaxf(top, x), base = raised * c;
        const float rest = fabsf(base) <= kFar ? __builtin_fmaf(raised, c, -base) : 0.f;
        const float f = raised == kNone ? 1.f : scaling(__builtin_fmaf(top - raised, c, rest - delta));
        top = raised;
        delta = rest;
        return f;
    }
    __device__ __forceinline__ bool is_far(float c) const { return top != kNone && !(fabsf(top * c) <= kFar); }
    __device__ __forceinline__ float origin() const { return top == kNone ? 0.f : top; }       // of far differences
    __device__ __forceinline__ float base(float c, bool far) const
    {
        return top == kNone ? 0.f : far ? -delta : __builtin_fmaf(top, c, -delta);
    }
};
// 2^(c (x - top)) for sums that were made with m' = x
__device__ __forceinline__ float rebased(float x, float top, float c)
{
    return scaling((x - (top == kNone ? 0.f : top)) * c);
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

// Bits 15 and 31 tell whether the BF16 halves of a pair are NaN or infinite.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; }
constexpr uint32_t kNotFinite = 0x80008000u;

// NaN and infinities among V rows that some rows of a tile see and others do
// not: the tile's product may not meet them, since 0 times either is a NaN.
// They are counted instead, by a product of their own: kinds(w) has 1 for
// +inf, 128 for -inf and 16384 for a NaN in either BF16 of a pair and else 0,
// a row's second operand is 1 where it sees the key, and the sums over at
// most 64 keys hold the three counts, exactly.  from_kinds(sum) is what the
// counted values add up to; finite(w) is what is left for the tile's product.
__device__ __forceinline__ uint32_t kinds(uint32_t w)
{
    const uint32_t ends = (not_finite(w) & kNotFinite) >> 15;                       // 1 in each such half
    const uint32_t nan = ends & (((w & 0x007F007Fu) + 0x007F007Fu) >> 7);           // mantissa not 0
    const uint32_t minus = ends & ~nan & (w >> 15), plus = ends & ~nan & ~(w >> 15);
    return nan * 0x4680u | minus * 0x4300u | plus * 0x3F80u;
}
__device__ __forceinline__ float from_kinds(float sum)
{
    const uint32_t c = (uint32_t)sum;
    const bool plus = c & 127u, minus = c & 16383u & ~127u;
    return c >= 16384u || (plus && minus) ? __builtin_nanf("") : minus ? kNone : plus ? -kNone : 0.f;
}
__device__ __forceinline__ uint32_t finite(uint32_t w)
{
    return w & ~(((not_finite(w) & kNotFinite) >> 15) * 0xFFFFu);
}
// 1.0 in the halves of a pair of keys that bits 0 and 1 say
__device__ __forceinline__ uint32_t seen_pair(uint64_t bits)
{
    return (bits & 1 ? 0x3F80u : 0u) | (bits & 2 ? 0x3F800000u : 0u);
}
// ... that [lo, hi] holds
__device__ __forceinline__ uint32_t seen_pair(int32_t key, int32_t lo, int32_t hi)
{
    return (key >= lo && key <= hi ? 0x3F80u : 0u) | (key + 1 >= lo && key + 1 <= hi ? 0x3F800000u : 0u);
}

// Partials that another workgroup of the same launch joins pass through the
// memory that all XCDs see: the relaxed atomic accesses of the device's scope
// write through an XCD's L2 and do not read what it holds, so a workgroup
// that has waited for its stores need not write that L2 back (a release
// fence) before it counts itself, nor the one that joins empty it.
__device__ __forceinline__ void publish(float *p, float x, float y)
{
    __hip_atomic_store(reinterpret_cast<uint64_t *>(p), __builtin_bit_cast(uint64_t, make_float2(x, y)),
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <bool SHARED>
__device__ __forceinline__ float2 partial2(const float *p)
{
    if constexpr (!SHARED) return *reinterpret_cast<const float2 *>(p);
    return __builtin_bit_cast(float2, __hip_atomic_load(reinterpret_cast<const uint64_t *>(p), __ATOMIC_RELAXED,
                                                        __HIP_MEMORY_SCOPE_AGENT));
}
template <bool SHARED>
__device__ __forceinline__ float4 partial4(const float *p)
{
    if constexpr (!SHARED) return *reinterpret_cast<const float4 *>(p);
    const float2 x = partial2<true>(p), y = partial2<true>(p + 2);
    return make_float4(x.x, x.y, y.x, y.y);
}

// Writes one row's EL consecutive values at d: the result, or a chunk's partial.
template <int D, int EL>
__device__ __forceinline__ void store_row(const AttnArgs &a, bool whole, uint32_t split, uint32_t token,
                                          uint32_t head, uint32_t d, const float (&o)[EL], float inv)
{
    const uint64_t r = (uint64_t)token * a.q_heads + head;
    if (whole) {
        uint32_t w[EL / 2];
#pragma unroll
        for (int e = 0; e < EL / 2; ++e) w[e] = bf16_pair(o[2 * e] * inv, o[2 * e + 1] * inv);
        uint32_t *p = reinterpret_cast<uint32_t *>(a.out + r * D + d);
        if constexpr (EL == 8)
            *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
        float *p = a.part + ((uint64_t)split * a.b.tokens * a.q_heads + r) * D + d;
#pragma unroll
        for (int e = 0; e < EL; e += 4) {
            if (a.arrived) {
                publish(p + e, o[e], o[e + 1]);
                publish(p + e + 2, o[e + 2], o[e + 3]);
            } else {
                *reinterpret_cast<float4 *>(p + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
        }
    }
}

// A row's statistics: its lse, or a chunk's (m', l).
__device__ __forceinline__ void store_stats(const AttnArgs &a, bool whole, uint32_t split, uint32_t token,
                                            uint32_t head, bool empty, float m, float l)
{
    const uint64_t r = (uint64_t)token * a.q_heads + head;
    if (!whole)
        publish(reinterpret_cast<float *>(a.part_ml + (uint64_t)split * a.b.tokens * a.q_heads + r), m, l);
    else if (a.lse)
        a.lse[r] = empty ? kNone : __builtin_fmaf(__log2f(l), 0.69314718055994530942f, m * a.scale);
}

// Chunks that sequence s has.  One is the whole result.
__device__ __forceinline__ uint32_t chunks_of(const Sequence &s, int32_t window, uint32_t chunk)
{
    return max(1u, ((uint32_t)(s.len - min(first_key(s, window), s.len)) + chunk - 1) / chunk);
}

// Joining chunks:  M = max m'_s;  f_s = 2^(c (m'_s - M));  o = sum f_s o_s /
// sum f_s l_s.  D/4 lanes hold a row.
struct Joined {
    float m = kNone, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void add(float2 ml, float4 v, float c)
    {
        const float raised = fmaxf(m, ml.x);
        const float f = rebased(m, raised, c), g = rebased(ml.x, raised, c);
        m = raised;
        l = l * f + ml.y * g;
        o = make_float4(o.x * f + v.x * g, o.y * f + v.y * g, o.z * f + v.z * g, o.w * f + v.w * g);
    }
};

// The visible chunks [s0, s1) of a token at position p.
// (Of a tree's: those from its first cached key, or the first new one, on.)
template <bool TREE>
__device__ __forceinline__ void chunk_range(const Sequence &s, int32_t p, int32_t window, uint32_t chunk, uint32_t &s0,
                                            uint32_t &s1, int32_t tree_lo)
{
    if constexpr (TREE) {
        const int32_t first = first_key(s, window);
        s0 = s.len == 0 ? 0 : (uint32_t)(min(tree_lo, max(s.len - s.n, 0)) - first) / chunk;
        s1 = s.len == 0 ? 0 : (uint32_t)(s.len - 1 - first) / chunk + 1;
        return;
    }
    int32_t lo, hi;
    visible(p, window, lo, hi);
    const int32_t first = first_key(s, window);
    s0 = hi < 0 ? 0 : (uint32_t)(lo - first) / chunk;
    s1 = hi < 0 ? 0 : (uint32_t)(hi - first) / chunk + 1;
}

// Every parts-th chunk of row r from s0 + part on, four in flight (eight of a
// launch's own, which come from further away).
template <int D, bool SHARED>
__device__ __forceinline__ void join_chunks(const AttnArgs &a, uint64_t r, uint32_t s0, uint32_t s1, uint32_t part,
                                            uint32_t parts, uint32_t lane, Joined &x)
{
    const uint64_t stride = (uint64_t)a.b.tokens * a.q_heads;
    constexpr int AHEAD = SHARED ? 8 : 4;
    for (uint32_t k = s0 + part; k < s1; k += AHEAD * parts) {
        float2 ml[AHEAD];
        float4 v[AHEAD];
#pragma unroll
        for (int e = 0; e < AHEAD; ++e) {
            const uint64_t at = min(k + e * parts, s1 - 1) * stride + r;
            ml[e] = partial2<SHARED>(reinterpret_cast<const float *>(a.part_ml + at));
            v[e] = partial4<SHARED>(a.part + at * D + lane * 4);
        }
#pragma unroll
        for (int e = 0; e < AHEAD; ++e)
            if (k + e * parts < s1) x.add(ml[e], v[e], a.c2);
    }
}

// ---------------------------------------------------------------------------
// sz_attn_rows: at most 16 NB rows.  A workgroup takes one chunk of one KV
// head's keys; its four waves take 32-key blocks in turn, each with its own
// (m', l, o) and no barrier, and meet in LDS at the end.  K and V go straight
// to registers in 16-byte loads, the next block's issued before the current
// one is used.  Per 32 keys a wave runs NB (2 D/32 + 2 D/16) 16x16x32 products.
//   K, 16 keys at a time: lane (key = lane % 16, g = lane / 16) holds d =
//     32 s + 8 g + 0..7 of step s (FP8: a 16-byte load covers two steps, d =
//     64 i + 16 g + 8 h + 0..7; q is loaded in the same order).
//   S^T: lane (row = lane % 16, g) holds keys 16 b + 4 g + 0..3, b = 0, 1.
//   V: lane (c = lane % 16, g) loads D/16 values of rows 16 b + 4 g + 0..3 at
//     d = c D/16; byte permutes turn its 8 rows x D/16 values into D/16
//     operands of 8 keys each.
// Bound by reading K and V.  Measured (MI355X, 8 KV heads of 128, four query
// heads each, contexts of 8,192; two cards differ by 3 %): 100 sequences in
// BF16 552 us, 6.1 TB/s; 64 in E4M3 194 us, 5.6 TB/s (with three waves a SIMD,
// half of BF16's bytes in flight, and converting); 64 of up to 8,192 119 us,
// 5.1 TB/s, for the chunks that end late.  One context of 64K (4 heads, BF16)
// 24 us and 4.5 to join, 4.7 TB/s: 256 workgroups of 1,024 keys.  The order of
// the loads and the waits that count them carry this: where a wait in the loop
// was for all loads in flight, 32 rows took 89 us instead of 83, and one
// spilled register in it cost 8 %.
// ---------------------------------------------------------------------------
template <int DT, int D>
struct KeyBlock {
    static constexpr uint32_t ES = DT == SZ_BF16 ? 2 : 1;
    static constexpr int KL = D * ES / 64;               // 16-byte loads per 16 keys
    static constexpr int VW = D / 16 * ES / 4;           // dwords per lane and V row
    u32x4 k[2][KL];
    uint32_t v[8][VW];
    uint32_t ks[2], vs[2];                               // scale bytes: of the four keys around the lane's, of its V rows
};

template <int DT, int D>
__device__ __forceinline__ void load_keys(const AttnArgs &a, uint32_t head, const uint32_t (&page)[2], int32_t kb,
                                          KeyBlock<DT, D> &x)
{
    constexpr uint32_t ES = KeyBlock<DT, D>::ES;
    const uint32_t lane = lane_id(), m = lane % 16, g = lane / 16;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint64_t r = row_index(a.c, page[b], 0, head, (uint32_t)(kb + 16 * b) & ((1u << a.c.lg_page) - 1));
        const uint8_t *p = a.c.data + r * (D * ES) + (m * (D * ES) + 16 * g);
#pragma unroll
        for (int i = 0; i < KeyBlock<DT, D>::KL; ++i) x.k[b][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p + 64 * i));
        if constexpr (DT != SZ_BF16) x.ks[b] = *reinterpret_cast<const uint32_t *>(a.c.scales + r + m / 4 * 4);
    }
}

template <int DT, int D>
__device__ __forceinline__ void load_values(const AttnArgs &a, uint32_t head, const uint32_t (&page)[2], int32_t kb,
                                            KeyBlock<DT, D> &x)
{
    constexpr uint32_t ES = KeyBlock<DT, D>::ES;
    const uint32_t lane = lane_id(), m = lane % 16, g = lane / 16;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const uint64_t r0 = row_index(a.c, page[b], 1, head, (uint32_t)(kb + 16 * b) & ((1u << a.c.lg_page) - 1));
        const uint8_t *p = a.c.data + r0 * (D * ES) + (4 * g * (D * ES) + m * (D / 16 * ES));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t off = r * (D * ES);
            if constexpr (KeyBlock<DT, D>::VW == 4) {
                const u32x4 w = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p + off));
#pragma unroll
                for (int e = 0; e < 4; ++e) x.v[4 * b + r][e] = w[e];
            } else if constexpr (KeyBlock<DT, D>::VW == 2) {
                const uint2 w = load_nt(reinterpret_cast<const uint2 *>(p + off));
                x.v[4 * b + r][0] = w.x;
                x.v[4 * b + r][1] = w.y;
            } else {
                x.v[4 * b + r][0] = *reinterpret_cast<const uint32_t *>(p + off);
            }
        }
        if constexpr (DT != SZ_BF16) x.vs[b] = *reinterpret_cast<const uint32_t *>(a.c.scales + r0 + 4 * g);
    }
}

// The k-th of up to kOrdered sequences by length: the longest `fold` first,
// longest in front, then the others, shortest in front; equal lengths, and those
// past 2^23, in their own order.  The largest key that more than k keys reach, bit
// by bit.  No loop: with a block of code in front, sz_attn_rows spilled 13 to 63
// registers.
constexpr uint32_t kOrdered = 256;
__device__ __forceinline__ uint32_t by_length(const PagedBatch &b, uint32_t k, uint32_t fold)
{
    constexpr int EACH = kOrdered / 64;
    int32_t key[EACH];
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
        const uint32_t i = lane_id() + 64 * e;
        const int32_t len = min(max(b.lens[min(i, b.seqs - 1)], 0), (1 << 23) - 1);
        key[e] = i < b.seqs ? len << 8 | (int32_t)(kOrdered - 1 - i) : -1;
    }
    const uint32_t at = k >= fold ? b.seqs - 1 - (k - fold) : k;
    uint32_t found = 0;
#pragma unroll
    for (int bit = 30; bit >= 0; --bit) {
        const uint32_t next = found | 1u << bit;
        uint32_t reach = 0;
#pragma unroll
        for (int e = 0; e < EACH; ++e) reach += (uint32_t)__popcll(__ballot(key[e] >= (int32_t)next));
        found = reach > at ? next : found;
    }
    return kOrdered - 1 - found % kOrdered;
}

template <int DT, int D, int NB, typename Args>
__global__ __launch_bounds__(kAttnThreads, NB == 2 ? 2 : D == 64 ? 4 : 3) void sz_attn_rows(Args a)
{
    constexpr bool TREE = Args::kTree;
    constexpr uint32_t ROWS = 16 * NB;
    constexpr int VD = D / 16;                      // d values of a lane
    constexpr int WAVES = kAttnThreads / 64;
    __shared__ float lds_o[WAVES][ROWS][D + 4];
    __shared__ float2 lds_ml[WAVES][ROWS];
    __shared__ uint32_t lds_last;
    // Of a row of a tree: its first cached key (INT32_MIN if it sees none at all) and the new tokens that it sees, a word
    // of zeros around them.  Every wave writes all of them, so each finds them without a barrier; only masked blocks look.
    constexpr uint32_t NAMED = TREE ? kRowsTokens / 32 + 2 : 1;
    __shared__ int32_t lds_lo[TREE ? ROWS : 1];
    __shared__ uint32_t lds_named[TREE ? ROWS : 1][NAMED];

    const uint32_t head = blockIdx.x % a.c.heads;
    uint32_t unit = blockIdx.x / a.c.heads, row0 = 0;                       // trees: the first of the workgroup's rows
    if constexpr (TREE) {                           // blocks of the same rows beside each other: they read the same keys
        row0 = unit % a.row_blocks * ROWS;
        unit /= a.row_blocks;
    }
    uint32_t seq = unit % a.b.seqs;
    const uint32_t split = unit / a.b.seqs;
    if constexpr (Args::kOrdered) seq = by_length(a.b, seq, a.rows_fold);
    const Sequence s = sequence(a.b, seq);
    const uint64_t all_rows = (uint64_t)s.n * a.group;
    if (TREE ? all_rows <= row0 || all_rows > a.rows_limit : all_rows == 0 || all_rows > min(a.rows_limit, ROWS)) return;
    const uint32_t rows = TREE ? min((uint32_t)all_rows - row0, ROWS) : (uint32_t)all_rows;
    const uint32_t chunks = chunks_of(s, a.window, a.rows_chunk);
    const bool whole = chunks == 1;
    const int64_t begin64 = (int64_t)first_key(s, a.window) + (int64_t)split * a.rows_chunk;
    if (split > 0 && begin64 >= s.len) return;
    const int32_t begin = (int32_t)begin64;
    const int32_t end = (int32_t)min((int64_t)s.len, begin64 + a.rows_chunk);

    const uint32_t lane = lane_id(), wave = uniform(threadIdx.x / 64);
    const uint32_t n = lane % 16, g = lane / 16;
    // Row 16 b + n; one that is not there computes what the last one does.
    const int32_t past = s.len - s.n;
    constexpr int32_t STEP = 32 * WAVES;
    int32_t kb = begin + 32 * (int32_t)wave;
    // The pages of this wave's next 32 blocks, two lanes to a block: one load,
    // so that no block's loads wait for its page number.  Positions behind the
    // end take the last one's page; their keys are hidden.
    uint32_t ahead = 0, at = 0;
    const auto look_ahead = [&](int32_t from) {
        ahead = page_of(a.c, a.b, seq,
                        (uint32_t)min((int64_t)from + (int64_t)(lane / 2) * STEP + 16 * (lane % 2), (int64_t)s.len - 1));
        at = 0;
    };
    if constexpr (TREE) {
        if (kb < end) look_ahead(kb);               // on its way beside the masks
#pragma unroll 1                                    // one row of a lane after another: the registers are q's
        for (int b = 0; b < NB; ++b) {
            const int32_t tok = (int32_t)((row0 + min(16 * b + n, rows - 1)) / a.group);
            uint32_t *named = lds_named[16 * b + n];
            int32_t count = 0;
#pragma unroll 1
            for (uint32_t w = 0; w < kRowsTokens / 64; ++w) {
                const uint64_t bits = new_seen(a, s, tok, 64 * (int32_t)w);
                count += (int32_t)__popcll(bits);
                if (g == 0) {
                    named[2 * w + 1] = (uint32_t)bits;
                    named[2 * w + 2] = (uint32_t)(bits >> 32);
                }
            }
            const int32_t first = first_seen(past + max(count, 1) - 1, a.window);
            if (g == 0) {
                lds_lo[16 * b + n] = count == 0 && first >= past ? INT32_MIN : first;
                named[0] = named[NAMED - 1] = 0;
            }
        }
    }
    int32_t lo[NB], hi[NB];
    bf16x8 q[NB][D / 32];                           // the products' second operand, in K's order of d
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const uint32_t r = row0 + min(16 * b + n, rows - 1), tok = r / a.group;
        if constexpr (!TREE) {
            visible(past + (int32_t)tok, a.window, lo[b], hi[b]);
        }
        const uint16_t *p = a.q + (uint64_t)(s.start + tok) * a.q_token + (uint64_t)(head * a.group + r % a.group) * a.q_head;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            q[b][i] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(
                                                     p + (DT == SZ_BF16 ? 32 * i + 8 * g
                                                                        : 64 * (i / 2) + 16 * g + 8 * (i % 2))));
    }

    f32x4 o[NB][VD];
    Reference ref[NB];
    float l[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        l[b] = 0.f;
#pragma unroll
        for (int j = 0; j < VD; ++j) o[b][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    bool far = false;

    const int32_t all_lo = first_seen(s.len - 1, a.window);                  // every row sees [all_lo, all_hi]
    const int32_t all_hi = TREE ? past - 1 : past;

    KeyBlock<DT, D> cur;
    uint32_t page[2];
    const auto next_pages = [&]() {
        page[0] = __builtin_amdgcn_readlane(ahead, at);
        page[1] = __builtin_amdgcn_readlane(ahead, at + 1);
        at += 2;
    };
    // q is here before the first keys are asked for (or no keys are): waits in
    // the loop count the loads behind the ones they wait for.
    const auto have_q = [&]() SZ_INLINE {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < D / 32; ++i) asm volatile("" : "+v"(q[b][i]));
    };
    if (kb < end) {
        if (!TREE) look_ahead(kb);
        next_pages();
        have_q();
        load_keys<DT, D>(a, head, page, kb, cur);
        __builtin_amdgcn_sched_barrier(0);       // keys always before values: a wait for keys leaves values in flight
        load_values<DT, D>(a, head, page, kb, cur);
    } else {
        have_q();
    }
    // One block.  MASKED: some row does not see some key of it; a path of its
    // own, so that the common one has the registers to itself.  more: another
    // block follows; the common path knows, so that its waits can count on the
    // loads behind the ones they wait for.
    const auto block = [&](auto masked_path, auto more) {
        constexpr bool MASKED = decltype(masked_path)::value;

        // scores
        f32x4 st[NB][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int b = 0; b < NB; ++b) st[b][k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                u32x4 w;
                if constexpr (DT == SZ_BF16) {
                    w = cur.k[k][i];
                } else {
                    const uint32_t sc = ((cur.ks[k] >> (8 * (n % 4))) & 0xFFu) << 23;
                    const uint32_t w0 = cur.k[k][i / 2][2 * (i % 2)], w1 = cur.k[k][i / 2][2 * (i % 2) + 1];
                    w = u32x4{fp8_pair_to_bf16<DT, false>(w0, sc), fp8_pair_to_bf16<DT, true>(w0, sc),
                              fp8_pair_to_bf16<DT, false>(w1, sc), fp8_pair_to_bf16<DT, true>(w1, sc)};
                }
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    st[b][k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), q[b][i], st[b][k],
                                                                       0, 0, 0);
            }
        }
        if (more) {
            if (at == 64) look_ahead(kb + STEP);
            next_pages();
            if (!MASKED) load_keys<DT, D>(a, head, page, kb + STEP, cur);
        }

        // V rows as BF16.  FP8 values of the common path take their registers
        // half at a time, the second half's after the first one's products.
        constexpr bool HALVES = DT != SZ_BF16 && !MASKED;
        uint32_t v[8][VD / 2];
        const auto convert = [&](int first, int last) SZ_INLINE {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                if constexpr (DT == SZ_BF16) {
#pragma unroll
                    for (int e = first; e < last; ++e) v[r][e] = cur.v[r][e];
                } else {
                    const uint32_t sc = ((cur.vs[r / 4] >> (8 * (r % 4))) & 0xFFu) << 23;
#pragma unroll
                    for (int e = first; e < last; ++e)
                        v[r][e] = e % 2 ? fp8_pair_to_bf16<DT, true>(cur.v[r][e / 2], sc)
                                        : fp8_pair_to_bf16<DT, false>(cur.v[r][e / 2], sc);
                }
            }
        };
        convert(0, HALVES ? VD / 4 : VD / 2);

        // Hidden keys: their scores are -inf whatever K holds; V rows that no
        // row sees (behind the end, before the window) become zeros, since 0
        // times a NaN is one.  NaN and infinities in the others are counted
        // further down.
        bool wild = false;
        uint32_t sees[NB];                           // trees: bit j, key kb + 4 g + j
        if constexpr (MASKED) {
            uint32_t found = 0;
            const int32_t any_lo = first_seen(past, a.window);
            if constexpr (TREE)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint32_t row = 16 * b + opaque(n);
                    const int32_t first = lds_lo[row], at = kb - past;            // at: the new token of bit 0
                    const int32_t from = max(first - kb, 0), end = first == INT32_MIN ? 0 : min(-at, 32);
                    uint32_t bits = from < end ? (~0u >> (32 - (end - from))) << from : 0u;
                    if (at > -32 && at < (int32_t)kRowsTokens) {
                        const uint32_t *named = lds_named[row] + ((at >> 5) + 1);
                        bits |= __builtin_amdgcn_alignbit(named[1], named[0], (uint32_t)at & 31);
                    }
                    sees[b] = bits >> (4 * g);
                }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int32_t key = kb + 16 * (r / 4) + 4 * (int32_t)g + r % 4;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    if constexpr (TREE) {
                        if ((sees[b] >> (16 * (r / 4) + r % 4) & 1) == 0) st[b][r / 4][r % 4] = kNone;
                    } else {
                        if (key < lo[b] || key > hi[b]) st[b][r / 4][r % 4] = kNone;
                    }
                }
                const bool dead = key < any_lo || key >= s.len;
#pragma unroll
                for (int e = 0; e < VD / 2; ++e) {
                    if (dead) v[r][e] = 0;
                    found |= not_finite(v[r][e]);
                }
            }
            wild = __any((found & kNotFinite) != 0);
        }

        // running maxima, raised only when some row needs it
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float top = kNone;
#pragma unroll
            for (int r = 0; r < 8; ++r) top = fmaxf(top, st[b][r / 4][r % 4]);
            if (__any(ref[b].below(top, a.c2))) {
                top = fmaxf(top, __shfl_xor(top, 16, 64));
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                const float f = ref[b].raise(top, a.c2);
                far = __any(ref[0].is_far(a.c2) || ref[NB - 1].is_far(a.c2));
                l[b] *= f;
#pragma unroll
                for (int j = 0; j < VD; ++j) o[b][j] *= f;
            }
        }
        bf16x8 pb[NB], pr[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (far)
#pragma unroll
                for (int r = 0; r < 8; ++r) st[b][r / 4][r % 4] -= ref[b].origin();
            const float base = ref[b].base(a.c2, far);
            float p[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                p[r] = exp2_fast(__builtin_fmaf(st[b][r / 4][r % 4], a.c2, -base));
                l[b] += p[r];
            }
            // Their upper 16 bits, and the rest in a second product: products
            // are cheap beside the reads (0 to 1 % of the time), and the result
            // is as exact as its own rounding.  Where every row sees every key
            // the rest of a probability above 0 (2^-126 at least) is 2^-133 at
            // least (BF16's smallest): 0 times an infinite value is a NaN.  A
            // probability of 0 has no rest: its value does not count.
            u32x4 pw, rw;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float rest[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float x = p[2 * e + h];
                    rest[h] = x - __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & 0xFFFF0000u);
                    if constexpr (!MASKED) rest[h] = __builtin_amdgcn_fmed3f(rest[h], x, 0x1p-133f);   // max(rest, min(x, ..))
                }
                pw[e] = perm(__builtin_bit_cast(uint32_t, p[2 * e + 1]), __builtin_bit_cast(uint32_t, p[2 * e]),
                             0x07060302u);
                rw[e] = bf16_pair(rest[0], rest[1]);
            }
            pb[b] = __builtin_bit_cast(bf16x8, pw);
            pr[b] = __builtin_bit_cast(bf16x8, rw);
        }

        if (MASKED && wild) {
            const int32_t key = kb + 4 * (int32_t)g;
            u32x4 sw[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b)
                sw[b] = TREE ? u32x4{seen_pair(sees[b]), seen_pair(sees[b] >> 2), seen_pair(sees[b] >> 16),
                                     seen_pair(sees[b] >> 18)}
                             : u32x4{seen_pair(key, lo[b], hi[b]), seen_pair(key + 2, lo[b], hi[b]),
                                     seen_pair(key + 16, lo[b], hi[b]), seen_pair(key + 18, lo[b], hi[b])};
            uint32_t even = 0x05040100u;
            asm volatile("" : "+s"(even));       // these permutes are not shared with the ones below, which would
#pragma unroll                                   // keep all of them in registers
            for (int j = 0; j < VD; ++j) {
                const uint32_t sel = even + (j % 2 ? 0x02020202u : 0u);
                const u32x4 w = {kinds(perm(v[1][j / 2], v[0][j / 2], sel)), kinds(perm(v[3][j / 2], v[2][j / 2], sel)),
                                 kinds(perm(v[5][j / 2], v[4][j / 2], sel)), kinds(perm(v[7][j / 2], v[6][j / 2], sel))};
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const f32x4 c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, sw[b]), f32x4{0.f, 0.f, 0.f, 0.f}, 0,
                        0, 0);
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[b][j][r] += from_kinds(c[r]);
                }
            }
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int e = 0; e < VD / 2; ++e) v[r][e] = finite(v[r][e]);
        }
#pragma unroll
        for (int j = 0; j < VD; ++j) {
            if (HALVES && j == VD / 2) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int r = 0; r < 8; ++r)
#pragma unroll
                    for (int e = VD / 8; e < VD / 4; ++e) asm volatile("" : "+v"(cur.v[r][e]));
                convert(VD / 4, VD / 2);
            }
            const uint32_t sel = j % 2 ? 0x07060302u : 0x05040100u;
            const u32x4 w = {perm(v[1][j / 2], v[0][j / 2], sel), perm(v[3][j / 2], v[2][j / 2], sel),
                             perm(v[5][j / 2], v[4][j / 2], sel), perm(v[7][j / 2], v[6][j / 2], sel)};
#pragma unroll
            for (int b = 0; b < NB; ++b)
                o[b][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), pb[b], o[b][j], 0, 0, 0);
#pragma unroll
            for (int b = 0; b < NB; ++b)
                o[b][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), pr[b], o[b][j], 0, 0, 0);
        }
        if (more) {
            if (MASKED) {
                load_keys<DT, D>(a, head, page, kb + STEP, cur);
                __builtin_amdgcn_sched_barrier(0);
            }
            load_values<DT, D>(a, head, page, kb + STEP, cur);
        }
    };
    while (kb < end) {
        for (; kb + STEP < end && kb >= all_lo && kb + 31 <= all_hi; kb += STEP)
            block(std::false_type{}, std::true_type{});
        block(std::true_type{}, kb + STEP < end);
        kb += STEP;
    }

    // the waves' sums meet in LDS
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        l[b] += __shfl_xor(l[b], 16, 64);
        l[b] += __shfl_xor(l[b], 32, 64);
        const float plain = exp2_fast(-ref[b].delta);   // to sums with m' itself as the reference
        if (g == 0) lds_ml[wave][16 * b + n] = make_float2(ref[b].top, l[b] * plain);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < VD; j += 4)
                *reinterpret_cast<float4 *>(&lds_o[wave][16 * b + n][(4 * g + r) * VD + j]) =
                    make_float4(o[b][j][r] * plain, o[b][j + 1][r] * plain, o[b][j + 2][r] * plain,
                                o[b][j + 3][r] * plain);
    }
    __syncthreads();
    // 256 threads, each VD values of one row of 16
    const uint32_t d = threadIdx.x % 16 * VD;
    for (uint32_t row = threadIdx.x / 16; row < rows; row += 16) {
        float top = kNone, sum = 0.f, acc[VD];
#pragma unroll
        for (int w = 0; w < WAVES; ++w) top = fmaxf(top, lds_ml[w][row].x);
#pragma unroll
        for (int j = 0; j < VD; ++j) acc[j] = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float2 ml = lds_ml[w][row];
            const float f = rebased(ml.x, top, a.c2);
            sum += ml.y * f;
#pragma unroll
            for (int j = 0; j < VD; ++j) acc[j] += lds_o[w][row][d + j] * f;
        }
        const uint32_t rtok = (row0 + row) / a.group, rhead = head * a.group + (row0 + row) % a.group;
        const bool empty = TREE ? lds_lo[row] == INT32_MIN : past + (int32_t)rtok < 0;
        store_row<D, VD>(a, whole, split, s.start + rtok, rhead, d, acc, empty ? 0.f : 1.f / sum);
        if (d == 0) store_stats(a, whole, split, s.start + rtok, rhead, empty, top, sum);
    }
    if (whole || a.arrived == nullptr) return;

    // The last chunk's workgroup to get here joins them.  Each has its
    // partials where all see them (publish, the wait and the barrier) before
    // it counts itself, and the last one's count wraps to 0 for the next call.
    // The order of the sums is that of the chunks, whichever comes last.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0)
        lds_last = atomicInc(a.arrived + (TREE ? blockIdx.x - (uint64_t)split * a.b.seqs * a.c.heads * row_blocks(a)
                                                : (uint64_t)seq * a.c.heads + head), chunks - 1) == chunks - 1;
    __syncthreads();
    if (!lds_last) return;
    constexpr uint32_t LANES = D / 4, GROUPS = kAttnThreads / LANES;
    float4(*meet_o)[LANES] = reinterpret_cast<float4(*)[LANES]>(&lds_o[0][0][0]);
    float2 *meet_ml = &lds_ml[0][0];
    uint32_t parts = GROUPS;                        // groups of lanes to a row
    while (parts > 1 && GROUPS / parts < rows) parts /= 2;
    const uint32_t lanes_group = threadIdx.x / LANES, jlane = threadIdx.x % LANES, part = lanes_group % parts;
    for (uint32_t r0 = 0; r0 < rows; r0 += GROUPS / parts) {
        const uint32_t r = r0 + lanes_group / parts;
        const uint32_t jtok = (row0 + r) / a.group, jhead = head * a.group + (row0 + r) % a.group;
        const int32_t jpos = past + (int32_t)jtok, jlo = TREE ? lds_lo[min(r, rows - 1)] : 0;
        const bool empty = TREE ? jlo == INT32_MIN : jpos < 0;
        Joined x;
        if (r < rows && !(TREE && empty)) {
            uint32_t s0, s1;
            chunk_range<TREE>(s, jpos, a.window, a.rows_chunk, s0, s1, jlo);
            join_chunks<D, true>(a, (uint64_t)(s.start + jtok) * a.q_heads + jhead, s0, s1, part, parts, jlane, x);
        }
        __syncthreads();
        meet_o[lanes_group][jlane] = x.o;
        if (jlane == 0) meet_ml[lanes_group] = make_float2(x.m, x.l);
        __syncthreads();
        if (r < rows && part == 0) {
            for (uint32_t k = 1; k < parts; ++k) x.add(meet_ml[lanes_group + k], meet_o[lanes_group + k][jlane], a.c2);
            const float w[4] = {x.o.x, x.o.y, x.o.z, x.o.w};
            store_row<D, 4>(a, true, 0, s.start + jtok, jhead, jlane * 4, w, empty ? 0.f : 1.f / x.l);
            if (jlane == 0) store_stats(a, true, 0, s.start + jtok, jhead, empty, x.m, x.l);
        }
    }
}

// ---------------------------------------------------------------------------
// sz_attn_tiles: 32 WAVES rows of one KV head, a wave 32 of them, over 64-key
// tiles in LDS, two tiles deep.  BF16 tiles go from HBM to LDS without
// registers (16 bytes a lane, whole rows; the lane picks which 16 bytes of
// the row it fetches so that the LDS reads meet no bank twice); FP8 tiles
// pass through registers, where one instruction converts and scales two
// values, once for all waves.  Products are 32x32x16: K rows from LDS as
// 16-byte reads, V transposed on the way out of LDS.
//   S^T: lane (row = lane % 32, g = lane / 32) holds keys 32 b + 8 i + 4 g +
//     0..3, b = 0, 1, i = 0..3.
// Bound by the matrix unit with the vector unit's powers beside it: of a
// tile's 4,400 cycles of a SIMD, which two waves share, 2,048 are products and
// 2,150 issue vector instructions, and a wave's own order keeps them apart
// (counters; 256 registers leave no third wave).  Measured (MI355X, 8 KV heads
// of 128, 32 query heads): 2,048 tokens over 16,384 in E5M2 541 us, 1,080
// TFLOP/s (534 to 559 on several cards); six BF16 prompts of up to 4,096 tokens
// 366 us, 914 TFLOP/s, 15 % of it the workgroups' starts.
// ---------------------------------------------------------------------------
// 16-byte pieces of a row are stored at piece ^ swizzle(row), so that 16 lanes
// meet no bank twice: K reads take the same piece of 32 rows, V reads four
// pieces of each of 8 rows, FP8 tiles' writes four pieces, D / 32 apart, of
// each of 16 rows.
template <int D>
__device__ __forceinline__ uint32_t k_swizzle(uint32_t row)
{
    return D == 128 ? row & 15u : (row >> 1) & 7u;
}
template <int D>
__device__ __forceinline__ uint32_t v_swizzle(uint32_t row)
{
    return D == 128 ? (row & 3u) * 5 : ((row >> 1) & 1u) * 5;
}

template <int D>
struct TileLds {
    uint16_t k[2][kTileKeys * D];
    uint16_t v[2][kTileKeys * D];
    uint32_t wild;
};

template <int D, int KV>
__device__ __forceinline__ uint32_t tile_swizzle(uint32_t row)
{
    return KV == 0 ? k_swizzle<D>(row) : v_swizzle<D>(row);
}

// Memory of the workgroup, known as such.
typedef __attribute__((address_space(3))) uint16_t *LdsPtr;

// A wave fetches ROWS = 64 / WAVES rows of a tile's K (KV = 0) and V: part of
// one page.  BF16: PARTS loads straight to LDS, through a buffer of the rows
// (unlike a flat load into LDS, a buffer load leaves the waits of the LDS
// reads beside it exact).
template <int D, int KV, int WAVES>
struct FetchBf16 {
    static constexpr uint32_t ROWS = kTileKeys / WAVES, PIECES = D / 8, RPI = 64 / PIECES, PARTS = ROWS / RPI;
#ifdef __HIP_DEVICE_COMPILE__        // the host pass does not know the type, and drops the kernel's second instance over it
    __amdgpu_buffer_rsrc_t rows;
#endif
    __device__ __forceinline__ FetchBf16(const AttnArgs &a, uint32_t head, uint32_t page, int32_t key0)
    {
        const uint32_t row0 = (uint32_t)key0 & ((1u << a.c.lg_page) - 1);
        uint16_t *p = reinterpret_cast<uint16_t *>(a.c.data) + row_index(a.c, page, KV, head, row0) * D;
#ifdef __HIP_DEVICE_COMPILE__
        rows = __builtin_amdgcn_make_buffer_rsrc(p, 0, ROWS * D * 2, 0x00027000);
#else
        (void)p;
#endif
    }
    __device__ __forceinline__ void part(uint32_t wave, uint32_t i, LdsPtr to) const
    {
        const uint32_t r = i * RPI + lane_id() / PIECES;
#ifdef __HIP_DEVICE_COMPILE__
        typedef __attribute__((address_space(3))) void *lds_ptr;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rows, (lds_ptr)(to + (ROWS * wave + i * RPI) * D), 16,
            (r * D + 8 * ((lane_id() % PIECES) ^ tile_swizzle<D, KV>(ROWS * wave + r))) * 2, 0, 0, 0);
#else
        (void)r;
#endif
    }
};

// FP8: lane l of wave w loads D / WAVES bytes of row ROWS w + l / WAVES, and
// places them as BF16 later, eight values (one LDS write) at a time.
template <int DT, int D, int KV, int WAVES>
struct FetchFp8 {
    static constexpr uint32_t ROWS = kTileKeys / WAVES, PARTS = D / WAVES / 8;
    uint32_t x[2 * PARTS], scale;
    __device__ __forceinline__ void load(const AttnArgs &a, uint32_t head, uint32_t page, int32_t key0)
    {
        const uint32_t r = lane_id() / WAVES, piece = lane_id() % WAVES;
        const uint32_t row0 = (uint32_t)key0 & ((1u << a.c.lg_page) - 1);
        const uint64_t first = row_index(a.c, page, KV, head, row0);
        const uint8_t *p = a.c.data + first * D + (r * D + piece * (D / WAVES));
        if constexpr (PARTS == 1) {
            const uint2 w = *reinterpret_cast<const uint2 *>(p);
            x[0] = w.x;
            x[1] = w.y;
        } else {
#pragma unroll
            for (uint32_t i = 0; i < PARTS / 2; ++i) {
                const u32x4 w = *reinterpret_cast<const u32x4 *>(p + 16 * i);
#pragma unroll
                for (uint32_t e = 0; e < 4; ++e) x[4 * i + e] = w[e];
            }
        }
        scale = *reinterpret_cast<const uint32_t *>(a.c.scales + first + r / 4 * 4);
    }
    __device__ __forceinline__ void place(uint32_t wave, uint32_t i, LdsPtr to) const
    {
        const uint32_t row = ROWS * wave + lane_id() / WAVES, c = lane_id() % WAVES * PARTS + i;
        const uint32_t s = ((scale >> (8 * (row % 4))) & 0xFFu) << 23;
        typedef __attribute__((address_space(3))) u32x4 *lds_ptr;
        *(lds_ptr)(to + row * D + 8 * (c ^ tile_swizzle<D, KV>(row))) =
            u32x4{fp8_pair_to_bf16<DT, false>(x[2 * i], s), fp8_pair_to_bf16<DT, true>(x[2 * i], s),
                  fp8_pair_to_bf16<DT, false>(x[2 * i + 1], s), fp8_pair_to_bf16<DT, true>(x[2 * i + 1], s)};
    }
};

// The places that a lane reads differ between the pieces of a row by an
// exclusive or of constants, and between rows by constants: one register
// holds them all; opaque() keeps the compiler from holding each.

// K of 32 keys as the first operand: key 32 b + lane % 32, d = 16 i + 8 g + 0..7.
template <int D>
__device__ __forceinline__ uint32_t k_place()
{
    const uint32_t row = lane_id() % 32, g = lane_id() / 32;
    return (row * D + 8 * (g ^ k_swizzle<D>(row))) * 2;
}
template <int D>
__device__ __forceinline__ bf16x8 k_operand(LdsPtr k, uint32_t place, int b, int i)
{
    typedef __attribute__((address_space(3))) const u32x4 *lds_ptr;
    return __builtin_bit_cast(bf16x8, *(lds_ptr)(k + ((place ^ (32 * i)) / 2 + 32 * b * D)));
}

// V^T of 16 keys and 32 d as the first operand: keys base + 4 g + 0..3 and
// base + 8 + 4 g + 0..3 of d = 32 j + lane % 32.  Each 16 lanes of a
// transposing read take 4 rows x 16 d.
template <int D>
__device__ __forceinline__ uint32_t v_place()
{
    const uint32_t lane = lane_id(), i = lane % 16, g = lane / 32, half = lane / 16 % 2;
    const uint32_t row = 4 * g + i / 4, col = 16 * half + 4 * (i % 4);
    return (row * D + 8 * ((col / 8) ^ v_swizzle<D>(row)) + col % 8) * 2;
}
template <int D>
__device__ __forceinline__ bf16x8 v_operand(LdsPtr v, uint32_t place, uint32_t base, int j)
{
    typedef __attribute__((address_space(3))) s16x4 *lds_ptr;
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    const uint32_t at = (place ^ (64 * j)) / 2 + base * D;
    const s16x4 w0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(v + at));
    const s16x4 w1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(v + at + 8 * D));
    return __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(w0, w1, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <int DT, int D, int WAVES, typename Args>
__global__ __launch_bounds__(64 * WAVES, 2) void sz_attn_tiles(Args a, uint32_t slots)
{
    constexpr bool TREE = Args::kTree;
    constexpr int DB = D / 32;
    constexpr uint32_t kTileRows = 32 * WAVES, ROWS = kTileKeys / WAVES;
    __shared__ TileLds<D> lds;
    // Of a row of a tree: its token and first cached key (INT32_MIN if it sees none at all).  A wave writes and reads its
    // own.  FP8 only, whose conversion wants the registers; where loads go to LDS by themselves (BF16), reading other LDS
    // would wait for them (301 us for 145, 64 sequences of up to 4,000, 120 rows).
    constexpr bool IN_LDS = TREE && DT != SZ_BF16;
    __shared__ int32_t lds_tok[IN_LDS ? kTileRows : 1], lds_lo[IN_LDS ? kTileRows : 1];

    const uint32_t head = blockIdx.x % a.c.heads;
    uint32_t slot = slots - 1 - blockIdx.x / a.c.heads % slots;                // later tiles see more keys: first
    if constexpr (TREE)
        if (a.fold) {
            const uint32_t back = slots - 1 - slot;
            slot = by_length(a.b, back / a.tiles_each, a.fold) * a.tiles_each + (a.tiles_each - 1 - back % a.tiles_each);
        }
    const uint32_t split = blockIdx.x / a.c.heads / slots;

    // Where all sequences may have as many rows, sequence i owns the slots from
    // i tiles_each on; else those from floor(starts[i] G / rows) + i on: at
    // least as many as its rows fill.  (One sequence after another: the heads
    // of one XCD then read the same keys out of its L2.  The longest tiles of
    // all sequences first measured 445 us where this took 385.)
    const auto first_slot = [&](uint32_t i) {
        if constexpr (TREE)
            if (a.tiles_each) return (int64_t)i * a.tiles_each;
        return (int64_t)(((uint64_t)(uint32_t)max(a.b.starts[i], 0) * a.group) / kTileRows) + i;
    };
    const int32_t found = [&]() {
        if constexpr (TREE)
            if (a.tiles_each) return (int32_t)(slot / a.tiles_each);
        return wave_last_not_above(a.b.seqs, slot, first_slot);
    }();
    if (found < 0) {                                                           // before the first sequence's slots
        if (a.b.starts[0] > (int32_t)a.b.tokens) flag_batch(a.b);              // which may own none
        return;
    }
    const uint32_t seq = uniform((uint32_t)found);
    const Sequence s = sequence(a.b, seq);
    const uint64_t all_rows = (uint64_t)s.n * a.group;
    if (all_rows <= a.rows_limit) return;                                      // none, or sz_attn_rows takes them
    const uint64_t row0 = (uint64_t)(slot - first_slot(seq)) * kTileRows;
    if (row0 >= all_rows) return;
    const uint32_t rows = (uint32_t)min((uint64_t)kTileRows, all_rows - row0);

    const uint32_t lane = lane_id(), wave = uniform(threadIdx.x / 64);
    const uint32_t n = lane % 32, g = lane / 32;
    const int32_t tok_first = (int32_t)(row0 / a.group), tok_last = (int32_t)((row0 + rows - 1) / a.group);
    const uint64_t my_row = row0 + min(wave * 32 + n, rows - 1);
    const bool mine = wave * 32 + n < rows;
    const int32_t tok = (int32_t)(my_row / a.group);
    const uint32_t q_head = head * a.group + (uint32_t)(my_row % a.group);
    const int32_t past = s.len - s.n, pos = past + tok;
    int32_t lo, hi;
    bool empty = pos < 0;
    if constexpr (TREE) {
        const Sight v = tree_sight(a, s, tok);
        lo = v.blind ? INT32_MIN : v.lo;
        if (IN_LDS && g == 0) {
            lds_tok[wave * 32 + n] = tok;
            lds_lo[wave * 32 + n] = lo;
        }
    } else {
        visible(pos, a.window, lo, hi);
    }

    // the keys of this tile of rows, and of its chunk: every row sees the ones up to p_first, none one behind p_last
    const int32_t p_first = TREE ? past - 1 : past + tok_first, p_last = TREE ? s.len - 1 : past + tok_last;
    const bool whole = a.tile_splits == 1 || chunks_of(s, a.window, a.tile_chunk) == 1;
    const int64_t chunk0 = (int64_t)first_key(s, a.window) + (int64_t)split * a.tile_chunk;
    const int32_t any_lo = first_seen(TREE ? past : p_first, a.window);        // some row may see [any_lo, p_last]
    const int32_t begin = (int32_t)max(chunk0, (int64_t)(any_lo & ~(int32_t)(kTileKeys - 1)));
    const int32_t end = (int32_t)min((int64_t)p_last + 1, chunk0 + a.tile_chunk);
    if (whole ? split > 0 : begin >= end) return;                              // no row's chunk: nobody reads it
    const int32_t all_lo = first_seen(p_last, a.window);                       // every row sees [all_lo, p_first]

    bf16x8 q[D / 16];               // a row that is not there computes what the last one does, and stores nothing
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
        q[i] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4 *>(a.q + (uint64_t)(s.start + tok) * a.q_token +
                                                                           (uint64_t)q_head * a.q_head + 16 * i + 8 * g));

    f32x16 o[DB];
#pragma unroll
    for (int j = 0; j < DB; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[j][r] = 0.f;
    Reference ref;
    bool far = false;
    float l = 0.f;

    // A wave's part of a tile is of one page.  The pages of 64 tiles, a lane
    // each, in one load; V follows K by two tiles.  Rows behind the sequence's
    // end come from its last page and are hidden.
    uint32_t ahead = 0, before = 0;
    const auto look_ahead = [&](uint32_t tile) SZ_INLINE {
        before = ahead;
        ahead = page_of(a.c, a.b, seq,
                        (uint32_t)min((int64_t)begin + ((int64_t)tile + lane) * kTileKeys + ROWS * wave,
                                      (int64_t)s.len - 1));
    };
    const uint32_t tiles = begin < end ? (uint32_t)(end - begin + (int32_t)kTileKeys - 1) / kTileKeys : 0;
    const auto first_of = [&](uint32_t t) SZ_INLINE { return begin + (int32_t)(t * kTileKeys + ROWS * wave); };
    // Every wave's part of what was fetched is in LDS, and what was read is free.
    const auto meet = [&]() SZ_INLINE {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    };

    const uint32_t k_at = k_place<D>(), v_at = v_place<D>();
    f32x16 st[2];
    const auto scores = [&](LdsPtr k, int b) SZ_INLINE {                               // of 32 keys
        const uint32_t place = opaque(k_at);
#pragma unroll
        for (int r = 0; r < 16; ++r) st[b][r] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            st[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k_operand<D>(k, place, b, i), q[i], st[b],
                                                            0, 0, 0);
    };
    const auto masked = [&](uint32_t t) SZ_INLINE {
        const int32_t kb = begin + (int32_t)(t * kTileKeys);
        return kb < all_lo || kb + (int32_t)kTileKeys - 1 > p_first;
    };
    // Trees: the keys of the tile at kb that the lane's row sees, from its own first four on.
    const auto tree_seen = [&](int32_t kb) SZ_INLINE {
        const int32_t first = IN_LDS ? lds_lo[wave * 32 + n] : lo;
        if (first == INT32_MIN) return (uint64_t)0;
        if constexpr (TREE)
            return (old_seen(first, past, kb) | new_seen(a, s, IN_LDS ? lds_tok[wave * 32 + n] : tok, kb - past)) >> (4 * g);
        return (uint64_t)0;
    };
    // Hides tile t's scores and raises the running maximum.  The sums of the
    // tile before are not in o yet when it rises: o is scaled after them.
    float late = 1.f;
    bool scale_late = false;
    float top0 = kNone;                                                        // of the first 32 keys, not hidden
    const auto settle = [&](uint32_t t) SZ_INLINE {
        float top = top0;
        if (masked(t)) {
            const int32_t kb = begin + (int32_t)(t * kTileKeys);
            uint64_t sees = 0;
            if constexpr (TREE) sees = tree_seen(kb);
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int32_t at = 32 * b + 8 * (r / 4) + r % 4, k = kb + at + 4 * (int32_t)g;
                    if (TREE ? (sees >> at & 1) == 0 : k < lo || k > hi) st[b][r] = kNone;
                }
            top = kNone;
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, st[0][r]);
        }
        float top1 = kNone;
#pragma unroll
        for (int r = 0; r < 16; ++r) top1 = fmaxf(top1, st[1][r]);
        top = fmaxf(top, top1);
        scale_late = __any(ref.below(top, a.c2));
        if (scale_late) {
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            late = ref.raise(top, a.c2);
            far = __any(ref.is_far(a.c2));
            l *= late;
        }
        if (far)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 16; ++r) st[b][r] -= ref.origin();
    };
    bf16x8 p[2][2];                                                            // probabilities, the second operand
    const auto values = [&](LdsPtr v, int b) SZ_INLINE {
        const uint32_t place = opaque(v_at);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < DB; ++j)
                o[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    v_operand<D>(v, place, 32 * b + 16 * k, j), p[b][k], o[j], 0, 0, 0);
    };
    const auto scale_sums = [&]() SZ_INLINE {
        if (scale_late)
#pragma unroll
            for (int j = 0; j < DB; ++j) o[j] *= late;
    };
    // V of a tile that some row does not see all of: rows that none sees
    // become zeros in LDS (0 times a NaN is one); NaN and infinities in the
    // others are counted and taken out.
    const auto clear_hidden = [&](uint32_t t) SZ_INLINE {
        const int32_t kb = begin + (int32_t)(t * kTileKeys);
        uint16_t *vt = lds.v[t % 2];
        constexpr int PIECES = D / WAVES / 8;                                  // 16 bytes each, of a lane
        if (threadIdx.x == 0) lds.wild = 0;
        __syncthreads();
        const int32_t key = kb + (int32_t)(threadIdx.x / WAVES);
        const bool dead = key < any_lo || key > p_last;
        u32x4 *mine4 = reinterpret_cast<u32x4 *>(vt + threadIdx.x / WAVES * D + threadIdx.x % WAVES * (D / WAVES));
        uint32_t found = 0;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            if (dead) {
                mine4[i] = u32x4{0, 0, 0, 0};
            } else {
                const u32x4 w = mine4[i];
                found |= not_finite(w[0]) | not_finite(w[1]) | not_finite(w[2]) | not_finite(w[3]);
            }
        }
        if (found & kNotFinite) lds.wild = 1;
        __syncthreads();
        if (lds.wild == 0) return;
#pragma unroll 1
        for (int j = 0; j < DB; ++j) {
            f32x16 c;
#pragma unroll
            for (int r = 0; r < 16; ++r) c[r] = 0.f;
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                const int32_t at = kb + 16 * k + 4 * (int32_t)g;
                u32x4 sw;
                if constexpr (TREE) {
                    const uint64_t sees = tree_seen(kb) >> (16 * k);
                    sw = u32x4{seen_pair(sees), seen_pair(sees >> 2), seen_pair(sees >> 8), seen_pair(sees >> 10)};
                } else {
                    sw = u32x4{seen_pair(at, lo, hi), seen_pair(at + 2, lo, hi), seen_pair(at + 8, lo, hi),
                               seen_pair(at + 10, lo, hi)};
                }
                u32x4 w = __builtin_bit_cast(u32x4, v_operand<D>((LdsPtr)vt, v_at, 16 * k, j));
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = kinds(w[e]);
                c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w),
                                                            __builtin_bit_cast(bf16x8, sw), c, 0, 0, 0);
            }
#pragma unroll
            for (int jj = 0; jj < DB; ++jj)
                if (jj == j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[jj][r] += from_kinds(c[r]);
        }
        __syncthreads();                                                       // every wave has counted
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const u32x4 w = mine4[i];
            mine4[i] = u32x4{finite(w[0]), finite(w[1]), finite(w[2]), finite(w[3])};
        }
        __syncthreads();
    };

    // Tile t's probabilities are worked out (vector unit) beside tile t - 1's
    // values and tile t + 1's scores (matrix unit): V is needed one tile
    // behind and K one ahead, and each is fetched the iteration before, into
    // the half that the iteration before that has read.  The order is laid
    // down here, one product to a slot with its share of the vector work (28
    // cycles an element, 32 a product), the LDS read of three slots on and,
    // every other slot, a load of the tiles to come: values first, since the
    // scores take the registers of the old ones.  FP8 tiles, loaded in the
    // first slots, are converted in the last ones, which have no
    // probabilities.  The last iterations' scores, and what they fetch beyond
    // the last tile, are unused.
    // (The four halves are named, and told apart by __restrict__, so that no
    // read waits for the loads into the others.)
    const auto beside = [&](uint32_t t, LdsPtr __restrict__ k_to, LdsPtr __restrict__ v_to,
                            LdsPtr __restrict__ k_from, LdsPtr __restrict__ v_from) SZ_INLINE {
        const uint32_t tk = min(t + 2, tiles - 1);
        if (tk == t + 2 && tk % 64 == 0) look_ahead(tk);
        const uint32_t k_page = __builtin_amdgcn_readlane(ahead, tk % 64);
        const uint32_t v_page = __builtin_amdgcn_readlane(tk / 64 == t / 64 ? ahead : before, t % 64);
        constexpr int V_SLOTS = 4 * DB, K_SLOTS = D / 16, SLOTS = V_SLOTS + 2 * K_SLOTS, AHEAD = 3;
        const uint32_t kp = opaque(k_at), vp = opaque(v_at);
        const auto operand = [&](int slot) SZ_INLINE {
            if (slot < V_SLOTS) return v_operand<D>(v_from, vp, 16 * (slot / DB), slot % DB);
            return k_operand<D>(k_from, kp, (slot - V_SLOTS) / K_SLOTS, (slot - V_SLOTS) % K_SLOTS);
        };
        const float base = ref.base(a.c2, far);
        __builtin_amdgcn_s_setprio(1);                                         // before a wave that settles or fetches
        uint32_t next[16];
        float even = 0.f;
        bf16x8 ring[AHEAD + 1];
        using Bf16K = FetchBf16<D, 0, WAVES>;
        using Fp8K = FetchFp8<DT, D, 0, WAVES>;
        const Bf16K bk(a, head, k_page, first_of(tk));
        const FetchBf16<D, 1, WAVES> bv(a, head, v_page, first_of(t));
        Fp8K fk;
        FetchFp8<DT, D, 1, WAVES> fv;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) ring[i] = operand(i);
#pragma unroll
        for (int slot = 0; slot < SLOTS; ++slot) {
            __builtin_amdgcn_sched_barrier(0);
            if (slot + AHEAD < SLOTS) ring[(slot + AHEAD) % (AHEAD + 1)] = operand(slot + AHEAD);
            const bf16x8 x = ring[slot % (AHEAD + 1)];
            if (slot < V_SLOTS) {
                o[slot % DB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, p[slot / DB / 2][slot / DB % 2], o[slot % DB],
                                                                       0, 0, 0);
            } else {
                const int b = (slot - V_SLOTS) / K_SLOTS, i = (slot - V_SLOTS) % K_SLOTS;
                if (i == 0)
#pragma unroll
                    for (int r = 0; r < 16; ++r) st[b][r] = 0.f;
                st[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, q[i], st[b], 0, 0, 0);
            }
            if constexpr (DT == SZ_BF16) {
                const int i = slot / 2;
                if (slot % 2 == 0 && i < (int)Bf16K::PARTS) bk.part(wave, i, k_to);
                if (slot % 2 == 1 && i < (int)Bf16K::PARTS) bv.part(wave, i, v_to);
            } else {
                if (slot == 0) fk.load(a, head, k_page, first_of(tk));
                if (slot == 1) fv.load(a, head, v_page, first_of(t));
                constexpr int PER = (2 * Fp8K::PARTS + K_SLOTS - 1) / K_SLOTS;
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    const int i = (slot - V_SLOTS - K_SLOTS) * PER + e;
                    if (i >= 0 && i < (int)Fp8K::PARTS) fk.place(wave, i, k_to);
                    if (i >= (int)Fp8K::PARTS && i < 2 * (int)Fp8K::PARTS) fv.place(wave, i - Fp8K::PARTS, v_to);
                }
            }
            constexpr int SHARE = V_SLOTS + K_SLOTS;                           // slots with vector work
#pragma unroll
            for (int e = slot * 32 / SHARE; e < (slot + 1) * 32 / SHARE && e < 32; ++e) {
                const float x1 = exp2_fast(__builtin_fmaf(st[e / 16][e % 16], a.c2, -base));
                if (e % 2 == 0) {
                    even = x1;
                } else {
                    l += even + x1;
                    next[e / 2] = bf16_pair(even, x1);
                    asm volatile("" : "+v"(l), "+v"(next[e / 2]));             // worked out here, not where they are used
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(0);
        top0 = kNone;
#pragma unroll
        for (int r = 0; r < 16; ++r) top0 = fmaxf(top0, st[0][r]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i / 2][i % 2] = __builtin_bit_cast(
                bf16x8, (u32x4{next[4 * i], next[4 * i + 1], next[4 * i + 2], next[4 * i + 3]}));
    };
    if (tiles > 0) {
        look_ahead(0);
#pragma unroll
        for (uint32_t t = 0; t < 2; ++t) {                                     // K of the first two tiles
            const uint32_t tk = min(t, tiles - 1);
            const uint32_t page = __builtin_amdgcn_readlane(ahead, tk);
            if constexpr (DT == SZ_BF16) {
                const FetchBf16<D, 0, WAVES> bk(a, head, page, first_of(tk));
#pragma unroll
                for (uint32_t i = 0; i < bk.PARTS; ++i) bk.part(wave, i, (LdsPtr)lds.k[t]);
            } else {
                FetchFp8<DT, D, 0, WAVES> fk;
                fk.load(a, head, page, first_of(tk));
#pragma unroll
                for (uint32_t i = 0; i < fk.PARTS; ++i) fk.place(wave, i, (LdsPtr)lds.k[t]);
            }
        }
        // "the tile before the first": no values, no probabilities
#pragma unroll
        for (int i = 0; i < D / 8 / WAVES; ++i)
            reinterpret_cast<u32x4 *>(lds.v[1])[threadIdx.x + 64 * WAVES * i] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int b = 0; b < 2; ++b) p[b][0] = p[b][1] = __builtin_bit_cast(bf16x8, (u32x4{0, 0, 0, 0}));
        meet();
        scores((LdsPtr)lds.k[0], 0);
        scores((LdsPtr)lds.k[0], 1);
#pragma unroll
        for (int r = 0; r < 16; ++r) top0 = fmaxf(top0, st[0][r]);
        settle(0);
        scale_late = false;                                                    // o is still zero
        __syncthreads();                                                       // every wave has read tile 0: its K's half is free
        uint32_t t = 0;
        while (true) {
            const uint32_t even = t % 2, odd = even ^ 1;
            beside(t, (LdsPtr)lds.k[even], (LdsPtr)lds.v[even], (LdsPtr)lds.k[odd], (LdsPtr)lds.v[odd]);
            scale_sums();
            scale_late = false;
            if (t + 1 < tiles) settle(t + 1);
            meet();
            if (masked(t)) clear_hidden(t);
            if (++t == tiles) break;
        }
        values((LdsPtr)lds.v[(tiles - 1) % 2], 0);
        values((LdsPtr)lds.v[(tiles - 1) % 2], 1);
    }

    l += __shfl_xor(l, 32, 64);
    if (!mine) return;
    if constexpr (TREE) empty = (IN_LDS ? lds_lo[wave * 32 + n] : lo) == INT32_MIN;
    const float plain = exp2_fast(-ref.delta);                                 // to sums with m' itself as the reference
    l *= plain;
    const float inv = whole ? empty ? 0.f : plain / l : plain;
#pragma unroll
    for (int j = 0; j < DB; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float w[4] = {o[j][4 * i] * inv, o[j][4 * i + 1] * inv, o[j][4 * i + 2] * inv, o[j][4 * i + 3] * inv};
            store_row<D, 4>(a, whole, split, s.start + tok, q_head, 32 * j + 8 * i + 4 * g, w, 1.f);
        }
    if (g == 0) store_stats(a, whole, split, s.start + tok, q_head, empty, ref.top, l);
}

// ---------------------------------------------------------------------------
// sz_attn_join: a workgroup joins the chunks of some heads' rows of one token.
// `parts` groups of D/4 lanes take a row, every parts-th of its chunks each,
// four in flight, and meet in LDS, in order.  With per_seq > 0 only sequences
// of sz_attn_rows were split: the grid is their tokens, at most per_seq each;
// else it is all tokens.  Bound by reading the partials: 512 tokens of 32
// heads of 128 in 4 chunks (34 MB) took 29 us with a workgroup to a row, and
// take 9.
// ---------------------------------------------------------------------------
template <int D>
constexpr uint32_t kJoinGroups = kAttnThreads / (D / 4);

template <int D, typename Args>
__global__ __launch_bounds__(kAttnThreads) void sz_attn_join(Args a, uint32_t per_seq, uint32_t parts)
{
    constexpr bool TREE = Args::kTree;
    constexpr uint32_t LANES = D / 4, GROUPS = kJoinGroups<D>;
    __shared__ float4 lds_o[GROUPS][LANES];
    __shared__ float2 lds_ml[GROUPS];
    const uint32_t rows = GROUPS / parts, blocks = (a.q_heads + rows - 1) / rows;
    uint32_t t = blockIdx.x / blocks;
    Sequence s;
    if (per_seq > 0) {
        s = sequence(a.b, t / per_seq);
        const uint32_t i = t % per_seq;
        if (i >= (uint32_t)s.n) return;
        t = (uint32_t)s.start + i;
    } else {
        const int32_t i = wave_last_not_above(a.b.seqs + 1, t, [&](uint32_t j) { return (int64_t)a.b.starts[j]; });
        if (i < 0 || i >= (int32_t)a.b.seqs) return;
        s = sequence(a.b, uniform((uint32_t)i));
        if ((int32_t)t < s.start || (int32_t)t >= s.start + s.n) return;
    }
    const bool few = (uint64_t)s.n * a.group <= a.rows_limit;
    const uint32_t chunk = few ? a.rows_chunk : a.tile_chunk;
    if ((few ? a.rows_splits : a.tile_splits) == 1 || chunks_of(s, a.window, chunk) == 1) return;      // already whole
    const int32_t p = s.len - s.n + ((int32_t)t - s.start);
    uint32_t s0, s1;
    Sight v{0, p < 0};
    if constexpr (TREE) v = tree_sight(a, s, (int32_t)t - s.start);
    chunk_range<TREE>(s, p, a.window, chunk, s0, s1, v.lo);
    const uint32_t group = threadIdx.x / LANES, lane = threadIdx.x % LANES, part = group % parts;
    const uint32_t head = blockIdx.x % blocks * rows + group / parts;
    Joined x;
    if (head < a.q_heads) join_chunks<D, false>(a, (uint64_t)t * a.q_heads + head, s0, s1, part, parts, lane, x);
    if (parts > 1) {
        lds_o[group][lane] = x.o;
        if (lane == 0) lds_ml[group] = make_float2(x.m, x.l);
        __syncthreads();
        if (part == 0)
            for (uint32_t g = 1; g < parts; ++g) x.add(lds_ml[group + g], lds_o[group + g][lane], a.c2);
    }
    if (head >= a.q_heads || part != 0) return;
    const float w[4] = {x.o.x, x.o.y, x.o.z, x.o.w};
    store_row<D, 4>(a, true, 0, t, head, lane * 4, w, v.blind ? 0.f : 1.f / x.l);
    if (lane == 0) store_stats(a, true, 0, t, head, v.blind, x.m, x.l);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
struct AttnPlan {
    bool rows, tiles;                 // which kernels the batch can need
    bool fused;                       // sz_attn_rows joins its chunks itself
    uint32_t tile_waves;
    uint32_t rows_limit;              // of sz_attn_rows
    uint32_t rows_chunk, rows_splits, tile_chunk, tile_splits, slots, tiles_each;
    uint32_t grid_slots;              // that the launch has: slots, or fewer
    uint32_t fold, rows_fold, row_blocks;
    bool row_pairs;                   // two products of rows to a workgroup of sz_attn_rows
};

constexpr uint64_t kMaxThreads = 0xFFFFFFFFull;                // of a launch
// Workgroups that sz_attn_rows wants, but for trees: enough to fill the card (768 run at a
// time, and some chunks are behind their sequence's end), and up to kRowsEven
// while their chunks have kRowsLong keys, to even out lengths.  Against 2,048
// whatever the chunk's length (8 KV heads of 128, four query heads each): 128
// sequences of up to 500 E4M3 tokens 21 us (26), 4 of up to 8,192 21 (25), 100
// of 8,192 in BF16 533 (549), 64 of 8,192 in E4M3 187 (180).  Against 768: 8
// of up to 8,192 22 us (27); against chunks of 2,048: 32 of up to 8,192 66 us
// (76).
constexpr uint64_t kRowsFill = 1024;
constexpr uint64_t kRowsEven = 3328;
constexpr uint64_t kRowsLong = 1024;
// Waves that sz_attn_tiles wants: two a SIMD.  With half, drafts of 16
// sequences (5 tokens, window 1,000, two heads of 64) take 14.9 us instead of
// 13.8; with twice as many nothing changes.
constexpr uint64_t kTileWaves = 2048;
// Keys of a chunk at least: a block for each wave, two tiles.  With 256 those
// drafts take 14.5 us instead of 13.8; 47 sequences of up to 217 tokens, which
// are then hardly cut, 10.5 instead of 12.9.
constexpr uint32_t kMinChunk = 128;
// Chunks of a long context have 1,024 keys at least: 64K tokens take 28.4 us,
// with 512 keys 30.6.
constexpr uint32_t kMaxLeast = 1024;
constexpr uint64_t kArrivals = SZ_ATTENTION_COUNTERS / 4;      // counters at the workspace's start
constexpr uint64_t kJoinChunks = 64;
// Up to so many chunks of a sequence's head, and workgroups in all, are joined
// by the workgroup that ends last, which saves a launch: 1 sequence of 1,001
// tokens 8.8 us (11.8), 1 of 2,001 9.7 (11.0), 4 of up to 2,001 10.8 (12.5), 47
// of up to 217 12.9 (13.5).  The limits are on the high side, and do not look at
// rows: at 24 and 32 chunks the launch is the shorter way again (1 of 3,001 11.6
// for 10.9, 1 of 4,001 12.7 for 11.7, 4 of up to 8,192 21.2 for 19.5), and by
// far where the one workgroup has 32 rows to read (15 of up to 15,241, two heads
// of eight, four tokens each, FP8: 59 us for 33).  With more workgroups their
// writes past the L2 cost more than the launch (64 of up to 8,192 tokens, six
// chunks each: 121 us for 119), with more chunks the one workgroup reads them
// for longer (64K tokens, 64 chunks: 34 us for 28).
constexpr uint32_t kFusedSplits = 32;
constexpr uint64_t kFusedGroups = 1024;
static_assert(kFusedGroups <= kArrivals);

inline uint64_t round_up(uint64_t x, uint64_t to) { return (x + to - 1) / to * to; }

inline uint64_t rows_wanted(uint64_t span, uint64_t groups)
{
    return std::max(kRowsFill / groups, std::min(kRowsEven / groups, span / kRowsLong));
}
// Trees have more rows, whose partials cost more, and every workgroup its start
// (4 to 5 us): no more of them than one a CU.  Over 676 shapes (1 to 200 sequences,
// 500 to 32,000 keys, 4 to 32 rows, every type, lengths equal and not) that takes
// 0.86 of the time of the rule above, 320 as many 0.87, 192 and 384 0.91.  8 KV
// heads of 128, E5M2, 32 rows: 32 sequences of 2,000 30 us (57), 64 of 4,000 95
// (120), and with the longest first (fold_of) 64 of up to 4,000 58 (82); 4 rows in
// BF16, 64 of up to 8,192 186 (210), 4 of up to 30,000 65 (72).  Where neither the
// order nor more chunks even out lengths it is the worse: 4 rows, 16 of up to 8,000
// 75 us (64), in E5M2 42 (37).
constexpr uint64_t kTreeFill = 256;
// Up to so many values of partials are joined in the launch: 8 KV heads of 128,
// E5M2, 4 sequences of 16,000 in 8 chunks, 4 rows 27.6 us (28.6 with a launch), 16
// rows 30.8 (29.0), 32 rows 37.9 (33.4).
constexpr uint64_t kTreeJoin = 1 << 14;
// A chunk's partials cost their way out and back, rows D 8 bytes; its keys are
// the time that the others do not take.  span / n + rows D n / kPartialKeys is
// least at n = sqrt(kPartialKeys span / (rows D)).  BF16, 8 KV heads of 128,
// four query heads each: 512 tokens by themselves then stay whole, 17 us (23
// with 16 times kPartialKeys), 700 take 20 (26); with a quarter 64 tokens
// behind 16,384 take 46 us (41), and with two query heads 64 tokens in each of
// 8 sequences of up to 1,064 27.8 (25.7; with half 24.1).
constexpr double kPartialKeys = 12500;
inline uint64_t tiles_wanted(uint64_t span, uint64_t groups, uint32_t waves, uint64_t values)
{
    return std::min<uint64_t>(kTileWaves / waves / groups, (uint64_t)std::sqrt(kPartialKeys * (double)span / (double)values));
}

// Splits of `span` keys into `want` chunks.  A chunk is not made shorter than
// a 64th of the keys (joining grows with their number) unless that is over
// kMaxLeast.
inline void split_keys(uint64_t span, uint64_t want, uint32_t &chunk, uint32_t &splits)
{
    const uint64_t n = std::max<uint64_t>(1, want);
    const uint64_t least = std::min<uint64_t>(kMaxLeast, round_up((span + kJoinChunks - 1) / kJoinChunks, kMinChunk));
    const uint64_t c = round_up(std::max<uint64_t>({kMinChunk, least, (span + n - 1) / n}), kMinChunk);
    chunk = (uint32_t)c;
    splits = (uint32_t)std::max<uint64_t>(1, (span + c - 1) / c);
}

// No span up to this one gives more chunks than:
inline uint64_t most_splits(uint64_t span, uint64_t want)
{
    return std::min<uint64_t>(std::max<uint64_t>(1, want), (span + kMinChunk - 1) / kMinChunk);
}

// Waves of sz_attn_tiles, 32 rows each.  Eight share one conversion of each
// FP8 tile where four need two: 541 against 557 us for 2,048 E5M2 tokens over
// 16,384 (E4M3 543 and 561), where the rows still fill the card; six E5M2
// prompts of up to 4,096 take 390 and 386.  BF16 tiles need no conversion, and
// eight waves at one barrier are slower (391 against 381 us for six prompts).
inline uint32_t tile_waves(uint32_t dtype, const PagedBatch &b, uint32_t kv_heads, uint32_t group)
{
    const uint64_t rows = (uint64_t)b.tokens * group;
    return dtype != SZ_BF16 && rows >= 256ull * b.seqs && rows * kv_heads >= 256ull * kTileWaves / 8 ? 8 : 4;
}

// Whether sz_attn_rows takes 17 to 32 rows, as two of its products.  8 KV
// heads, FP8: 64 sequences of up to 4,000 tokens, 32 rows, 79 us where
// sz_attn_tiles takes 119, 15 of up to 15,246, 26 rows, 69 (129), with 4 heads
// 60 (74); BF16 with D = 64, 64 of up to 4,000: 73 (80).  Where chunks are
// joined in the launch (kFusedGroups) it is slower: 15 of up to 15,241 of two
// heads, 32 rows, FP8 59 us (43; 33 if a launch joins them), BF16 with D = 64
// 34 (29; 25).  With BF16 and D = 128 its registers leave two waves a SIMD: 15
// of up to 15,241, 32 rows, 8 heads 112 us (135), but 4 heads 88 (71) and 2
// heads 72 (39), and 20 rows over 1,005 tokens 14 (13).  33 to 64 rows in two
// such workgroups gained little or nothing (FP8 58 for 65 us and 38 for 38,
// BF16 90 for 60).
constexpr bool row_pairs(uint32_t dtype, uint32_t head_dim) { return dtype != SZ_BF16 || head_dim == 64; }

// Whether sz_attn_rows takes all rows of a batch of trees, 16 of them to a
// workgroup, which read the same keys out of the L2.  Such calls wait for
// latency, and its workgroups start and join sooner than sz_attn_tiles'.  Over
// 374 shapes within these limits (1 to 16 sequences, 60 to 3,000 keys, 20 to 800
// rows, every type) it took 0.79 of the time.  8 heads of 128, one sequence, 13
// tokens of four heads each in BF16: over 300 keys 10.8 us (11.8), 1,000 12.9
// (13.2), 1,900 13.2 (15.4); FP8 over 300 10.5 (12.4).  Far beyond the limits the
// products win (16 sequences of up to 500, 104 rows, BF16: 25.2 us for 19.2; 9 of
// 25 tokens over up to 22,943, three heads, 198 for 57).  They are on the low side,
// as they were set when one workgroup joined all chunks of a block: now 13 tokens
// over 3,000 keys, E4M3, would take 14.0 us in blocks (17.8), 26 of four sequences
// of up to 500, BF16, 10.0 (16.4).
constexpr uint64_t kBlocksKeys = 2048;
constexpr uint64_t kBlocksBytes = 1 << 17;       // workgroups times 128-key steps times bytes of a row
inline uint64_t row_blocks(const PagedBatch &b, uint32_t group)             // one also for no rows at all
{
    return std::max<uint64_t>(1, ((uint64_t)b.max_new * group + kRowsMax - 1) / kRowsMax);
}
inline bool rows_in_blocks(const sz_cache *c, const PagedBatch &b, uint32_t group)
{
    const uint64_t steps = std::max<uint64_t>(1, ((uint64_t)b.max_kv + 127) / 128), row = c->head_dim * (c->dtype == SZ_BF16 ? 2 : 1);
    return b.max_new <= kRowsTokens && b.max_kv <= kBlocksKeys &&
           (uint64_t)b.seqs * c->kv_heads * row_blocks(b, group) * steps <= kBlocksBytes / row;
}

// How trees' workgroups, `each` of a sequence, follow the sequences' lengths, as
// far as one wave can sort them and more than one comes to a CU (0: not): the long
// ones first, and if no more than two come to a CU, the shortest beside the longest.
// 64 trees of 8 tokens over up to 4,000 keys, 8 KV heads, E5M2 58 us (74), 128 of up
// to 8,000 223 (278), of up to 1,000 47 (50), 24 of up to 8,000 with 16 heads 97
// (130); 30 tokens in BF16, 128 of up to 8,000 445 (509); equal lengths the same.
inline uint32_t fold_of(const PagedBatch &b, uint64_t each, uint64_t cus)
{
    const uint64_t all = each * b.seqs;
    if (b.seqs < 2 || b.seqs > kOrdered || all <= cus) return 0;
    return all <= 2 * cus ? (uint32_t)std::max<uint64_t>(1, cus / each) : b.seqs;
}

inline AttnPlan attn_plan(const sz_cache *c, const PagedBatch &b, uint32_t group, uint32_t window, bool tree)
{
    AttnPlan p{};
    // chunks start at a multiple of kKeyAlign: up to kKeyAlign - 1 keys more than the visible ones
    uint64_t span = b.max_kv;
    if (window) span = std::min<uint64_t>(span, (uint64_t)window + b.max_new + kKeyAlign - 1);
    p.rows_limit = (uint64_t)b.max_new * group <= kRowsMax || !row_pairs(c->dtype, c->head_dim) ? kRowsMax : 2 * kRowsMax;
    p.tiles = (uint64_t)b.max_new * group > p.rows_limit;
    if (p.tiles) p.rows_limit = kRowsMax;
    // Sequences of few rows beside others: none if there is one sequence (its
    // rows all go the same way) or every sequence has max_new tokens.
    p.rows = !p.tiles || (b.seqs > 1 && group <= kRowsMax && b.tokens != (uint64_t)b.seqs * b.max_new);
    if (!p.rows) p.rows_limit = 0;
    p.row_blocks = 1;
    p.row_pairs = p.rows_limit > kRowsMax;
    if (tree && rows_in_blocks(c, b, group)) {
        p.rows = true;
        p.tiles = p.row_pairs = false;
        p.rows_limit = b.max_new * group;
        p.row_blocks = (uint32_t)row_blocks(b, group);
    }
    p.tile_waves = tree ? 4 : tile_waves(c->dtype, b, c->kv_heads, group);
    p.slots = (uint32_t)std::min<uint64_t>((uint64_t)b.tokens * group / (32 * p.tile_waves) + b.seqs, 0x7FFFFFFFu);
    const uint64_t each = ((uint64_t)b.max_new * group + 32 * p.tile_waves - 1) / (32 * p.tile_waves);
    if (tree && each * b.seqs <= p.slots) p.tiles_each = (uint32_t)each;
    p.grid_slots = p.tiles_each ? p.tiles_each * b.seqs : p.slots;
    p.rows_splits = p.tile_splits = 1;
    p.rows_chunk = p.tile_chunk = kMinChunk;
    const uint64_t groups = (uint64_t)b.seqs * c->kv_heads * p.row_blocks;
    const uint64_t values = (uint64_t)b.tokens * group * c->kv_heads * c->head_dim;
    if (p.rows) split_keys(span, tree ? kTreeFill / groups : rows_wanted(span, groups), p.rows_chunk, p.rows_splits);
    if (p.tiles) {
        // Trees count the workgroups that there are, not the slots that other
        // lengths could need: 16 of up to 8,192, 61 tokens of 32 heads, E4M3 134 us
        // (173), 30 tokens in BF16 87 (105); 16 of up to 1,500, 30 tokens, BF16 33
        // (30).  With a window a tile of rows sees less than its sequence's tokens
        // together: no chunks where that would not be split (488 new tokens
        // with a window of 14: one KV head of eight 15 us in chunks, 11
        // without; behind 3,000, four heads of four, 17 and 11).
        const uint64_t tiles = (uint64_t)p.grid_slots * c->kv_heads, tokens = 32 * p.tile_waves / group + 2;
        const uint64_t seen = window ? std::min(span, window + tokens + kTileKeys) : span;
        const bool split = tiles_wanted(seen, tiles, p.tile_waves, values) > 1;
        split_keys(span, split ? tiles_wanted(span, tiles, p.tile_waves, values) : 1, p.tile_chunk, p.tile_splits);
    }
    if (p.tiles_each && p.tile_splits == 1) p.fold = fold_of(b, (uint64_t)p.tiles_each * c->kv_heads, 256 * 4 / p.tile_waves);
    if (tree && p.rows && p.rows_splits == 1) p.rows_fold = fold_of(b, (uint64_t)c->kv_heads * p.row_blocks, 256);
    p.fused = p.rows_splits > 1 && p.rows_splits <= kFusedSplits && p.tile_splits == 1 &&
              groups * p.rows_splits <= kFusedGroups;
    const uint64_t rows = p.row_blocks > 1 ? kRowsMax : std::min<uint64_t>((uint64_t)b.max_new * group, p.rows_limit);
    if (tree && p.rows_splits * rows * c->head_dim > kTreeJoin) p.fused = false;
    return p;
}

// Workspace: kArrivals counters, then the partials of the chunks.
inline uint64_t attn_ws_bytes(uint64_t splits, uint64_t rows, uint32_t head_dim)
{
    return 4 * kArrivals + (splits == 1 ? 0 : up256(splits * rows * head_dim * 4) + up256(splits * rows * 8));
}

// sz_attn_join's tokens per sequence (0: all tokens of the batch), groups of
// lanes to a row (four chunks each, as far as a workgroup goes) and workgroups.
struct JoinPlan {
    uint32_t per_seq, parts;
    uint64_t groups;
};
inline JoinPlan join_plan(const PagedBatch &b, const AttnPlan &p, uint32_t group, uint32_t q_heads, uint32_t head_dim)
{
    JoinPlan j{};
    const uint32_t rows_splits = p.fused ? 1 : p.rows_splits, splits = std::max(rows_splits, p.tile_splits);
    if (splits == 1) return j;
    const uint32_t most = kAttnThreads / (head_dim / 4);
    j.per_seq = p.tile_splits > 1 ? 0 : std::min(b.max_new, p.rows_limit / group);
    for (j.parts = 1; j.parts < most && 4 * j.parts < splits;) j.parts *= 2;
    const uint32_t rows = most / j.parts;
    j.groups = (j.per_seq ? (uint64_t)b.seqs * j.per_seq : (uint64_t)b.tokens) * ((q_heads + rows - 1) / rows);
    return j;
}

// Whether the launches stay within a launch's threads.
inline bool launchable(const PagedCache &c, const PagedBatch &b, const AttnPlan &p, const JoinPlan &j)
{
    return (!p.rows || (uint64_t)c.heads * b.seqs * p.rows_splits * p.row_blocks * kAttnThreads <= kMaxThreads) &&
           (!p.tiles || (uint64_t)c.heads * p.grid_slots * p.tile_splits * 64 * p.tile_waves <= kMaxThreads) &&
           j.groups * kAttnThreads <= kMaxThreads;
}

template <int DT, int D, typename Args>
int launch_attention(const Args &a, const AttnPlan &p, const JoinPlan &j, hipStream_t s)
{
    if (p.rows) {
        const uint64_t groups = (uint64_t)a.c.heads * a.b.seqs * p.rows_splits * p.row_blocks;
        LaunchScope scope("sz_attn_rows", s);
        const auto launch = [&](const auto &args) {
            using A = std::decay_t<decltype(args)>;
            if (!p.row_pairs)
                hipLaunchKernelGGL((sz_attn_rows<DT, D, 1, A>), dim3((uint32_t)groups), dim3(kAttnThreads), 0, s, args);
            else if constexpr (row_pairs(DT, D))
                hipLaunchKernelGGL((sz_attn_rows<DT, D, 2, A>), dim3((uint32_t)groups), dim3(kAttnThreads), 0, s, args);
        };
        if constexpr (Args::kTree) {
            if (p.rows_fold)
                launch(OrderedArgs{a});
            else
                launch(a);
        } else {
            launch(a);
        }
    }
    if (p.tiles) {
        const uint64_t groups = (uint64_t)a.c.heads * p.grid_slots * p.tile_splits;
        LaunchScope scope("sz_attn_tiles", s);
        if (p.tile_waves == 4)
            hipLaunchKernelGGL((sz_attn_tiles<DT, D, 4, Args>), dim3((uint32_t)groups), dim3(256), 0, s, a, p.grid_slots);
        else if constexpr (DT != SZ_BF16 && !Args::kTree)
            hipLaunchKernelGGL((sz_attn_tiles<DT, D, 8, Args>), dim3((uint32_t)groups), dim3(512), 0, s, a, p.grid_slots);
    }
    if (j.groups) {
        LaunchScope scope("sz_attn_join", s);
        hipLaunchKernelGGL((sz_attn_join<D, Args>), dim3((uint32_t)j.groups), dim3(kAttnThreads), 0, s, a, j.per_seq,
                           j.parts);
    }
    return hipGetLastError() == hipSuccess ? SZ_OK : SZ_E_HIP;
}

// Both calls; `a` has the trees' own fields.
template <typename Args>
int attend(Args a, const sz_cache *cache, const sz_batch *batch, const void *d_q, uint32_t q_heads,
                  uint64_t q_token_stride, uint64_t q_head_stride, float scale, uint32_t window, void *d_out, float *d_lse,
                  void *d_ws, uint64_t ws_bytes, int32_t *d_status, void *stream)
{
    int rc = check_paged(cache, batch, d_status, a.c, a.b);
    if (rc != SZ_OK) return rc;
    if (q_heads == 0 || q_heads > kMaxQueryHeads || q_heads % a.c.heads) return SZ_E_ARG;
    a.c2 = scale * 1.44269504088896340736f;
    if (!(scale > 0.f) || !std::isfinite(a.c2) || window > 0x7FFFFFFFu) return SZ_E_ARG;
    if ((rc = check_rows(d_q, q_token_stride, q_head_stride, a.b.tokens, q_heads)) != SZ_OK) return rc;
    if (!aligned16(d_out) || !aligned16(d_ws) || (reinterpret_cast<uintptr_t>(d_lse) & 3u)) return SZ_E_ALIGN;
    if (a.b.tokens == 0 || a.b.seqs == 0) return SZ_OK;
    a.group = q_heads / a.c.heads;
    a.window = window_keys(window);
    const AttnPlan p = attn_plan(cache, a.b, a.group, (uint32_t)a.window, Args::kTree);
    const JoinPlan j = join_plan(a.b, p, a.group, q_heads, cache->head_dim);
    if (!launchable(a.c, a.b, p, j)) return SZ_E_ARG;
    const uint32_t splits = std::max(p.rows_splits, p.tile_splits);
    const uint64_t rows = (uint64_t)a.b.tokens * q_heads;
    if (!d_ws) return SZ_E_ARG;
    if (ws_bytes < attn_ws_bytes(splits, rows, cache->head_dim)) return SZ_E_WORKSPACE;
    if (!d_out) return SZ_E_ARG;
    a.q = static_cast<const uint16_t *>(d_q);
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.out = static_cast<uint16_t *>(d_out);
    a.lse = d_lse;
    a.arrived = p.fused ? static_cast<uint32_t *>(d_ws) : nullptr;
    a.part = static_cast<float *>(d_ws) + kArrivals;
    a.part_ml = reinterpret_cast<float2 *>(reinterpret_cast<uint8_t *>(a.part) +
                                           up256(splits * rows * cache->head_dim * 4));
    a.scale = scale;
    a.q_heads = q_heads;
    a.rows_limit = p.rows_limit;
    a.rows_chunk = p.rows_chunk;
    a.rows_splits = p.rows_splits;
    a.tile_chunk = p.tile_chunk;
    a.tile_splits = p.tile_splits;
    if constexpr (Args::kTree) {
        a.tiles_each = p.tiles_each;
        a.fold = p.fold;
        a.row_blocks = p.row_blocks;
        a.rows_fold = p.rows_fold;
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool wide = cache->head_dim == 128;
    switch (cache->dtype) {
    case SZ_BF16: return wide ? launch_attention<SZ_BF16, 128>(a, p, j, s) : launch_attention<SZ_BF16, 64>(a, p, j, s);
    case SZ_FP8_E5M2:
        return wide ? launch_attention<SZ_FP8_E5M2, 128>(a, p, j, s) : launch_attention<SZ_FP8_E5M2, 64>(a, p, j, s);
    default: return wide ? launch_attention<SZ_FP8_E4M3, 128>(a, p, j, s) : launch_attention<SZ_FP8_E4M3, 64>(a, p, j, s);
    }
}

}  // namespace
}  // namespace sz
