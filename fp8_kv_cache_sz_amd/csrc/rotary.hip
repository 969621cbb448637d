// Rotary positions on the way into the paged cache: new tokens' queries and
// keys are turned by their positions, keys and values written into pages.
//
// Frequency f_i turns the pair (x, y) of a row, d = (i, i + R/2) ("half") or
// (2i, 2i + 1) ("interleaved"), i < R/2, of a token at position p:
//   x' = x c - y s,  y' = y c + x s,  c = A cos(p f_i),  s = A sin(p f_i)
// and values from R on stay.
//
// The angle is taken modulo a turn before it is a floating number: the caller
// gives f_i / 2 pi as a 64-bit fraction F_i of a turn, and p F_i wraps around
// exactly as the angle does, off by at most p 2^-65 turns at any position
// (2^-34 at 2^31), where 32-bit p f_i has lost a turn's 2^-7 at 2^17.  What is
// left after the nearest quarter turn, at most pi/4, is rounded to its type as it
// is, not at a fixed place (cut at 2^-32 turns, the slowest pairs of base 10^7 were
// off by 1 % at the first positions where a value's partner is 0), and goes through
// the Taylor series of sine and cosine, to the last bits of its type.
//
// Queries, and keys of BF16 caches, are computed in 32 bits.  Keys of FP8
// caches in 64, rounded to 32: a row's scale depends on which side of a power
// of two (times 1.75) its largest value is, and so should not depend on the
// order of a kernel's roundings.
//
// A wave takes 4 (D = 64: 8) tokens and some heads of q, k or v: the sines are
// worked out once for the heads.  Its first rows are on their way before it
// looks up whose its tokens are.  Bound by HBM in the large, in the small by the
// latency of loads that wait for each other (starts and lengths, page or
// position, the store).  Measured (MI355X): 32,254 tokens of prompts, 32 + 8 heads
// of 128, E5M2 (727 MB) 111.5 us, 6.5 TB/s, what a large copy reaches; 64 trees of
// up to 24 tokens, 28 + 4 heads in BF16 (28 MB) 8.7 us; one token 6.6 us on the GPU.
#include "paged.hpp"

#include <cmath>
#include <type_traits>

namespace sz {
namespace {

constexpr uint32_t kRotaryThreads = 256;
// Heads of a wave.  64 trees of 24 tokens, 28 + 4 heads in BF16: 9.9 us (4: 10.5,
// 16: 11.4); 32,254 tokens of prompts, 32 + 8 heads, E5M2: 116 (125, 117).
constexpr uint32_t kHeads = 8;
constexpr int kAhead = 4;                // rows that a lane has in flight

struct RotaryArgs {
    PagedCache c;
    PagedBatch b;
    const uint64_t *turns;    // [R / 2]
    const int32_t *positions; // [tokens] or null: where the tokens stand
    const uint16_t *q, *k, *v;
    uint16_t *out;            // q's, turned
    uint64_t q_token, q_head, out_token, out_head, k_token, k_head, v_token, v_head;
    double amplitude;
    uint32_t dim, q_heads;    // R; heads of q
    uint32_t heads_each, q_units, kv_units;           // heads of a wave; waves of a token's heads
};

// x - x^3/3! + ..., 1 - x^2/2! + ... for |x| <= pi/4.  The first term left out
// is below 2^-28 (float) and 2^-56 (double).
template <typename T>
__device__ __forceinline__ void sin_cos_small(T x, T &s, T &c)
{
    constexpr int TERMS = std::is_same<T, float>::value ? 6 : 9;
    const T z = x * x;
    T a = 0, b = 0;
#pragma unroll
    for (int n = TERMS - 1; n >= 0; --n) {           // sum (-1)^n z^n / (2n+1)!, / (2n)!
        double up = 1;
        for (int i = 2; i <= 2 * n; ++i) up *= i;
        const T even = (T)((n % 2 ? -1.0 : 1.0) / up), odd = (T)((n % 2 ? -1.0 : 1.0) / (up * (2 * n + 1)));
        a = fma(a, z, odd);
        b = fma(b, z, even);
    }
    s = a * x;
    c = b;
}

// Sine and cosine of a 64-bit fraction of a turn.
template <typename T>
__device__ __forceinline__ void sin_cos(uint64_t turn, T &s, T &c)
{
    const uint64_t quarter = (turn + (1ull << 61)) >> 62;
    const int64_t rest = (int64_t)(turn - (quarter << 62));              // [-1/8, 1/8) of a turn
    T x;
    if constexpr (std::is_same<T, float>::value)         // both halves: a small angle keeps its 24 bits
        x = fmaf((float)(int32_t)(rest >> 32), (float)(6.283185307179586476925 / 4294967296.0),
                 (float)(uint32_t)rest * (float)(6.283185307179586476925 / 18446744073709551616.0));
    else
        x = (double)rest * (6.283185307179586476925 / 18446744073709551616.0);
    T a, b;
    sin_cos_small(x, a, b);
    const bool swap = quarter & 1;
    s = swap ? b : a;
    c = swap ? a : b;
    if (quarter & 2) s = -s;
    if ((quarter + 1) & 2) c = -c;
}

__device__ __forceinline__ float low_value(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float high_value(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

// How a lane's eight values of a row lie, and where their partners are.
//   kPairs   interleaved: d = 8 l.., four pairs
//   kHalves  half, R a multiple of 16: d = 8 l.., the partners in the lane R/16
//            away, which has the same sines
//   kRuns    half, other R: d = 4 l.. and R/2 + 4 l.., four pairs; lanes that do
//            not turn split what is behind R alike
// kRuns needs no other lane's values, but its 8-byte pieces are worth less where
// a run of them is short.  42,000 tokens of 36 heads and 4 of V, FP8, kHalves
// (kRuns): D = 64 71 us (91), D = 128 R = 64 127 (172), R = 128 127 (127).
enum Layout { kPairs, kHalves, kRuns };

template <int D, int L>
__device__ __forceinline__ void lane_runs(uint32_t l, uint32_t dim, bool turns, uint32_t &first, uint32_t &second)
{
    first = L != kRuns ? 8 * l : turns ? 4 * l : dim + 4 * (l - dim / 8);
    second = L != kRuns ? 8 * l + 4 : first + (turns ? dim : D - dim) / 2;
}
template <int L>
constexpr int kSines = L == kHalves ? 8 : 4;             // of a lane
// The first of the four frequencies whose sines a lane finds.  kHalves: the
// lanes of two partners find four each of their eight.
template <int L>
__device__ __forceinline__ uint32_t frequencies(uint32_t l, uint32_t dim)
{
    return L != kHalves ? 4 * l : l < dim / 16 ? 8 * l : 8 * (l - dim / 16) + 4;
}

// Eight values.  Lanes that do not turn keep them (0 times an infinity is a
// NaN).  kHalves: s has the sign that the partner's value takes.
template <int L, typename T>
__device__ __forceinline__ void turn(const uint4 &own, const uint4 &partner, bool turns, const T (&s)[kSines<L>],
                                     const T (&c)[kSines<L>], float (&x)[8])
{
    const uint32_t w[4] = {own.x, own.y, own.z, own.w}, p[4] = {partner.x, partner.y, partner.z, partner.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[2 * e] = low_value(w[e]);
        x[2 * e + 1] = high_value(w[e]);
    }
    float y[8];
    if constexpr (L == kHalves) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const T v = e % 2 ? high_value(p[e / 2]) : low_value(p[e / 2]);
            y[e] = (float)fma((T)x[e], c[e], v * s[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = L == kRuns ? e : 2 * e, j = L == kRuns ? e + 4 : 2 * e + 1;
            const T u = x[i], v = x[j];
            y[i] = (float)fma(u, c[e], -(v * s[e]));
            y[j] = (float)fma(v, c[e], u * s[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = turns ? y[e] : x[e];
}

// Eight values into a row of the cache, runs at `first` and `second`.  All of
// a row's lanes take part.
template <int DT, int D, int L>
__device__ __forceinline__ void put_values(const PagedCache &c, uint64_t at, uint32_t first, uint32_t second, bool scale,
                                           const float (&x)[8])
{
    if constexpr (DT == SZ_BF16) {
        uint16_t *p = reinterpret_cast<uint16_t *>(c.data) + at * D;
        const uint4 t = make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
        if constexpr (L == kRuns) {
            *reinterpret_cast<uint2 *>(p + first) = make_uint2(t.x, t.y);
            *reinterpret_cast<uint2 *>(p + second) = make_uint2(t.z, t.w);
        } else {
            *reinterpret_cast<uint4 *>(p + first) = t;
        }
    } else {
        uint32_t a = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t m = __builtin_bit_cast(uint32_t, x[e]) & 0x7FFFFFFFu;
            a = max(a, m < 0x7F800000u ? m : 0u);
        }
        a = row_max<kRowLanes<D>>(a);
        // as for BF16 rows: a <= 1.75 2^(EMAX+k)
        constexpr int32_t EMAX = DT == SZ_FP8_E4M3 ? 8 : 15;
        const int32_t byte = max(1, (int32_t)(a >> 23) - EMAX + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0));
        const float inv = __builtin_bit_cast(float, (uint32_t)(254 - byte) << 23);
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e / 2] = fp8_pair<DT>(x[2 * e] * inv, x[2 * e + 1] * inv, w[e / 2], e % 2 == 1);
        if constexpr (L == kRuns) {
            *reinterpret_cast<uint32_t *>(c.data + at * D + first) = w[0];
            *reinterpret_cast<uint32_t *>(c.data + at * D + second) = w[1];
        } else {
            *reinterpret_cast<uint2 *>(c.data + at * D + first) = make_uint2(w[0], w[1]);
        }
        if (scale) c.scales[at] = (uint8_t)byte;
    }
}

// A wave's tokens: t0 on, a row of lanes each.
struct Token {
    uint32_t t;               // the lane's row's
    bool there;               // it has a place
    uint64_t place;           // of its key in head 0, as a row of the cache
    uint64_t turn;            // its position, as a factor of turns
};
template <int D, bool PLACES>
__device__ __forceinline__ Token find_token(const RotaryArgs &a, uint32_t t0, bool edges)
{
    constexpr uint32_t TOKENS = 64 / kRowLanes<D>;
    constexpr uint64_t NONE = ~0ull;
    const uint32_t lane = lane_id();
    int32_t at = a.positions && lane < TOKENS ? a.positions[min(t0 + lane, a.b.tokens - 1)] : 0, pos = 0;
    uint32_t i;
    uint64_t mine = NONE;
    if (token_position<TOKENS>(a.b, t0, edges, i, pos)) {
        if (!a.positions) at = pos;
        mine = 0;
        if constexpr (PLACES) {
            const uint32_t page = (uint32_t)a.b.table[(uint64_t)i * a.b.width + ((uint32_t)pos >> a.c.lg_page)];
            mine = NONE;
            if (page < a.c.pages)
                mine = row_index(a.c, page, 0, 0, (uint32_t)pos & ((1u << a.c.lg_page) - 1));
            else
                flag_batch(a.b);
        }
    }
    const int sub = (int)(lane / kRowLanes<D>);
    Token x;
    x.t = t0 + (uint32_t)sub;
    x.place = __shfl(mine, sub, 64);
    x.there = x.place != NONE;
    x.turn = (uint64_t)(int64_t)__shfl(at, sub, 64);
    return x;
}

// Heads [head0, head0 + heads) of a wave's tokens, queries or keys.
template <int DT, int D, int L, bool QUERIES>
__device__ __forceinline__ void turn_heads(const RotaryArgs &a, uint32_t t0, bool edges, uint32_t head0, uint32_t heads)
{
    using T = typename std::conditional<!QUERIES && DT != SZ_BF16, double, float>::type;
    const uint32_t l = lane_id() % kRowLanes<D>, last = a.b.tokens - 1;
    const bool turns = 8 * l < a.dim;
    uint32_t first, second;
    lane_runs<D, L>(l, a.dim, turns, first, second);
    const uint32_t token = min(t0 + lane_id() / kRowLanes<D>, last);
    const uint16_t *from = QUERIES ? a.q + (uint64_t)token * a.q_token + (uint64_t)head0 * a.q_head
                                   : a.k + (uint64_t)token * a.k_token + (uint64_t)head0 * a.k_head;
    const uint64_t step = QUERIES ? a.q_head : a.k_head;
    uint4 x[kAhead];
    const auto load = [&](uint32_t h0) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const uint16_t *p = from + (uint64_t)min(h0 + j, heads - 1) * step;
            if constexpr (L == kRuns) {
                const uint2 u = load_nt(reinterpret_cast<const uint2 *>(p + first)), v = load_nt(reinterpret_cast<const uint2 *>(p + second));
                x[j] = make_uint4(u.x, u.y, v.x, v.y);
            } else {
                x[j] = load_nt(reinterpret_cast<const uint4 *>(p + first));
            }
        }
    };
    constexpr int SINES = kSines<L>;
    uint64_t f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = a.turns[turns ? frequencies<L>(l, a.dim) + e : 0];
    const bool low = l < a.dim / 16;                                     // kHalves: the pairs' first values
    const int partner = (int)(lane_id() + (!turns ? 0 : low ? a.dim / 16 : 0u - a.dim / 16));
    load(0);
    const Token w = find_token<D, !QUERIES>(a, t0, edges);
    T s[SINES], c[SINES];
    const T amplitude = (T)a.amplitude;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        sin_cos<T>(w.turn * f[e], s[e], c[e]);
        s[e] *= amplitude;
        c[e] *= amplitude;
    }
    if constexpr (L == kHalves) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const T u = __shfl(s[e], partner, 64), v = __shfl(c[e], partner, 64);
            s[e + 4] = low ? -u : s[e];
            c[e + 4] = low ? v : c[e];
            s[e] = low ? -s[e] : u;
            c[e] = low ? c[e] : v;
        }
    }
    if (!w.there) return;                                                // whole rows: a row's lanes agree
    for (uint32_t h0 = 0;;) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (h0 + j >= heads) break;
            float v[8];
            uint4 other = x[j];
            if constexpr (L == kHalves)
                other = make_uint4((uint32_t)__shfl((int)x[j].x, partner, 64), (uint32_t)__shfl((int)x[j].y, partner, 64),
                                   (uint32_t)__shfl((int)x[j].z, partner, 64), (uint32_t)__shfl((int)x[j].w, partner, 64));
            turn<L, T>(x[j], other, turns, s, c, v);
            const uint32_t head = head0 + h0 + j;
            if constexpr (QUERIES) {
                uint16_t *p = a.out + (uint64_t)w.t * a.out_token + (uint64_t)head * a.out_head;
                const uint4 t = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
                if constexpr (L == kRuns) {
                    store_nt(reinterpret_cast<uint2 *>(p + first), make_uint2(t.x, t.y));
                    store_nt(reinterpret_cast<uint2 *>(p + second), make_uint2(t.z, t.w));
                } else {
                    store_nt(reinterpret_cast<uint4 *>(p + first), t);
                }
            } else {
                put_values<DT, D, L>(a.c, w.place + ((uint64_t)head << a.c.lg_page), first, second, l == 0, v);
            }
        }
        h0 += kAhead;
        if (h0 >= heads) break;
        load(h0);
    }
}

// The same heads' values, as sz_cache_write writes them.
template <int DT, int D>
__device__ __forceinline__ void write_heads(const RotaryArgs &a, uint32_t t0, bool edges, uint32_t head0, uint32_t heads)
{
    const uint32_t off = lane_id() % kRowLanes<D> * 8;
    const uint32_t token = min(t0 + lane_id() / kRowLanes<D>, a.b.tokens - 1);
    const uint16_t *from = a.v + (uint64_t)token * a.v_token + (uint64_t)head0 * a.v_head + off;
    uint4 x[kAhead];
    const auto load = [&](uint32_t h0) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            x[j] = load_nt(reinterpret_cast<const uint4 *>(from + (uint64_t)min(h0 + j, heads - 1) * a.v_head));
    };
    load(0);
    const Token w = find_token<D, true>(a, t0, edges);
    if (!w.there) return;
    for (uint32_t h0 = 0;;) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (h0 + j < heads)
                put_chunk<DT, D>(a.c, w.place + ((uint64_t)(a.c.heads + head0 + h0 + j) << a.c.lg_page), off, x[j]);
        h0 += kAhead;
        if (h0 >= heads) break;
        load(h0);
    }
}

template <int DT, int D, int L>
__global__ __launch_bounds__(kRotaryThreads) void sz_rotary_move(RotaryArgs a)
{
    constexpr uint32_t TOKENS = 64 / kRowLanes<D>;
    const uint32_t units = a.q_units + 2 * a.kv_units;
    const uint32_t unit = uniform(blockIdx.x * (kRotaryThreads / 64) + threadIdx.x / 64);
    const uint64_t t64 = (uint64_t)(unit / units) * TOKENS;
    if (t64 >= a.b.tokens) return;
    const uint32_t t0 = (uint32_t)t64;
    uint32_t part = unit % units;
    if (part < a.q_units) {
        const uint32_t head0 = part * a.heads_each;
        turn_heads<DT, D, L, true>(a, t0, unit == 0, head0, min(a.heads_each, a.q_heads - head0));
        return;
    }
    part -= a.q_units;
    const uint32_t head0 = part % a.kv_units * a.heads_each, heads = min(a.heads_each, a.c.heads - head0);
    if (part < a.kv_units)
        turn_heads<DT, D, L, false>(a, t0, unit == 0, head0, heads);
    else                                                                 // V lies behind K: heads [H, 2 H) of the page
        write_heads<DT, D>(a, t0, false, head0, heads);
}

template <int DT, int D>
void launch_layout(const RotaryArgs &a, bool interleaved, uint32_t groups, hipStream_t s)
{
    const dim3 grid(groups), block(kRotaryThreads);
    if (interleaved)
        hipLaunchKernelGGL((sz_rotary_move<DT, D, kPairs>), grid, block, 0, s, a);
    else if (a.dim % 16 == 0)
        hipLaunchKernelGGL((sz_rotary_move<DT, D, kHalves>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((sz_rotary_move<DT, D, kRuns>), grid, block, 0, s, a);
}
template <int DT>
void launch_rotary(const RotaryArgs &a, uint32_t head_dim, bool interleaved, uint32_t groups, hipStream_t s)
{
    if (head_dim == 128)
        launch_layout<DT, 128>(a, interleaved, groups, s);
    else
        launch_layout<DT, 64>(a, interleaved, groups, s);
}

}  // namespace
}  // namespace sz

using namespace sz;

extern "C" int sz_rotary_write(const sz_cache *cache, const sz_batch *batch, const sz_rotary *rotary,
                               const int32_t *d_positions, const void *d_q, uint32_t q_heads, uint64_t q_token_stride,
                               uint64_t q_head_stride, void *d_out, uint64_t out_token_stride, uint64_t out_head_stride,
                               const void *d_k, uint64_t k_token_stride, uint64_t k_head_stride, const void *d_v,
                               uint64_t v_token_stride, uint64_t v_head_stride, int32_t *d_status, void *stream)
{
    RotaryArgs a{};
    int rc = check_paged(cache, batch, d_status, a.c, a.b);
    if (rc != SZ_OK) return rc;
    if (!rotary || rotary->dim < 8 || rotary->dim % 8 || rotary->dim > cache->head_dim || !rotary->d_turns) return SZ_E_ARG;
    if (rotary->interleaved > 1 || !std::isfinite((float)rotary->amplitude) || q_heads > kMaxQueryHeads) return SZ_E_ARG;
    if (reinterpret_cast<uintptr_t>(rotary->d_turns) & 7u || reinterpret_cast<uintptr_t>(d_positions) & 3u) return SZ_E_ALIGN;
    if (q_heads) {
        if ((rc = check_rows(d_q, q_token_stride, q_head_stride, a.b.tokens, q_heads)) != SZ_OK) return rc;
        if ((rc = check_rows(d_out, out_token_stride, out_head_stride, a.b.tokens, q_heads)) != SZ_OK) return rc;
    }
    if ((rc = check_rows(d_k, k_token_stride, k_head_stride, a.b.tokens, a.c.heads)) != SZ_OK) return rc;
    if ((rc = check_rows(d_v, v_token_stride, v_head_stride, a.b.tokens, a.c.heads)) != SZ_OK) return rc;
    if (a.b.tokens == 0 || a.b.seqs == 0) return SZ_OK;
    a.turns = rotary->d_turns;
    a.positions = d_positions;
    a.q = static_cast<const uint16_t *>(d_q);
    a.k = static_cast<const uint16_t *>(d_k);
    a.v = static_cast<const uint16_t *>(d_v);
    a.out = static_cast<uint16_t *>(d_out);
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.out_token = out_token_stride;
    a.out_head = out_head_stride;
    a.k_token = k_token_stride;
    a.k_head = k_head_stride;
    a.v_token = v_token_stride;
    a.v_head = v_head_stride;
    a.amplitude = rotary->amplitude;
    a.dim = rotary->dim;
    a.q_heads = q_heads;
    a.heads_each = kHeads;
    a.q_units = (q_heads + a.heads_each - 1) / a.heads_each;
    a.kv_units = (a.c.heads + a.heads_each - 1) / a.heads_each;
    const uint32_t tokens = 512 / cache->head_dim;                       // of a wave
    const uint64_t waves = (((uint64_t)a.b.tokens + tokens - 1) / tokens) * (a.q_units + 2 * a.kv_units);
    const uint64_t groups = (waves + 3) / 4;
    if (groups * kRotaryThreads > 0xFFFFFFFFull) return SZ_E_ARG;        // a launch's threads
    hipStream_t s = static_cast<hipStream_t>(stream);
    LaunchScope scope("sz_rotary_write", s);
    if (cache->dtype == SZ_BF16)
        launch_rotary<SZ_BF16>(a, cache->head_dim, rotary->interleaved != 0, (uint32_t)groups, s);
    else if (cache->dtype == SZ_FP8_E5M2)
        launch_rotary<SZ_FP8_E5M2>(a, cache->head_dim, rotary->interleaved != 0, (uint32_t)groups, s);
    else
        launch_rotary<SZ_FP8_E4M3>(a, cache->head_dim, rotary->interleaved != 0, (uint32_t)groups, s);
    return hipGetLastError() == hipSuccess ? SZ_OK : SZ_E_HIP;
}
