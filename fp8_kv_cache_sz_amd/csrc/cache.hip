// Paged KV cache: new tokens' rows into pages, quantised to FP8 on the way,
// and tokens' rows back out of pages as BF16.
//
// A row is one token's one head, K or V: D values x.  FP8 caches keep
//   a = max |x_d| over the finite x_d
//   k = max(-126, the smallest integer with a <= MAX 2^k)
//       MAX = 1.75 2^8 (E4M3) or 1.75 2^15 (E5M2), the largest finite value
//   q_d = x_d 2^-k rounded to FP8, nearest even;  scale byte = k + 127
// and read back q_d 2^k.  The scale is a power of two because then x_d 2^-k
// is exact and each value is rounded once, to FP8, and because q_d 2^k is
// exact in BF16, so that what attention reads is what sz_cache_read returns.
// NaN stays NaN; infinities stay infinite in E5M2 and become NaN in E4M3,
// which has none.
//
// Both directions stream: 2 bytes per value on the BF16 side, 1 (or 2) plus
// 1 byte per row on the cache's.  They are bound by HBM, small calls by the
// latency of three dependent loads (starts -> length -> page).
#include "paged.hpp"

namespace sz {
namespace {

constexpr uint32_t kMoveThreads = 256;
constexpr uint32_t kMoveTokens = 16;     // of a wave: their places are found once

// Lanes per row: each moves 8 values (16 bytes of BF16).
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

struct Rows {
    uint16_t *p[2];           // K and V: [tokens][heads][D]
    uint64_t token[2], head[2];
};

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

// A wave moves 16 tokens' rows of one (K or V, head) pair, WRITE: tensors ->
// pages, else pages -> tensors.  Its lanes 0..15 find a token's place each; a
// pass then takes 4 (D = 64: 8) tokens, which lie next to each other in a
// page, and the passes have their loads in flight together.  Waves that run
// together take neighbouring heads of the same tokens, whose rows are
// neighbours in the tensors.
// The BF16 side streams past the caches (non-temporal); the cache's side does
// not, since attention reads it next.  Measured (MI355X): 65,536 tokens of 4
// heads of 128, E5M2 -> BF16, 31 us, 6.5 TB/s (42 us with plain stores);
// 74,251 tokens of 8 heads, E4M3 -> BF16, 85 us, 5.4 TB/s; 32,254 tokens of 8
// heads, BF16 -> E4M3, 40 us, 5.0 TB/s (44 us with plain loads).  Of the last
// two 7 and 2 us are the lookups.  8 tokens to a wave take 104 and 45 us, 32
// 90 and 45, four pairs to a wave 99 (too few waves to even out).
template <int DT, int D, bool WRITE>
__global__ __launch_bounds__(kMoveThreads) void sz_cache_move(PagedCache c, PagedBatch b, Rows x)
{
    constexpr uint32_t LPR = kRowLanes<D>, RPP = 64 / LPR;
    constexpr int PASSES = kMoveTokens / RPP;
    const uint32_t unit = uniform(blockIdx.x * (kMoveThreads / 64) + threadIdx.x / 64);
    const uint32_t t0 = unit / (2 * c.heads) * kMoveTokens, pair = unit % (2 * c.heads);
    if (t0 >= b.tokens) return;
    const uint32_t lane = lane_id();

    // The place of token t0 + lane as a row of pair 0, or none.  Loads that
    // wait for one another are most of a wave's time, so the starts and
    // lengths of the 64 sequences from t0's on come in one (up to 63
    // sequences: the first), and each token counts its own from there.
    constexpr uint64_t NONE = ~0ull;
    uint64_t mine = NONE;
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
    // What no token's own sequence shows: starts that descend, and (the first
    // wave's) an axis that begins or ends outside [0, tokens].
    const int32_t after = __shfl_down(start, 1, 64);
    bool wrong = lane < 63 && there && after < start;
    if (unit == 0 && lane < 2) {
        const int32_t edge = b.starts[lane * b.seqs];
        wrong |= edge < 0 || edge > (int32_t)b.tokens;
    }
    if (wrong) flag_batch(b);
    uint32_t count = 0;                              // of the starts up to this lane's token
#pragma unroll
    for (uint32_t j = 0; j < kMoveTokens; ++j) {
        const uint64_t passed = __ballot(start <= (int32_t)(t0 + j));
        if (lane == j) count = (uint32_t)__popcll(passed);
    }
    const int32_t my_start = __shfl(start, (int)max(count, 1u) - 1, 64), my_next = __shfl(start, (int)min(count, 63u), 64);
    const int32_t my_len = __shfl(len, (int)max(count, 1u) - 1, 64);
    if (lane < kMoveTokens && t0 + lane < b.tokens && count > 0) {
        const uint32_t t = t0 + lane;
        uint32_t i = base + count - 1;
        Sequence s{0, 0, 0};
        if (count < 64) {
            if (i < b.seqs) s = checked(b, my_start, my_next, my_len);
        } else {                                     // 64 sequences on, or more
            for (uint32_t past = b.seqs; past - i > 1;) {
                const uint32_t mid = i + (past - i) / 2;
                (b.starts[mid] <= (int32_t)t ? i : past) = mid;
            }
            if (i < b.seqs) s = sequence(b, i);
        }
        const int32_t pos = s.len - s.n + ((int32_t)t - s.start);
        if ((int32_t)t >= s.start && (int32_t)t < s.start + s.n && pos >= 0) {
            const uint32_t page = (uint32_t)b.table[(uint64_t)i * b.width + ((uint32_t)pos >> c.lg_page)];
            if (page < c.pages)
                mine = row_index(c, page, 0, 0, (uint32_t)pos & ((1u << c.lg_page) - 1));
            else
                flag_batch(b);
        }
    }
    const uint32_t sub = lane / LPR, off = (lane % LPR) * 8;
    uint64_t place[PASSES];
#pragma unroll
    for (int j = 0; j < PASSES; ++j) {
        const int from = (int)(j * RPP + sub);
        place[j] = (uint64_t)(uint32_t)__shfl((int)(uint32_t)mine, from, 64) |
                   (uint64_t)(uint32_t)__shfl((int)(uint32_t)(mine >> 32), from, 64) << 32;
    }

    const uint32_t kv = pair >= c.heads ? 1u : 0u;
    uint16_t *rows = x.p[kv] + (uint64_t)(pair - kv * c.heads) * x.head[kv] + off;
    uint4 v[PASSES];
    uint32_t sc[PASSES];
#pragma unroll
    for (int j = 0; j < PASSES; ++j) {
        if (place[j] == NONE) continue;
        place[j] += (uint64_t)pair << c.lg_page;
        if constexpr (WRITE) {
            v[j] = load_nt(reinterpret_cast<const uint4 *>(rows + (uint64_t)(t0 + j * RPP + sub) * x.token[kv]));
        } else if constexpr (DT == SZ_BF16) {
            v[j] = *reinterpret_cast<const uint4 *>(c.data + (place[j] * D + off) * 2);
        } else {
            const uint2 q = *reinterpret_cast<const uint2 *>(c.data + place[j] * D + off);
            v[j].x = q.x;
            v[j].y = q.y;
            sc[j] = c.scales[place[j]];
        }
    }
#pragma unroll
    for (int j = 0; j < PASSES; ++j) {
        if (place[j] == NONE) continue;                              // whole rows: a row's lanes agree
        if constexpr (WRITE) {
            put_chunk<DT, D>(c, place[j], off, v[j]);
        } else {
            uint4 w = v[j];
            if constexpr (DT != SZ_BF16) {
                const uint32_t s = sc[j] << 23;
                w = make_uint4(fp8_pair_to_bf16<DT, false>(v[j].x, s), fp8_pair_to_bf16<DT, true>(v[j].x, s),
                               fp8_pair_to_bf16<DT, false>(v[j].y, s), fp8_pair_to_bf16<DT, true>(v[j].y, s));
            }
            store_nt(reinterpret_cast<uint4 *>(rows + (uint64_t)(t0 + j * RPP + sub) * x.token[kv]), w);
        }
    }
}

template <bool WRITE>
int move(const sz_cache *cache, const sz_batch *batch, void *d_k, uint64_t k_token, uint64_t k_head, void *d_v,
         uint64_t v_token, uint64_t v_head, int32_t *d_status, void *stream)
{
    PagedCache c;
    PagedBatch b;
    int rc = check_paged(cache, batch, d_status, c, b);
    if (rc != SZ_OK) return rc;
    if ((rc = check_rows(d_k, k_token, k_head, b.tokens, c.heads)) != SZ_OK) return rc;
    if ((rc = check_rows(d_v, v_token, v_head, b.tokens, c.heads)) != SZ_OK) return rc;
    if (b.tokens == 0 || b.seqs == 0) return SZ_OK;
    const Rows x{{static_cast<uint16_t *>(d_k), static_cast<uint16_t *>(d_v)}, {k_token, v_token}, {k_head, v_head}};
    hipStream_t s = static_cast<hipStream_t>(stream);
    const uint64_t tiles = ((uint64_t)b.tokens + kMoveTokens - 1) / kMoveTokens;
    const uint64_t groups = (tiles * 2 * c.heads + 3) / 4;
    if (groups * kMoveThreads > 0xFFFFFFFFull) return SZ_E_ARG;      // a launch's threads
    LaunchScope scope(WRITE ? "sz_cache_write" : "sz_cache_read", s);
    const dim3 grid((uint32_t)groups), block(kMoveThreads);
#define SZ_MOVE(DT)                                                                                         \
    do {                                                                                                    \
        if (cache->head_dim == 128)                                                                         \
            hipLaunchKernelGGL((sz_cache_move<DT, 128, WRITE>), grid, block, 0, s, c, b, x);         \
        else                                                                                                \
            hipLaunchKernelGGL((sz_cache_move<DT, 64, WRITE>), grid, block, 0, s, c, b, x);          \
    } while (0)
    if (cache->dtype == SZ_BF16)
        SZ_MOVE(SZ_BF16);
    else if (cache->dtype == SZ_FP8_E5M2)
        SZ_MOVE(SZ_FP8_E5M2);
    else
        SZ_MOVE(SZ_FP8_E4M3);
#undef SZ_MOVE
    return hipGetLastError() == hipSuccess ? SZ_OK : SZ_E_HIP;
}

// ---------------------------------------------------------------------------
// sz_cache_check: everything the other calls check as they go, and that no
// page is written from two places of the batch.  Clears the status word and
// the claims in one launch, then one wave per sequence walks its pages; a
// page that a new token falls into is claimed with an atomic exchange, and
// whoever finds it claimed has found a page that two places write.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void sz_cache_check_clear(uint32_t *claims, uint32_t pages, int32_t *status)
{
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    if (i < pages) claims[i] = 0;
    if (i == 0) *status = SZ_OK;
}

__global__ __launch_bounds__(256) void sz_cache_check_walk(PagedCache c, PagedBatch b, uint32_t *claims)
{
    const uint32_t i = uniform(blockIdx.x * 4 + threadIdx.x / 64);
    if (i >= b.seqs) return;
    if (i > 0 && b.starts[i] < b.starts[i - 1]) flag_batch(b);
    const Sequence s = sequence(b, i);
    const uint32_t used = ((uint32_t)s.len + (1u << c.lg_page) - 1) >> c.lg_page;
    const int32_t lo = max(0, s.len - s.n);
    for (uint32_t w = lane_id(); w < used; w += 64) {
        const uint32_t page = (uint32_t)b.table[(uint64_t)i * b.width + w];
        if (page >= c.pages)
            flag_batch(b);
        else if (s.n > 0 && w >= ((uint32_t)lo >> c.lg_page) && atomicExch(&claims[page], 1u) != 0u)
            flag_batch(b);
    }
}

}  // namespace
}  // namespace sz

using namespace sz;

extern "C" int sz_cache_write(const sz_cache *cache, const sz_batch *batch, const void *d_k, uint64_t k_token_stride,
                              uint64_t k_head_stride, const void *d_v, uint64_t v_token_stride,
                              uint64_t v_head_stride, int32_t *d_status, void *stream)
{
    return move<true>(cache, batch, const_cast<void *>(d_k), k_token_stride, k_head_stride, const_cast<void *>(d_v),
                      v_token_stride, v_head_stride, d_status, stream);
}

extern "C" int sz_cache_read(const sz_cache *cache, const sz_batch *batch, void *d_k, uint64_t k_token_stride,
                             uint64_t k_head_stride, void *d_v, uint64_t v_token_stride, uint64_t v_head_stride,
                             int32_t *d_status, void *stream)
{
    return move<false>(cache, batch, d_k, k_token_stride, k_head_stride, d_v, v_token_stride, v_head_stride, d_status,
                       stream);
}

extern "C" uint64_t sz_cache_check_workspace_size(const sz_cache *cache)
{
    return cache ? up256(4 * cache->pages) : 0;
}

extern "C" int sz_cache_check(const sz_cache *cache, const sz_batch *batch, void *d_ws, uint64_t ws_bytes,
                              int32_t *d_status, void *stream)
{
    PagedCache c;
    PagedBatch b;
    const int rc = check_paged(cache, batch, d_status, c, b);
    if (rc != SZ_OK) return rc;
    if (!d_ws) return SZ_E_ARG;
    if (!aligned16(d_ws)) return SZ_E_ALIGN;
    if (ws_bytes < sz_cache_check_workspace_size(cache)) return SZ_E_WORKSPACE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    uint32_t *claims = static_cast<uint32_t *>(d_ws);
    {
        LaunchScope scope("sz_cache_check_clear", s);
        hipLaunchKernelGGL(sz_cache_check_clear, dim3((c.pages + 255) / 256), dim3(256), 0, s, claims, c.pages,
                           d_status);
    }
    if (b.seqs) {
        LaunchScope scope("sz_cache_check_walk", s);
        hipLaunchKernelGGL(sz_cache_check_walk, dim3((b.seqs + 3) / 4), dim3(256), 0, s, c, b, claims);
    }
    return hipGetLastError() == hipSuccess ? SZ_OK : SZ_E_HIP;
}
