// Trees of drafted tokens: who is above whom, and the rows of those that were
// accepted.
#include "paged.hpp"

namespace sz {
namespace {

// ---------------------------------------------------------------------------
// sz_draft_tree: token i of a sequence has a parent p_i < i or none.
//   mask(i) = {i} + mask(p_i)        position(i) = len - n + |mask(i)| - 1
// A wave takes 64 tokens, a lane each.  Parents inside the 64 are followed by
// doubling: mask |= mask of the token pointed at, pointer = its pointer, six
// times at most.  What is left is one parent in an earlier 64, that of the
// token that the pointers end at; its row of earlier words is complete when
// that wave's is, so the waves of a sequence finish one after another, through
// LDS.  Bound by latency: a launch, the starts, the parents, the doubling.  16
// trees of 26 tokens take 2.4 us, 128 of up to 500 6 us (2.6 MB; MI355X).
// ---------------------------------------------------------------------------
struct TreeArgs {
    PagedBatch b;
    const int32_t *parents;
    uint64_t *masks;          // [tokens][words]
    int32_t *positions;       // [tokens]
    uint32_t words;
};

// The caller may have no status word here.
__device__ __forceinline__ void report(const PagedBatch &b)
{
    if (b.status) flag_batch(b);
}
__device__ __forceinline__ Sequence tree_sequence(const PagedBatch &b, uint32_t i)
{
    const int32_t start = b.starts[i], next = b.starts[i + 1], len = b.lens[i];
    if (!consistent(b, start, next, len)) {
        report(b);
        return Sequence{0, 0, 0};
    }
    return Sequence{start, next - start, len};
}

// Tokens above lane's own in its 64, itself included, and the parent before
// the 64 (or -1).
__device__ __forceinline__ uint64_t above(const TreeArgs &a, const Sequence &s, int32_t i0, int32_t &outer)
{
    const int32_t lane = (int32_t)lane_id(), i = i0 + lane;
    int32_t parent = -1;
    if (i < s.n) {
        parent = a.parents[s.start + i];
        if (parent < -1 || parent >= i) {
            report(a.b);
            parent = -1;
        }
    }
    outer = parent < i0 ? parent : -1;
    uint64_t mask = 1ull << lane;
    int to = parent >= i0 ? parent - i0 : lane;
#pragma unroll
    for (int k = 0; k < 6; ++k) {
        if (__all(to == lane)) break;                // nobody has a parent here
        mask |= __shfl(mask, to, 64);
        const int further = __shfl(to, to, 64);
        const bool done = __all(further == to);
        to = further;
        if (done) break;
    }
    outer = __shfl(outer, to, 64);
    return mask;
}

// Sequences of up to 64 tokens: a wave each.
__global__ __launch_bounds__(256) void sz_draft_tree_one(TreeArgs a)
{
    const uint32_t i = uniform(blockIdx.x * 4 + threadIdx.x / 64);
    if (i >= a.b.seqs) return;
    const Sequence s = tree_sequence(a.b, i);
    if (s.n == 0) return;
    int32_t outer;
    const uint64_t mask = above(a, s, 0, outer);
    const int32_t lane = (int32_t)lane_id();
    if (lane >= s.n) return;
    const uint64_t t = (uint64_t)(s.start + lane);
    a.masks[t * a.words] = mask;
    for (uint32_t w = 1; w < a.words; ++w) a.masks[t * a.words + w] = 0;
    a.positions[t] = s.len - s.n + (int32_t)__popcll(mask) - 1;
}

// Sequences of up to 64 W tokens: a workgroup of W waves each.
template <int W>
__global__ __launch_bounds__(64 * W) void sz_draft_tree_many(TreeArgs a)
{
    __shared__ uint64_t rows[64 * W][W + 1];         // an odd number of words: neighbours in other banks
    __shared__ int32_t depth[64 * W];
    const Sequence s = tree_sequence(a.b, blockIdx.x);
    const int32_t wave = (int32_t)uniform(threadIdx.x / 64), i = (int32_t)threadIdx.x;
    int32_t outer = -1;
    uint64_t mask = 0;
    if (64 * wave < s.n) mask = above(a, s, 64 * wave, outer);
    for (int32_t k = 0; k < W && 64 * k < s.n; ++k) {
        if (wave == k) {
            int32_t d = (int32_t)__popcll(mask);
            if (outer >= 0) d += depth[outer];
            for (int32_t w = 0; w < W; ++w) rows[i][w] = w == k ? mask : w < k && outer >= 0 ? rows[outer][w] : 0;
            depth[i] = d;
        }
        __syncthreads();
    }
    for (uint32_t x = threadIdx.x; x < (uint32_t)s.n * a.words; x += 64 * W) {
        const uint32_t w = x % a.words;              // the caller may have more words than the trees need
        a.masks[(uint64_t)s.start * a.words + x] = w < W ? rows[x / a.words][w] : 0;
    }
    if (i < s.n) a.positions[s.start + i] = s.len - s.n + depth[i] - 1;
}

// ---------------------------------------------------------------------------
// sz_cache_keep: row len - n + kept[k] goes to place len - n + k, for K and V,
// all heads and layers.  kept ascends, so kept[k] >= k: a row is read before
// any row that comes to its place is written if a head's rows are taken in
// the order of k, some of them read, then written, then the next.  A wave does
// that for `pairs_each` (K or V, head) pairs of one sequence and layer; its
// lanes look the places up once, 64 of them.  Bound by latency in the small (a
// launch, the lengths beside the kept tokens, their pages, the rows) and by
// HBM in the large.  32 layers of 8 heads, 5 of 26 tokens of 16 sequences, BF16
// (13 MB) take 6 us, 28 layers of 4 heads, 8 of 64 tokens of 64 sequences, E5M2
// (24 MB) 7 to 8 us (MI355X; a call each: 7.1 and 7.4).
// ---------------------------------------------------------------------------
constexpr uint32_t kLayers = 64;             // of a launch: their pointers are its arguments
constexpr int kKeepPasses = 8;               // reads in flight
// Rows of a wave, and waves that a call should have.  32 layers of 8 heads, 5 of
// 26 tokens of 16 sequences, BF16: 9.5 us with a pair (5 rows) to a wave, 8.9
// with two, 7.7 with four, 7.4 with eight; 28 layers of 4 heads, 8 of 64 tokens
// of 64 sequences, FP8: 12.8, 9.7, 7.9 and 8.0.
constexpr uint32_t kKeepRows = 40;
constexpr uint64_t kKeepWaves = 1024;

struct KeepArgs {
    PagedBatch b;
    const int32_t *kept;      // [seqs][width]
    const int32_t *counts;    // [seqs]
    uint32_t pages, heads, lg_page, width, layers, pairs_each, parts;        // parts: waves of a sequence's layer
    uint8_t *data[kLayers], *scales[kLayers];
};

template <int DT, int D>
__global__ __launch_bounds__(256) void sz_cache_keep_rows(KeepArgs a)
{
    constexpr uint32_t BYTES = D * (DT == SZ_BF16 ? 2 : 1), LPR = BYTES / 16, RPP = 64 / LPR;
    const uint32_t unit = uniform(blockIdx.x * 4 + threadIdx.x / 64);
    const uint32_t part = unit % (a.parts * a.layers), seq = unit / (a.parts * a.layers);
    if (seq >= a.b.seqs) return;
    const uint32_t layer = part / a.parts, pair0 = part % a.parts * a.pairs_each;
    const uint32_t pairs = min(a.pairs_each, 2 * a.heads - pair0);
    // what the wave needs to know, in loads that do not wait for each other
    const int32_t lane = (int32_t)lane_id(), *kept = a.kept + (uint64_t)seq * a.width;
    int32_t frm = kept[min(lane, (int32_t)a.width - 1)];
    const int32_t count = a.counts[seq];
    const Sequence s = sequence(a.b, seq);
    const int32_t past = s.len - s.n;
    bool good = count >= 0 && count <= (int32_t)a.width && count <= s.n;
    if (good) {
        const int32_t before = __shfl_up(frm, 1, 64);
        if (lane < count) good = frm < s.n && frm > (lane == 0 ? -1 : before);
        for (int32_t k = lane + 64; k < count; k += 64) good &= kept[k] < s.n && kept[k] > kept[k - 1];
    }
    if (!__all(good)) {
        flag_batch(a.b);
        return;
    }
    uint8_t *data = a.data[layer], *scales = a.scales[layer];
    const uint32_t page_mask = (1u << a.lg_page) - 1;
    for (int32_t k0 = 0; k0 < count; k0 += 64) {
        // lane: the rows of kept token k0 + lane, in pair 0
        constexpr uint64_t NONE = ~0ull;
        uint64_t from = NONE, to = NONE;
        const int32_t k = k0 + lane;
        if (k < count) {
            if (k0 > 0) frm = kept[k];
            const int32_t src = past + frm, dst = past + k;
            if (src != dst && dst >= 0) {
                const int32_t *row = a.b.table + (uint64_t)seq * a.b.width;
                const uint32_t x = (uint32_t)row[(uint32_t)src >> a.lg_page], y = (uint32_t)row[(uint32_t)dst >> a.lg_page];
                if (x < a.pages && y < a.pages) {
                    from = (((uint64_t)x * 2 * a.heads) << a.lg_page) + ((uint32_t)src & page_mask);
                    to = (((uint64_t)y * 2 * a.heads) << a.lg_page) + ((uint32_t)dst & page_mask);
                } else {
                    flag_batch(a.b);
                }
            }
        }
        // rows (pair, k) in order of k within a pair, the first ones that stay where they are left out
        const uint64_t moving = __ballot(from != NONE);
        if (moving == 0) continue;
        const uint32_t first = (uint32_t)__builtin_ctzll(moving), many = (uint32_t)min(count - k0, 64) - first;
        const uint32_t rows = pairs * many, piece = lane_id() % LPR;
        for (uint32_t r0 = 0; r0 < rows; r0 += kKeepPasses * RPP) {
            v4u v[kKeepPasses];
            uint8_t sc[kKeepPasses];
            uint64_t put[kKeepPasses];
#pragma unroll
            for (int p = 0; p < kKeepPasses; ++p) {
                const uint32_t r = r0 + p * RPP + lane_id() / LPR;
                const uint32_t at = r % many + first;
                uint64_t get = __shfl(from, (int)at, 64);
                put[p] = __shfl(to, (int)at, 64);
                if (r >= rows) put[p] = NONE;
                if (put[p] == NONE) continue;
                const uint64_t pair = (uint64_t)(pair0 + r / many) << a.lg_page;
                get += pair;
                put[p] += pair;
                v[p] = *reinterpret_cast<const v4u *>(data + get * BYTES + 16 * piece);
                if (DT != SZ_BF16 && piece == 0) sc[p] = scales[get];
            }
#pragma unroll
            for (int p = 0; p < kKeepPasses; ++p) {
                if (put[p] == NONE) continue;
                *reinterpret_cast<v4u *>(data + put[p] * BYTES + 16 * piece) = v[p];
                if (DT != SZ_BF16 && piece == 0) scales[put[p]] = sc[p];
            }
        }
    }
}

template <int DT>
void launch_keep(const KeepArgs &a, uint32_t head_dim, uint32_t groups, hipStream_t s)
{
    LaunchScope scope("sz_cache_keep", s);
    if (head_dim == 128)
        hipLaunchKernelGGL((sz_cache_keep_rows<DT, 128>), dim3(groups), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((sz_cache_keep_rows<DT, 64>), dim3(groups), dim3(256), 0, s, a);
}

}  // namespace
}  // namespace sz

using namespace sz;

extern "C" int sz_draft_tree(const sz_batch *batch, const int32_t *d_parents, uint64_t *d_masks, uint32_t words,
                             int32_t *d_positions, int32_t *d_status, void *stream)
{
    if (!batch) return SZ_E_ARG;
    TreeArgs a{};
    const int rc = check_batch(batch, d_status, a.b);
    if (rc != SZ_OK) return rc;
    if (words == 0 || words > SZ_TREE_WORDS || (uint64_t)a.b.max_new > 64ull * words) return SZ_E_ARG;
    if ((reinterpret_cast<uintptr_t>(d_parents) | reinterpret_cast<uintptr_t>(d_positions)) & 3u) return SZ_E_ALIGN;
    if (reinterpret_cast<uintptr_t>(d_masks) & 7u) return SZ_E_ALIGN;
    if (a.b.tokens == 0 || a.b.seqs == 0) return SZ_OK;
    if (!d_parents || !d_masks || !d_positions) return SZ_E_ARG;
    a.parents = d_parents;
    a.masks = d_masks;
    a.positions = d_positions;
    a.words = words;
    const uint32_t blocks = (a.b.max_new + 63) / 64;                 // of a sequence's tokens
    if ((uint64_t)a.b.seqs * 64 * (blocks <= 4 ? 4 : blocks <= 8 ? 8 : 16) > 0xFFFFFFFFull) return SZ_E_ARG;   // a launch's threads
    hipStream_t s = static_cast<hipStream_t>(stream);
    LaunchScope scope("sz_draft_tree", s);
    if (blocks <= 1)
        hipLaunchKernelGGL(sz_draft_tree_one, dim3((a.b.seqs + 3) / 4), dim3(256), 0, s, a);
    else if (blocks <= 2)
        hipLaunchKernelGGL(sz_draft_tree_many<2>, dim3(a.b.seqs), dim3(128), 0, s, a);
    else if (blocks <= 4)
        hipLaunchKernelGGL(sz_draft_tree_many<4>, dim3(a.b.seqs), dim3(256), 0, s, a);
    else if (blocks <= 8)
        hipLaunchKernelGGL(sz_draft_tree_many<8>, dim3(a.b.seqs), dim3(512), 0, s, a);
    else
        hipLaunchKernelGGL(sz_draft_tree_many<16>, dim3(a.b.seqs), dim3(1024), 0, s, a);
    return hipGetLastError() == hipSuccess ? SZ_OK : SZ_E_HIP;
}

extern "C" int sz_cache_keep(const sz_cache *caches, uint32_t layers, const sz_batch *batch, const int32_t *d_kept,
                             uint32_t kept_width, const int32_t *d_counts, int32_t *d_status, void *stream)
{
    if (!caches || layers == 0 || layers > SZ_KEEP_LAYERS) return SZ_E_ARG;
    PagedCache c;
    KeepArgs a{};
    for (uint32_t i = 0; i < layers; ++i) {
        const sz_cache &x = caches[i], &first = caches[0];
        const int rc = check_paged(&x, batch, d_status, c, a.b);
        if (rc != SZ_OK) return rc;
        if (x.dtype != first.dtype || x.page_tokens != first.page_tokens || x.kv_heads != first.kv_heads ||
            x.head_dim != first.head_dim || x.pages != first.pages)
            return SZ_E_ARG;
    }
    if ((reinterpret_cast<uintptr_t>(d_kept) | reinterpret_cast<uintptr_t>(d_counts)) & 3u) return SZ_E_ALIGN;
    if (a.b.tokens == 0 || a.b.seqs == 0 || kept_width == 0) return SZ_OK;
    if (!d_kept || !d_counts || kept_width > kMaxTokens) return SZ_E_ARG;
    a.kept = d_kept;
    a.counts = d_counts;
    a.pages = c.pages;
    a.heads = c.heads;
    a.lg_page = c.lg_page;
    a.width = kept_width;
    hipStream_t s = static_cast<hipStream_t>(stream);
    for (uint32_t i0 = 0; i0 < layers; i0 += kLayers) {
        a.layers = std::min(layers - i0, kLayers);
        for (uint32_t i = 0; i < a.layers; ++i) {
            a.data[i] = static_cast<uint8_t *>(caches[i0 + i].data);
            a.scales[i] = static_cast<uint8_t *>(caches[i0 + i].scales);
        }
        // as many rows as a wave has in flight, unless that leaves the card without waves
        const uint64_t all = (uint64_t)a.b.seqs * a.layers * 2 * a.heads;
        const uint64_t rows = std::max<uint64_t>(1, std::min<uint64_t>(kKeepRows / kept_width, all / kKeepWaves));
        a.pairs_each = (uint32_t)std::min<uint64_t>(rows, 2 * a.heads);
        a.parts = (2 * a.heads + a.pairs_each - 1) / a.pairs_each;
        const uint64_t units = (uint64_t)a.b.seqs * a.layers * a.parts;
        const uint64_t groups = (units + 3) / 4;
        if (groups * 256 > 0xFFFFFFFFull) return SZ_E_ARG;               // a launch's threads
        if (caches->dtype == SZ_BF16)
            launch_keep<SZ_BF16>(a, caches->head_dim, (uint32_t)groups, s);
        else
            launch_keep<SZ_FP8_E5M2>(a, caches->head_dim, (uint32_t)groups, s);   // E4M3 rows are moved alike
    }
    return hipGetLastError() == hipSuccess ? SZ_OK : SZ_E_HIP;
}
