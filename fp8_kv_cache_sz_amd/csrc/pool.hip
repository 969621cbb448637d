// Pages for sequences, from their lengths: the page table, the ring of free
// pages and the slots of new tokens, without the host seeing a length.
//
//   need_i = ceil(len_i / P)
//   take_i = max(need_i - held_i, 0)         give_i = max(held_i - need_i, 0)
//   A_i = sum take_j, j <= i                 B_i = sum give_j, j < i
//   sequence i is served where A_i <= count:
//     table[i][held_i + e] = queue[head + A_i - take_i + e],  e < take_i
//   and else its fresh entries become -1, which no call reads or writes at;
//     queue[head + count + B_i + e] = table[i][need_i + e],   e < give_i
//   (ring positions modulo the ring's size).
//
// Free pages leave at one end of a ring and come back at the other: what a
// call takes and what it gives never meet, so every entry moves by itself once
// the two prefix sums are known, and a page that was given up is not handed
// out again while the step that read it may still run.  The pages that are free
// and those that rows hold are the ring's size at most, unless a row holds what
// it does not own: what then comes back beyond the ring's free places, where it
// would meet the free pages that others read, is dropped and reported.
//
// Bound by latency: a launch, the lengths, the sums, the entries.  Up to
// kOneSeqs sequences every workgroup of one launch works out all sums for
// itself (they are a few KB, which the L2 has) and moves its share.  Where held
// or the ring's ends are updated in place, the workgroup that arrives last
// writes them, when all have read them; a count costs 4 to 11 ns, one after
// another, so beyond kOneCounts workgroups, as for more sequences, a launch of one
// workgroup sums and a second one moves.  Measured (MI355X): a step of 256
// sequences 5.6 us on the GPU (launch, lengths, sums, a page's number, its entry);
// 1,000 prompts of up to 2,048 tokens, 73,000 pages of 16 and 1.15M slots (9.8 MB)
// 10.1 us, in place 10.8.
#include "paged.hpp"

namespace sz {
namespace {

constexpr uint32_t kSumThreads = 1024;       // with 256, 1,000 prompts' slots (1.15M) take 18 us instead of 11
constexpr uint32_t kThreads = 256;
constexpr uint32_t kOneSeqs = 2048;          // of one launch: their moves fill 32 KB of LDS
constexpr uint32_t kWaveTokens = 256;        // four a lane
constexpr uint64_t kOneTokens = 1u << 18;    // that get slots, one a lane
// In place, one launch (two), prompts of pages of 16 whose slots make so many
// workgroups: 1,000 sequences 128 7.2 us (8.4), 196 7.9 (8.4), 254 8.8 (8.5), 281
// 12.2 (10.8); 256 sequences 196 7.4 (7.9), 281 11.8 (9.8); 16 sequences 128 6.8
// (7.7), 196 7.7 (7.6), 281 18.7 (15.6), and 69 of more tokens each 9.2 (7.9).
constexpr uint64_t kOneCounts = 128;
constexpr uint32_t kNothing = 0xFFFFFFFFu;
constexpr uint32_t kMaxPages = 1u << 30;     // ring positions: twice this stays in 32 bits
constexpr uint32_t kMany = 0x7FFFFFFFu;      // sums stop here: above any ring's pages

// What happens to a sequence, or happened: where its fresh entries come from
// behind the ring's head (kNothing: not served), where those it gives go to
// behind the free pages, what it held (kNothing: it contradicts itself) and
// what it needs.
struct Move {
    uint32_t take_at, give_at, held, need;
};

struct Pool {
    int32_t *queue;
    const int32_t *ends;
    int32_t *ends_out;
    const int32_t *held;
    int32_t *held_out;
    int32_t *table;           // the batch's, which this call writes
    int64_t *slots;           // or null
    uint4 *moves;             // [seqs] Moves and the ring's ends, large batches
    uint32_t pages, lg_page;
};

__device__ __forceinline__ Move want(const Pool &p, const PagedBatch &b, int32_t len, int32_t held)
{
    if (len < 0 || len > (int32_t)b.max_kv || held < 0 || (uint32_t)held > b.width) {
        flag_batch(b);
        return Move{kNothing, 0, kNothing, kNothing};
    }
    return Move{kNothing, 0, (uint32_t)held, ((uint32_t)len + (1u << p.lg_page) - 1) >> p.lg_page};
}
__device__ __forceinline__ uint32_t taken(const Move &m) { return m.need > m.held ? m.need - m.held : 0; }
__device__ __forceinline__ uint32_t given(const Move &m) { return m.held > m.need ? m.held - m.need : 0; }

// The ring's free pages; none if the two numbers contradict the ring.
struct Ring {
    uint32_t head, count, pages;
    __device__ __forceinline__ uint32_t at(uint32_t behind) const             // up to pages
    {
        const uint32_t x = head + behind;
        return x >= pages ? x - pages : x;
    }
    __device__ __forceinline__ uint32_t room() const { return pages - count; }       // of pages that come back
};
__device__ __forceinline__ Ring ring(const Pool &p, const PagedBatch &b)
{
    const int32_t head = p.ends[0], count = p.ends[1];
    if (head < 0 || (uint32_t)head >= p.pages || count < 0 || (uint32_t)count > p.pages) {
        flag_batch(b);
        return Ring{0, 0, p.pages};
    }
    return Ring{(uint32_t)head, (uint32_t)count, p.pages};
}

// Sums of pages stop at kMany.
__device__ __forceinline__ uint32_t plus(uint32_t x, uint32_t y) { return min(x + y, kMany); }
struct Pair {
    uint32_t take, give;
};
__device__ __forceinline__ Pair plus(Pair x, Pair y) { return Pair{plus(x.take, y.take), plus(x.give, y.give)}; }
// Over the first `lanes` lanes up to this one.
__device__ __forceinline__ Pair wave_sum(Pair x, int lanes)
{
    for (int d = 1; d < lanes; d *= 2) {
        const Pair y{(uint32_t)__shfl_up((int)x.take, d, 64), (uint32_t)__shfl_up((int)x.give, d, 64)};
        if (lane_id() >= (uint32_t)d) x = plus(x, y);
    }
    return x;
}
// Over the threads of a workgroup before this one; all: over all of them.
// Called by all threads.
__device__ __forceinline__ Pair group_sum(Pair *lds, Pair mine, Pair &all)
{
    const uint32_t wave = threadIdx.x / 64, waves = blockDim.x / 64, lane = lane_id();
    const Pair upto = wave_sum(mine, 64);
    __syncthreads();                                                 // what was there has been read
    if (lane == 63) lds[wave] = upto;
    __syncthreads();
    const Pair w = wave_sum(lds[min(lane, waves - 1)], 16);          // of at most 16 waves
    all = Pair{(uint32_t)__shfl((int)w.take, (int)waves - 1, 64), (uint32_t)__shfl((int)w.give, (int)waves - 1, 64)};
    const int last = (int)max(wave, 1u) - 1;
    Pair before{(uint32_t)__shfl((int)w.take, last, 64), (uint32_t)__shfl((int)w.give, last, 64)};
    if (wave == 0) before = Pair{0, 0};
    const Pair lanes{(uint32_t)__shfl_up((int)upto.take, 1, 64), (uint32_t)__shfl_up((int)upto.give, 1, 64)};
    return lane == 0 ? before : plus(before, lanes);
}

// A sequence's move, from the sums over those before it.
__device__ __forceinline__ Move placed(const Ring &r, Move m, Pair before)
{
    if (m.held != kNothing && plus(before.take, taken(m)) <= r.count) m.take_at = before.take;
    m.give_at = before.give;
    return m;
}
__device__ __forceinline__ void store_held(const Pool &p, uint32_t i, const Move &m)
{
    if (m.held == kNothing) {
        if (p.held_out != p.held) p.held_out[i] = p.held[i];
    } else {
        p.held_out[i] = (int32_t)(m.need > m.held && m.take_at == kNothing ? m.held : m.need);
    }
}

// The ring after the call.  A shortage is a state that the caller serves by and by:
// it is reported where nothing else is, so that what is wrong (plain stores, in
// this launch or an earlier call's) stays to be seen whichever comes first.
__device__ __forceinline__ void store_ends(const Pool &p, const PagedBatch &b, const Ring &r, uint32_t wanted, uint32_t served,
                                           uint32_t given)
{
    if (wanted > r.count) atomicCAS(b.status, SZ_OK, SZ_E_CAPACITY);
    if (given > r.room()) flag_batch(b);
    p.ends_out[0] = (int32_t)r.at(served);
    p.ends_out[1] = (int32_t)(r.count - served + min(given, r.room()));
}

// One sequence's entries, a wave's worth at a time.
__device__ __forceinline__ void move_entries(const Pool &p, const PagedBatch &b, const Ring &r, uint32_t i, const Move &m)
{
    int32_t *row = p.table + (uint64_t)i * b.width;
    for (uint32_t e = lane_id(); e < taken(m); e += 64)
        row[m.held + e] = m.take_at == kNothing ? -1 : p.queue[r.at(m.take_at + e)];
    const uint32_t fits = r.room() > m.give_at ? min(given(m), r.room() - m.give_at) : 0;
    for (uint32_t e = lane_id(); e < fits; e += 64)
        p.queue[r.at(r.count + m.give_at + e)] = row[m.need + e];
}

// Where the page of token t's place is read: the table's old entry, or the
// ring's free page that comes there.  The call writes neither: nobody waits for
// the new table.  row: in the page, or -1 for a token without a place.
template <typename Moves>
__device__ __forceinline__ const int32_t *page_at(const Pool &p, const PagedBatch &b, const Ring &r, const int32_t *starts,
                                                  const int32_t *lens, int32_t i, int32_t t, Moves moves, int32_t &row)
{
    const uint32_t j = (uint32_t)max(i, 0);
    const Move m = moves(j);
    const Sequence s = i < 0 ? Sequence{0, 0, 0} : checked(b, starts[j], starts[j + 1], lens[j]);
    const int32_t pos = s.len - s.n + (t - s.start);
    const uint32_t w = (uint32_t)pos >> p.lg_page;
    const bool there = m.held != kNothing && t >= s.start && t < s.start + s.n && pos >= 0, old = w < m.held;
    row = there && (old || m.take_at != kNothing) ? pos & ((1 << p.lg_page) - 1) : -1;
    if (row < 0) return p.queue;
    return old ? p.table + (uint64_t)j * b.width + w : p.queue + r.at(m.take_at + (w - m.held));
}

// The sequences of a wave's tokens t0 + 64 k + lane, k < COUNT, or -1.  The
// starts of the 64 sequences from t0's on come in one load.  Few of them begin
// among the wave's tokens: counted one after another (1,000 prompts: 9 us where
// a search takes 13); more: searched in registers.
template <int COUNT>
__device__ __forceinline__ void token_sequences(const PagedBatch &b, const int32_t *starts, uint32_t t0, int32_t (&seq)[COUNT])
{
    if (b.seqs == 0) {                               // and starts may be null
#pragma unroll
        for (int k = 0; k < COUNT; ++k) seq[k] = -1;
        return;
    }
    const int32_t first = wave_last_not_above(b.seqs + 1, t0, [&](uint32_t j) { return (int64_t)starts[j]; });
    const uint32_t base = (uint32_t)max(first, 0), lane = lane_id();
    const int32_t start = base + lane <= b.seqs ? starts[base + lane] : INT32_MAX;
    const int32_t top = __shfl(start, 63, 64), end = (int32_t)(t0 + 64 * COUNT - 1);
    uint64_t inside = __ballot(start > (int32_t)t0 && start <= end);
    if (__popcll(inside) <= 16 && top > end) {
#pragma unroll
        for (int k = 0; k < COUNT; ++k) seq[k] = first;
        for (; inside; inside &= inside - 1) {
            const int32_t at = __builtin_amdgcn_readlane(start, (int)__builtin_ctzll(inside));
#pragma unroll
            for (int k = 0; k < COUNT; ++k) seq[k] += (int32_t)(t0 + 64 * k + lane) >= at ? 1 : 0;
        }
#pragma unroll
        for (int k = 0; k < COUNT; ++k)
            if (seq[k] >= (int32_t)b.seqs || t0 + 64 * k + lane >= b.tokens) seq[k] = -1;
        return;
    }
#pragma unroll
    for (int k = 0; k < COUNT; ++k) {
        const int32_t t = (int32_t)(t0 + 64 * k + lane);
        uint32_t count = 0;                                          // of them up to t
#pragma unroll
        for (uint32_t step = 32; step; step /= 2)
            if (__shfl(start, (int)(count + step - 1), 64) <= t) count += step;
        if (count == 63 && top <= t) ++count;
        uint32_t i = base + count;
        if (count == 64)                                             // 64 sequences on, or more
            for (uint32_t past = b.seqs + 1; past > i;) {
                const uint32_t mid = i + (past - i) / 2;
                if (starts[mid] <= t)
                    i = mid + 1;
                else
                    past = mid;
            }
        seq[k] = i == 0 || i > b.seqs || t >= (int32_t)b.tokens ? -1 : (int32_t)i - 1;
    }
}

template <int COUNT, typename Moves>
__device__ __forceinline__ void store_slots(const Pool &p, const PagedBatch &b, const Ring &r, const int32_t *starts,
                                            const int32_t *lens, uint32_t t0, Moves moves)
{
    int32_t seq[COUNT];
    token_sequences(b, starts, t0, seq);
    int32_t row[COUNT];
    uint32_t page[COUNT];
#pragma unroll
    for (int k = 0; k < COUNT; ++k)
        page[k] = (uint32_t)*page_at(p, b, r, starts, lens, seq[k], (int32_t)(t0 + 64 * k + lane_id()), moves, row[k]);
#pragma unroll
    for (int k = 0; k < COUNT; ++k)
        if (t0 + 64 * k + lane_id() < b.tokens)
            p.slots[t0 + 64 * k + lane_id()] = row[k] < 0 || page[k] >= p.pages ? -1 : ((int64_t)page[k] << p.lg_page) + row[k];
}

// One launch: all sums in every workgroup, a share of the entries and tokens,
// EACH tokens a lane.
template <int EACH>
__global__ __launch_bounds__(kSumThreads) void sz_pages_assign_one(Pool p, PagedBatch b, uint32_t *arrived)
{
    constexpr uint32_t SEQS = kOneSeqs / kSumThreads;                // of a thread
    __shared__ Move moves[kOneSeqs];
    __shared__ Pair sums[kSumThreads / 64];
    __shared__ int32_t starts[kOneSeqs + 1], lens[kOneSeqs];
    __shared__ uint32_t last;
    const uint32_t wave = uniform(threadIdx.x / 64), waves = gridDim.x * (kSumThreads / 64), mine = blockIdx.x * (kSumThreads / 64) + wave;
    const Ring r = ring(p, b);
    Move m[SEQS];
    const uint32_t seqs_each = (b.seqs + kSumThreads - 1) / kSumThreads, i0 = threadIdx.x * seqs_each;
    int32_t len[SEQS], held[SEQS];
#pragma unroll
    for (uint32_t k = 0; k < SEQS; ++k) {
        const uint32_t i = min(i0 + min(k, seqs_each - 1), b.seqs - 1);
        len[k] = b.seqs ? b.lens[i] : 0;
        held[k] = b.seqs ? p.held[i] : 0;
    }
    if (p.slots && b.seqs) {
        for (uint32_t i = threadIdx.x; i <= b.seqs; i += kSumThreads) starts[i] = b.starts[i];
        for (uint32_t i = threadIdx.x; i < b.seqs; i += kSumThreads) lens[i] = b.lens[i];
    }
    Pair sum{0, 0}, all;
#pragma unroll
    for (uint32_t k = 0; k < SEQS; ++k) {
        m[k] = Move{kNothing, 0, kNothing, kNothing};
        if (k < seqs_each && i0 + k < b.seqs) m[k] = want(p, b, len[k], held[k]);
    }
#pragma unroll
    for (uint32_t k = 0; k < SEQS; ++k) sum = plus(sum, Pair{taken(m[k]), given(m[k])});
    Pair before = group_sum(sums, sum, all);
    uint32_t got = 0;
#pragma unroll
    for (uint32_t k = 0; k < SEQS; ++k) {
        if (k >= seqs_each || i0 + k >= b.seqs) break;
        m[k] = placed(r, m[k], before);
        before = plus(before, Pair{taken(m[k]), given(m[k])});
        if (m[k].take_at != kNothing) got += taken(m[k]);            // served: at most the ring's pages together
        moves[i0 + k] = m[k];
    }
    bool writes = blockIdx.x == 0;
    if (arrived) {
        // held and the ring's ends, which this call may write, are here: the
        // loads have been used.  Whoever counts last knows it of all.
        __syncthreads();
        if (threadIdx.x == 0) last = atomicInc(arrived, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (arrived) writes = last;
    if (writes) {
        uint32_t served = all.take;
        if (all.take > r.count) {
            Pair sum_got;
            group_sum(sums, Pair{got, 0}, sum_got);
            served = sum_got.take;
        }
#pragma unroll
        for (uint32_t k = 0; k < SEQS; ++k)
            if (k < seqs_each && i0 + k < b.seqs) store_held(p, i0 + k, m[k]);
        if (threadIdx.x == 0) store_ends(p, b, r, all.take, served, all.give);
    }
    const uint32_t t0 = mine * 64 * EACH;
    if (p.slots && t0 < b.tokens) store_slots<EACH>(p, b, r, starts, lens, t0, [&](uint32_t j) { return moves[j]; });
    for (uint32_t j0 = mine; j0 < b.seqs; j0 += 64 * waves) {        // every waves-th sequence, 64 looked at together
        const uint32_t j = j0 + lane_id() * waves;
        uint64_t some = __ballot(j < b.seqs && moves[min(j, b.seqs - 1)].need != moves[min(j, b.seqs - 1)].held);
        while (some) {
            const uint32_t x = j0 + (uint32_t)__builtin_ctzll(some) * waves;
            some &= some - 1;
            move_entries(p, b, r, x, moves[x]);
        }
    }
}

// The sums of a large batch, kSumThreads sequences at a time.
__global__ __launch_bounds__(kSumThreads) void sz_pages_assign_sum(Pool p, PagedBatch b)
{
    __shared__ Pair sums[kSumThreads / 64];
    const Ring r = ring(p, b);
    Pair base{0, 0}, all;
    uint32_t got = 0;
    for (uint32_t i0 = 0; i0 < b.seqs; i0 += kSumThreads) {
        const uint32_t i = i0 + threadIdx.x;
        Move m{kNothing, 0, kNothing, kNothing};
        if (i < b.seqs) m = want(p, b, b.lens[i], p.held[i]);
        const Pair before = group_sum(sums, Pair{taken(m), given(m)}, all);
        m = placed(r, m, plus(base, before));
        base = plus(base, all);
        if (i >= b.seqs) continue;
        if (m.take_at != kNothing) got += taken(m);
        p.moves[i] = make_uint4(m.take_at, m.give_at, m.held, m.need);
        store_held(p, i, m);
    }
    group_sum(sums, Pair{got, 0}, all);
    if (threadIdx.x == 0) {
        p.moves[b.seqs] = make_uint4(r.head, r.count, 0, 0);         // ends_out may be ends
        store_ends(p, b, r, base.take, all.take, base.give);
    }
}

// The entries and slots of a large batch: in the first `fills` workgroups a
// wave takes a sequence, in the others kWaveTokens tokens.
__global__ __launch_bounds__(kThreads) void sz_pages_assign_move(Pool p, PagedBatch b, uint32_t fills)
{
    const uint4 ends = p.moves[b.seqs];
    const Ring r{ends.x, ends.y, p.pages};
    const auto move = [&](uint32_t j) {
        const uint4 x = p.moves[j];
        return Move{x.x, x.y, x.z, x.w};
    };
    const uint32_t wave = threadIdx.x / 64;
    if (blockIdx.x < fills) {
        const uint32_t i = uniform(blockIdx.x * (kThreads / 64) + wave);
        if (i < b.seqs) move_entries(p, b, r, i, move(i));
        return;
    }
    const uint64_t from = ((uint64_t)(blockIdx.x - fills) * (kThreads / 64) + wave) * kWaveTokens;
    if (from >= b.tokens) return;
    const uint32_t t0 = uniform((uint32_t)from);
    store_slots<kWaveTokens / 64>(p, b, r, b.starts, b.lens, t0, move);
}

}  // namespace
}  // namespace sz

using namespace sz;

extern "C" uint64_t sz_pages_assign_workspace_size(const sz_batch *batch)
{
    return batch ? (uint32_t)SZ_ASSIGN_COUNTERS + up256(16 * ((uint64_t)batch->seqs + 1)) : 0;
}

extern "C" int sz_pages_assign(const sz_pool *pool, const sz_batch *batch, const int32_t *d_held, int32_t *d_held_out,
                               int32_t *d_ends_out, int64_t *d_slots, void *d_ws, uint64_t ws_bytes, int32_t *d_status,
                               void *stream)
{
    if (!pool || !batch) return SZ_E_ARG;
    PagedBatch b;
    int rc = check_batch(batch, d_status, b);
    if (rc != SZ_OK) return rc;
    if (!d_status) return SZ_E_ARG;
    Pool p{};
    if ((rc = page_size(pool->page_tokens, p.lg_page)) != SZ_OK) return rc;
    if (pool->pages == 0 || pool->pages > kMaxPages || !pool->queue || !pool->ends || !d_ends_out) return SZ_E_ARG;
    if ((uint64_t)b.max_kv > (uint64_t)b.width * pool->page_tokens) return SZ_E_ARG;
    for (const void *x : {(const void *)pool->queue, (const void *)pool->ends, (const void *)d_held, (const void *)d_held_out,
                          (const void *)d_ends_out})
        if (reinterpret_cast<uintptr_t>(x) & 3u) return SZ_E_ALIGN;
    if (reinterpret_cast<uintptr_t>(d_slots) & 7u || !aligned16(d_ws)) return SZ_E_ALIGN;
    if (!d_ws || (b.seqs && (!d_held || !d_held_out))) return SZ_E_ARG;
    if (ws_bytes < sz_pages_assign_workspace_size(batch)) return SZ_E_WORKSPACE;
    p.queue = pool->queue;
    p.ends = pool->ends;
    p.ends_out = d_ends_out;
    p.held = d_held;
    p.held_out = d_held_out;
    p.table = const_cast<int32_t *>(b.table);
    p.slots = b.tokens ? d_slots : nullptr;
    p.moves = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(d_ws) + (uint32_t)SZ_ASSIGN_COUNTERS);
    p.pages = pool->pages;
    hipStream_t s = static_cast<hipStream_t>(stream);
    // one token a lane as long as the card has room for the waves
    const uint64_t slots = p.slots ? b.tokens : 0;
    const uint32_t each = slots <= kOneTokens ? 1 : kWaveTokens / 64;
    const uint64_t groups = std::max<uint64_t>({1, (slots + kSumThreads * each - 1) / (kSumThreads * each), (b.seqs + 127) / 128});
    const bool in_place = (d_held_out == d_held && b.seqs) || d_ends_out == pool->ends;
    if (b.seqs <= kOneSeqs && (!in_place || groups <= kOneCounts)) {
        uint32_t *arrived = in_place && groups > 1 ? static_cast<uint32_t *>(d_ws) : nullptr;
        LaunchScope scope("sz_pages_assign", s);
        const dim3 grid((uint32_t)groups), block(kSumThreads);
        if (each == 1)
            hipLaunchKernelGGL(sz_pages_assign_one<1>, grid, block, 0, s, p, b, arrived);
        else
            hipLaunchKernelGGL(sz_pages_assign_one<kWaveTokens / 64>, grid, block, 0, s, p, b, arrived);
    } else {
        const uint32_t fills = (b.seqs + 3) / 4;
        const uint32_t tokens = p.slots ? (b.tokens + 4 * kWaveTokens - 1) / (4 * kWaveTokens) : 0;
        {
            LaunchScope scope("sz_pages_assign_sum", s);
            hipLaunchKernelGGL(sz_pages_assign_sum, dim3(1), dim3(kSumThreads), 0, s, p, b);
        }
        LaunchScope scope("sz_pages_assign_move", s);
        hipLaunchKernelGGL(sz_pages_assign_move, dim3(fills + tokens), dim3(kThreads), 0, s, p, b, fills);
    }
    return hipGetLastError() == hipSuccess ? SZ_OK : SZ_E_HIP;
}
