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
// out again while the step that read it may still run.
//
// Bound by latency: a launch, the lengths, the sums, the entries.  A small
// batch is one workgroup's; of a large one a workgroup sums and a second
// launch, as wide as the batch, moves.
#include "paged.hpp"

namespace sz {
namespace {

constexpr uint32_t kSumThreads = 1024;
constexpr uint32_t kSmallSeqs = 1024;        // a thread each
constexpr uint64_t kSmallPages = 4096;       // that the new tokens may fill
constexpr uint32_t kSmallTokens = 4096;      // that get slots
constexpr uint32_t kMoveGroup = 256;
constexpr uint32_t kNothing = 0xFFFFFFFFu;
constexpr uint32_t kMaxPages = 1u << 30;     // ring positions: four times this stays in 32 bits

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

__device__ __forceinline__ Move want(const Pool &p, const PagedBatch &b, uint32_t i)
{
    const int32_t len = b.lens[i], held = p.held[i];
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
    __device__ __forceinline__ uint32_t at(uint32_t behind) const             // below 3 pages
    {
        uint32_t x = head + behind;
#pragma unroll
        for (int k = 0; k < 3; ++k) x = x >= pages ? x - pages : x;
        return x;
    }
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

// Sum over the lanes up to this one.
__device__ __forceinline__ uint64_t wave_sum_up_to(uint64_t x)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint64_t y = __shfl_up(x, d, 64);
        if (lane_id() >= (uint32_t)d) x += y;
    }
    return x;
}

// Sums over the workgroup's threads up to this one, and over all of them.
// Called by all threads; lds holds a wave's sums.
struct Sums {
    uint64_t take[kSumThreads / 64], give[kSumThreads / 64];
};
__device__ __forceinline__ void group_sums(Sums &lds, uint64_t &take, uint64_t &give, uint64_t &all_take, uint64_t &all_give)
{
    const uint32_t wave = threadIdx.x / 64, lane = lane_id();
    take = wave_sum_up_to(take);
    give = wave_sum_up_to(give);
    __syncthreads();                                                 // what was there has been read
    if (lane == 63) {
        lds.take[wave] = take;
        lds.give[wave] = give;
    }
    __syncthreads();
    all_take = all_give = 0;
    for (uint32_t w = 0; w < blockDim.x / 64; ++w) {
        if (w == wave) {
            take += all_take;
            give += all_give;
        }
        all_take += lds.take[w];
        all_give += lds.give[w];
    }
}

// With the sums up to a sequence, its own included.
__device__ __forceinline__ bool served(const Ring &r, const Move &m, uint64_t take) { return m.held != kNothing && take <= r.count; }
__device__ __forceinline__ Move placed(const Ring &r, Move m, uint64_t take, uint64_t give)
{
    if (served(r, m, take)) m.take_at = (uint32_t)take - taken(m);
    give -= given(m);
    m.give_at = give < r.pages ? (uint32_t)give : 0;                 // over that: reported with the ends
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

// The ring after the call.  More pages than the ring has: some sequence holds
// what it does not own.
__device__ __forceinline__ void store_ends(const Pool &p, const PagedBatch &b, const Ring &r, uint64_t all_taken, uint64_t all_given)
{
    uint64_t count = r.count - all_taken + all_given;
    if (count > r.pages) {
        flag_batch(b);
        count = r.pages;
    }
    p.ends_out[0] = (int32_t)r.at((uint32_t)all_taken);
    p.ends_out[1] = (int32_t)count;
}

// One sequence's entries, a wave's worth at a time.
__device__ __forceinline__ void move_entries(const Pool &p, const PagedBatch &b, const Ring &r, uint32_t i, const Move &m)
{
    int32_t *row = p.table + (uint64_t)i * b.width;
    for (uint32_t e = lane_id(); e < taken(m); e += 64)
        row[m.held + e] = m.take_at == kNothing ? -1 : p.queue[r.at(m.take_at + e)];
    const uint32_t most = min(given(m), r.pages);
    for (uint32_t e = lane_id(); e < most; e += 64)
        p.queue[r.at(r.count + m.give_at + e)] = row[m.need + e];
}

// Token t's slot after the call, or -1.  Its page is read from where the
// table's entry comes from, the old table or the free pages, neither of which
// the call writes: nobody waits for the new table.
template <typename Moves>
__device__ __forceinline__ int64_t slot_of(const Pool &p, const PagedBatch &b, const Ring &r, int32_t i, int32_t t, Moves moves)
{
    if (i < 0 || t >= (int32_t)b.tokens) return -1;
    const Move m = moves((uint32_t)i);
    const Sequence s = sequence(b, (uint32_t)i);
    const int32_t pos = s.len - s.n + (t - s.start);
    if (m.held == kNothing || t < s.start || t >= s.start + s.n || pos < 0) return -1;
    const uint32_t w = (uint32_t)pos >> p.lg_page;
    uint32_t page = kNothing;
    if (w < m.held)
        page = (uint32_t)p.table[(uint64_t)(uint32_t)i * b.width + w];
    else if (m.take_at != kNothing)
        page = (uint32_t)p.queue[r.at(m.take_at + (w - m.held))];
    if (page >= p.pages) return -1;
    return ((int64_t)page << p.lg_page) + (pos & ((1 << p.lg_page) - 1));
}

// Token t's sequence, or -1: a wave's tokens from t0 on.  The starts of the 64
// sequences from t0's on come in one load and are searched in registers.
__device__ __forceinline__ int32_t token_sequence(const PagedBatch &b, uint32_t t0, uint32_t t)
{
    const int32_t first = wave_last_not_above(b.seqs + 1, t0, [&](uint32_t j) { return (int64_t)b.starts[j]; });
    const uint32_t base = (uint32_t)max(first, 0), lane = lane_id();
    const int32_t start = base + lane <= b.seqs ? b.starts[base + lane] : INT32_MAX;
    uint32_t count = 0;                                              // of them up to t
#pragma unroll
    for (uint32_t step = 32; step; step /= 2)
        if (__shfl(start, (int)(count + step - 1), 64) <= (int32_t)t) count += step;
    if (count == 63 && __shfl(start, 63, 64) <= (int32_t)t) ++count;
    uint32_t i = base + count;
    if (count == 64)                                                 // 64 sequences on, or more
        for (uint32_t past = b.seqs + 1; past > i;) {
            const uint32_t mid = i + (past - i) / 2;
            if (b.starts[mid] <= (int32_t)t)
                i = mid + 1;
            else
                past = mid;
        }
    return i == 0 || i > b.seqs ? -1 : (int32_t)i - 1;
}

// A small batch: a thread per sequence sums, threads take tokens, and waves
// move the entries of the sequences that have any.
__global__ __launch_bounds__(kSumThreads) void sz_pages_assign_small(Pool p, PagedBatch b)
{
    __shared__ Sums sums;
    __shared__ Move moves[kSmallSeqs];
    const uint32_t i = threadIdx.x;
    const Ring r = ring(p, b);
    Move m{kNothing, 0, kNothing, kNothing};
    if (i < b.seqs) m = want(p, b, i);
    uint64_t take = taken(m), give = given(m), all_take, all_give;
    group_sums(sums, take, give, all_take, all_give);
    m = placed(r, m, take, give);
    if (all_take > r.count) {                                        // of those that are served
        uint64_t some = m.take_at == kNothing ? 0 : taken(m), none = 0, no;
        if (i == 0) *b.status = SZ_E_CAPACITY;
        group_sums(sums, some, none, all_take, no);
    }
    moves[i] = m;
    __syncthreads();                                                 // held and ends, which may be the outputs, have been read
    if (i < b.seqs) store_held(p, i, m);
    if (i == 0) store_ends(p, b, r, all_take, all_give);
    if (p.slots)
        for (uint32_t t0 = uniform(threadIdx.x / 64 * 64); t0 < b.tokens; t0 += kSumThreads) {
            const uint32_t t = t0 + lane_id();
            const int64_t slot = slot_of(p, b, r, token_sequence(b, t0, t), (int32_t)t, [&](uint32_t j) { return moves[j]; });
            if (t < b.tokens) p.slots[t] = slot;
        }
    uint64_t some = __ballot(m.need != m.held);
    while (some) {
        const uint32_t j = threadIdx.x / 64 * 64 + (uint32_t)__builtin_ctzll(some);
        some &= some - 1;
        move_entries(p, b, r, j, moves[j]);
    }
}

// The sums of a large batch, kSumThreads sequences at a time.
__global__ __launch_bounds__(kSumThreads) void sz_pages_assign_sum(Pool p, PagedBatch b)
{
    __shared__ Sums sums;
    const Ring r = ring(p, b);
    uint64_t base_take = 0, base_give = 0, some = 0;
    for (uint32_t i0 = 0; i0 < b.seqs; i0 += kSumThreads) {
        const uint32_t i = i0 + threadIdx.x;
        Move m{kNothing, 0, kNothing, kNothing};
        if (i < b.seqs) m = want(p, b, i);
        uint64_t take = taken(m), give = given(m), all_take, all_give;
        group_sums(sums, take, give, all_take, all_give);
        m = placed(r, m, take + base_take, give + base_give);
        if (i < b.seqs) {
            if (m.take_at != kNothing) some += taken(m);
            p.moves[i] = make_uint4(m.take_at, m.give_at, m.held, m.need);
            store_held(p, i, m);
        }
        base_take += all_take;
        base_give += all_give;
    }
    uint64_t none = 0, all_some, no;
    group_sums(sums, some, none, all_some, no);
    if (threadIdx.x == 0) {
        if (base_take > r.count) *b.status = SZ_E_CAPACITY;
        p.moves[b.seqs] = make_uint4(r.head, r.count, 0, 0);         // ends_out may be ends
        store_ends(p, b, r, all_some, base_give);
    }
}

// The entries and slots of a large batch: in the first `fills` workgroups a
// wave takes a sequence, in the others kWaveTokens tokens.
constexpr uint32_t kWaveTokens = 256;
__global__ __launch_bounds__(kMoveGroup) void sz_pages_assign_move(Pool p, PagedBatch b, uint32_t fills)
{
    const uint4 ends = p.moves[b.seqs];
    const Ring r{ends.x, ends.y, p.pages};
    const auto move = [&](uint32_t j) {
        const uint4 x = p.moves[j];
        return Move{x.x, x.y, x.z, x.w};
    };
    const uint32_t wave = threadIdx.x / 64;
    if (blockIdx.x < fills) {
        const uint32_t i = uniform(blockIdx.x * (kMoveGroup / 64) + wave);
        if (i < b.seqs) move_entries(p, b, r, i, move(i));
        return;
    }
    const uint64_t from = ((uint64_t)(blockIdx.x - fills) * (kMoveGroup / 64) + wave) * kWaveTokens;
    for (uint32_t k = 0; k < kWaveTokens; k += 64) {
        if (from + k >= b.tokens) return;
        const uint32_t t0 = uniform((uint32_t)from + k), t = t0 + lane_id();
        const int64_t slot = slot_of(p, b, r, token_sequence(b, t0, t), (int32_t)t, move);
        if (t < b.tokens) p.slots[t] = slot;
    }
}

}  // namespace
}  // namespace sz

using namespace sz;

extern "C" uint64_t sz_pages_assign_workspace_size(const sz_batch *batch)
{
    return batch ? up256(16 * ((uint64_t)batch->seqs + 1)) : 0;
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
    if (b.seqs && (!d_held || !d_held_out || !d_ws)) return SZ_E_ARG;
    if (b.seqs && ws_bytes < sz_pages_assign_workspace_size(batch)) return SZ_E_WORKSPACE;
    p.queue = pool->queue;
    p.ends = pool->ends;
    p.ends_out = d_ends_out;
    p.held = d_held;
    p.held_out = d_held_out;
    p.table = const_cast<int32_t *>(b.table);
    p.slots = b.tokens ? d_slots : nullptr;
    p.moves = static_cast<uint4 *>(d_ws);
    p.pages = pool->pages;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const uint64_t fresh = (uint64_t)b.seqs * ((b.max_new >> p.lg_page) + 1);
    if (b.seqs <= kSmallSeqs && fresh <= kSmallPages && (!p.slots || b.tokens <= kSmallTokens)) {
        LaunchScope scope("sz_pages_assign_small", s);
        hipLaunchKernelGGL(sz_pages_assign_small, dim3(1), dim3(kSumThreads), 0, s, p, b);
    } else {
        const uint32_t fills = (b.seqs + 3) / 4;
        const uint32_t tokens = p.slots ? (b.tokens + 4 * kWaveTokens - 1) / (4 * kWaveTokens) : 0;
        {
            LaunchScope scope("sz_pages_assign_sum", s);
            hipLaunchKernelGGL(sz_pages_assign_sum, dim3(1), dim3(kSumThreads), 0, s, p, b);
        }
        if (fills + tokens) {
            LaunchScope scope("sz_pages_assign_move", s);
            hipLaunchKernelGGL(sz_pages_assign_move, dim3(fills + tokens), dim3(kMoveGroup), 0, s, p, b, fills);
        }
    }
    return hipGetLastError() == hipSuccess ? SZ_OK : SZ_E_HIP;
}
