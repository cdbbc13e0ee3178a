// kv_pages.hip - page operations of a key/value cache for gfx950: checking,
// freeing, forking, reserving, copying and compacting pages.
//
// All state lives on the device: references of every page (i32, 0 = free),
// the page table [rows][width] and the lengths [rows]. Free pages are handed
// out in ascending order to the slots in call order: slot i's pages are the
// free pages of rank [take(0) + .. + take(i-1), + take(i)), and pages move in
// compaction by the same ranks, so no atomic decides a result. The ranks come
// from counts of 2,048 pages each (a block of 256 threads, 8 pages a thread),
// which every later block adds up for itself: the counts of a million pages
// are 512 words, cheaper to read again than another launch or a look-back.
// Bound: the launches and the dependent loads for a few rows (free, fork, reserve
// and copy for 24 rows: 2.7, 2.8, 3.3 + 5.3 and 2.8 us; for 4,096 rows and 410,000
// pages 3.6, 4.7, 4.2 + 9.2 and 6.2 us), HBM bytes of the copied pages where there
// are many.
#include "dd_internal.h"
#include "dd_kv.hpp"

namespace dd {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                             // pages of a thread
constexpr uint32_t kChunk = kThreads * kPer;        // pages of a block
constexpr uint32_t kNone = 0xffffffffu;

struct Table {
    int32_t *refs;
    int32_t *table;
    int32_t *lens;
    uint32_t npages, rows, width, tshift;
};

__device__ __forceinline__ bool page_ok(const Table &t, int32_t p)
{
    return p >= 0 && (uint32_t)p < t.npages;
}

// Columns that a row of `len` tokens uses; len is 0..width * page tokens.
__device__ __forceinline__ uint32_t columns(const Table &t, int64_t len)
{
    return (uint32_t)((len + (1 << t.tshift) - 1) >> t.tshift);
}

__device__ __forceinline__ bool len_ok(const Table &t, int64_t len)
{
    return len >= 0 && len <= ((int64_t)t.width << t.tshift);
}

__global__ __launch_bounds__(kThreads) void k_kv_check(KvView c, const int32_t *q_start,
                                                      uint32_t total, int appending,
                                                      uint8_t *status)
{
    __shared__ uint32_t bad;
    const uint32_t b = blockIdx.x;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    const int64_t len = c.lens[b];
    bool inval = len < 0 || len > ((int64_t)c.width << c.tshift);
    if (q_start) {
        const int64_t s0 = q_start[b], s1 = q_start[b + 1];
        inval |= s0 < 0 || s1 < s0 || s1 > total || (b == 0 && s0 != 0) ||
                 (b == c.rows - 1 && s1 != total);
        inval |= appending && s1 - s0 > len;
    }
    if (!inval) {
        const uint32_t n = (uint32_t)((len + (1 << c.tshift) - 1) >> c.tshift);
        for (uint32_t k = threadIdx.x; k < n; k += kThreads) {
            const int32_t p = c.table[(uint64_t)b * c.width + k];
            if (p < 0 || (uint32_t)p >= c.npages) bad = 1;      // every writer writes 1
        }
    }
    __syncthreads();
    if (threadIdx.x == 0)
        status[b] = inval ? DMADESC_KV_EINVAL : bad ? DMADESC_KV_EPAGE : DMADESC_KV_OK;
}

// As k_kv_check for a call that brings trees: also refuses requests of more new
// tokens than a tree may have, and parents that are no earlier token of theirs.
__global__ __launch_bounds__(kThreads) void k_kv_tree_check(KvView c, const int32_t *q_start,
                                                           const int32_t *parent, uint32_t total,
                                                           uint8_t *status)
{
    __shared__ uint32_t bad, wrong;
    const uint32_t b = blockIdx.x;
    if (threadIdx.x == 0) bad = wrong = 0;
    __syncthreads();
    const int64_t len = c.lens[b], s0 = q_start[b], s1 = q_start[b + 1], n = s1 - s0;
    const bool inval = len < 0 || len > ((int64_t)c.width << c.tshift) || s0 < 0 || n < 0 || s1 > total ||
                       (b == 0 && s0 != 0) || (b == c.rows - 1 && s1 != total) || n > len ||
                       n > (int64_t)DMADESC_TREE_MOST;
    if (!inval) {
        for (int64_t i = threadIdx.x; i < n; i += kThreads) {
            const int32_t p = parent[s0 + i];
            if (p < -1 || p >= i) wrong = 1;                    // every writer writes 1
        }
        const uint32_t pages = (uint32_t)((len + (1 << c.tshift) - 1) >> c.tshift);
        for (uint32_t k = threadIdx.x; k < pages; k += kThreads)
            if ((uint32_t)c.table[(uint64_t)b * c.width + k] >= c.npages) bad = 1;
    }
    __syncthreads();
    if (threadIdx.x == 0)
        status[b] = inval || wrong ? DMADESC_KV_EINVAL : bad ? DMADESC_KV_EPAGE : DMADESC_KV_OK;
}

// One block per listed row: drops the references of the columns past `keep`
// tokens and clears them.
__global__ __launch_bounds__(kThreads) void k_kv_free(Table t, const int32_t *row,
                                                     const int32_t *keep, uint8_t *status)
{
    const uint32_t i = blockIdx.x;
    const int32_t r = row[i];
    const int64_t left = keep ? keep[i] : 0;
    const int64_t len = r >= 0 && (uint32_t)r < t.rows ? t.lens[r] : -1;
    if (!len_ok(t, len) || left < 0) {
        if (threadIdx.x == 0) status[i] = DMADESC_KV_EINVAL;
        return;
    }
    __syncthreads();                                   // every thread has read the length
    const uint32_t from = columns(t, left < len ? left : len), to = columns(t, len);
    int32_t *const tab = t.table + (uint64_t)r * t.width;
    for (uint32_t k = from + threadIdx.x; k < t.width; k += kThreads) {
        if (k < to) {
            const int32_t p = tab[k];
            if (page_ok(t, p)) atomicSub(&t.refs[p], 1);   // a sum: any order, one result
        }
        tab[k] = -1;
    }
    if (threadIdx.x == 0) {
        if (left < len) t.lens[r] = (int32_t)left;
        status[i] = DMADESC_KV_OK;
    }
}

// One block per child: the parent's table row and length, a reference more
// for each of its pages.
__global__ __launch_bounds__(kThreads) void k_kv_fork(Table t, const int32_t *parent,
                                                     const int32_t *child, uint8_t *status)
{
    const uint32_t i = blockIdx.x;
    const int32_t p = parent[i], c = child[i];
    const bool in = p >= 0 && (uint32_t)p < t.rows && c >= 0 && (uint32_t)c < t.rows && p != c;
    const int64_t len = in ? t.lens[p] : -1;
    const bool ok = len_ok(t, len) && t.lens[c] == 0;
    __syncthreads();                                   // read before the length is written
    if (!ok) {
        if (threadIdx.x == 0) status[i] = DMADESC_KV_EINVAL;
        return;
    }
    const uint32_t used = columns(t, len);
    const int32_t *const from = t.table + (uint64_t)p * t.width;
    int32_t *const to = t.table + (uint64_t)c * t.width;
    for (uint32_t k = threadIdx.x; k < t.width; k += kThreads) {
        const int32_t page = from[k];
        to[k] = page;
        if (k < used && page_ok(t, page)) atomicAdd(&t.refs[page], 1);
    }
    if (threadIdx.x == 0) {
        t.lens[c] = (int32_t)len;
        status[i] = DMADESC_KV_OK;
    }
}

// ---------------------------------------------------------------- reserve ---

// Two launches. The first counts the free pages of every chunk of 2,048 and
// works out what every slot takes, with running sums within chunks of 256
// slots. In the second, a page's thread knows its rank among the free pages
// and finds the slot whose ranks hold it (the chunk of slots in LDS, then the
// slot among 256 running sums), so that no list of free pages is written and
// read between: a third launch cost 4 us and its call 3 us more. Slots' threads write what does not depend on a page.
struct ReserveArgs {
    Table t;
    const int32_t *slot, *n_new;
    uint32_t n;
    int32_t *src, *dst;
    uint8_t *status;
    uint32_t page_chunks, slot_chunks;
    uint32_t *free_count;      // [page chunks] free pages
    uint8_t *free_bits;        // [page chunks][256] which of a thread's 8 pages are free, on entry
    uint64_t *slot_sum;        // [slot chunks] pages taken
    uint32_t *take;            // [n] pages taken; bit 31: the last page is copied; kNone, kBadPage: refused
    uint64_t *upto;            // [n] pages taken by the chunk's slots up to this one
    uint32_t *from;            // [n] first table column the slot writes
};

constexpr uint32_t kShared = 1u << 31, kBadPage = kNone - 1;

__device__ __forceinline__ uint32_t taken(uint32_t take) { return take >= kBadPage ? 0u : take & ~kShared; }

// What slot i needs: its pages, whether its last page is shared and partly
// filled; kNone where the slot is refused, kBadPage where it is for that page.
__device__ __forceinline__ uint32_t slot_take(const ReserveArgs &a, uint32_t i, uint32_t &from)
{
    const Table &t = a.t;
    const int32_t r = a.slot[i];
    const int64_t add = a.n_new[i];
    from = 0;
    if (r < 0 || (uint32_t)r >= t.rows) return kNone;
    const int64_t len = t.lens[r];
    if (add < 0 || !len_ok(t, len) || !len_ok(t, len + add)) return kNone;
    if (add == 0) return 0;
    const uint32_t have = columns(t, len), want = columns(t, len + add);
    bool shared = false;
    if (len & ((1 << t.tshift) - 1)) {
        const int32_t last = t.table[(uint64_t)r * t.width + have - 1];
        if (!page_ok(t, last)) return kBadPage;
        shared = t.refs[last] > 1;
    }
    from = have - (shared ? 1u : 0u);
    return (want - from) | (shared ? kShared : 0u);
}

// Flags of the chunk's pages in page order: thread k holds pages 8k .. 8k+7.
template <typename Pred>
__device__ __forceinline__ uint32_t page_flags(const Table &t, uint32_t chunk, Pred pred)
{
    const uint32_t p0 = chunk * kChunk + threadIdx.x * kPer;
    uint32_t f = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (p0 + k < t.npages && pred(p0 + k, t.refs[p0 + k])) f |= 1u << k;
    return f;
}

template <typename T>
__device__ __forceinline__ T block_sum(T v, T *scratch)
{
    v = wave_sum(v);
    __syncthreads();
    if (lane() == 0) scratch[wave()] = v;
    __syncthreads();
    T s = 0;
#pragma unroll
    for (int k = 0; k < kThreads / kWave; ++k) s += scratch[k];
    return s;
}

__global__ __launch_bounds__(kThreads) void k_reserve_count(ReserveArgs a)
{
    __shared__ uint32_t scratch[kThreads / kWave];
    __shared__ uint64_t sums[kThreads / kWave];
    if (blockIdx.x < a.page_chunks) {
        const uint32_t f = page_flags(a.t, blockIdx.x, [](uint32_t, int32_t r) { return r == 0; });
        const uint32_t s = block_sum<uint32_t>(__popc(f), scratch);
        a.free_bits[blockIdx.x * kThreads + threadIdx.x] = (uint8_t)f;
        if (threadIdx.x == 0) a.free_count[blockIdx.x] = s;
        return;
    }
    const uint32_t chunk = blockIdx.x - a.page_chunks, i = chunk * kThreads + threadIdx.x;
    uint32_t take = 0, from = 0;
    if (i < a.n) take = slot_take(a, i, from);
    // In 64 bits: 256 slots may ask for up to 2^27 pages each.
    uint64_t all;
    const uint64_t before = block_excl_scan<kThreads, uint64_t>(taken(take), sums, &all);
    if (i < a.n) {
        a.take[i] = take;
        a.from[i] = from;
        a.upto[i] = before + taken(take);
    }
    if (threadIdx.x == 0) a.slot_sum[chunk] = all;
}

constexpr uint32_t kSums = 1024;                    // running sums kept in LDS

__global__ __launch_bounds__(kThreads) void k_reserve_give(ReserveArgs a)
{
    __shared__ uint64_t scratch[kThreads / kWave];
    __shared__ uint64_t sums[kSums];
    __shared__ uint16_t order[kChunk];
    const Table &t = a.t;
    const bool is_page = blockIdx.x < a.page_chunks;
    const uint32_t chunk = is_page ? blockIdx.x : blockIdx.x - a.page_chunks;

    uint64_t nfree = 0, before = 0;                 // free pages of all, of the chunks before
    for (uint32_t k = threadIdx.x; k < a.page_chunks; k += kThreads) {
        const uint32_t v = a.free_count[k];
        nfree += v;
        if (is_page && k < chunk) before += v;
    }
    nfree = block_sum(nfree, scratch);
    if (!is_page) {
        uint64_t first = 0;                         // pages of the slots of the chunks before
        for (uint32_t k = threadIdx.x; k < chunk; k += kThreads) first += a.slot_sum[k];
        first = block_sum(first, scratch);
        const uint32_t i = chunk * kThreads + threadIdx.x;
        if (i >= a.n) return;
        const uint32_t v = a.take[i];
        const bool full = taken(v) > 0 && first + a.upto[i] > nfree;
        const bool refused = v >= kBadPage;
        if (refused || full || !(v & kShared)) a.src[i] = a.dst[i] = -1;
        a.status[i] = v == kNone      ? DMADESC_KV_EINVAL
                      : v == kBadPage ? DMADESC_KV_EPAGE
                      : full          ? DMADESC_KV_ENOSPC
                                      : DMADESC_KV_OK;
        if (!refused && !full) t.lens[a.slot[i]] += a.n_new[i];
        return;
    }
    before = block_sum(before, scratch);
    // As the first launch found them: references drop in this one.
    const uint32_t f = a.free_bits[chunk * kThreads + threadIdx.x];
    __syncthreads();                                // scratch is read before it is reused
    uint64_t count;
    const uint64_t rank = before + block_excl_scan<kThreads, uint64_t>(__popc(f), scratch, &count);
    const uint64_t end = before + count;
    // The chunk's free pages in rank order, so that every thread takes one rank
    // at a time: the pages handed out are the first ones, all in a few chunks.
    for (int k = 0, at = (int)(rank - before); k < kPer; ++k)
        if (f >> k & 1) order[at++] = (uint16_t)(threadIdx.x * kPer + k);

    // Chunks of slots, kSums at a time; sums[k] is what the slots of chunks up to k take.
    uint64_t run = 0;
    for (uint32_t c0 = 0; c0 < a.slot_chunks && run < end; c0 += kSums) {
        const uint32_t m = a.slot_chunks - c0 < kSums ? a.slot_chunks - c0 : kSums;
        __syncthreads();
        const uint64_t start = run;
        for (uint32_t k0 = 0; k0 < m; k0 += kThreads) {
            const uint32_t k = k0 + threadIdx.x;
            const uint64_t v = k < m ? a.slot_sum[c0 + k] : 0;
            uint64_t all;
            const uint64_t ex = block_excl_scan<kThreads, uint64_t>(v, scratch, &all);
            if (k < m) sums[k] = run + ex + v;
            run += all;
        }
        __syncthreads();
        const uint64_t lo_rank = start > before ? start : before, hi_rank = run < end ? run : end;
        for (uint64_t mine = lo_rank + threadIdx.x; mine < hi_rank; mine += kThreads) {
            uint32_t lo = 0, hi = m;                // first chunk of slots with sums > mine
            while (lo < hi) {
                const uint32_t mid = (lo + hi) / 2;
                if (sums[mid] > mine) hi = mid;
                else lo = mid + 1;
            }
            const uint64_t first = lo ? sums[lo - 1] : start;
            const uint64_t in = mine - first;
            // First slot of it with upto > in: of 16 groups of 16, then of 16 slots, so
            // that there are two waits and not eight.
            const uint32_t s0 = (c0 + lo) * kThreads, last_slot = a.n - 1;
            uint32_t x = s0;
#pragma unroll
            for (int step = 16; step >= 1; step /= 16) {
                uint32_t below = 0;
#pragma unroll
                for (uint32_t g = 0; g < 15; ++g) {
                    const uint32_t at = x + (g + 1) * step - 1;
                    below += a.upto[at < last_slot ? at : last_slot] <= in ? 1u : 0u;
                }
                x += below * step;
            }
            const uint32_t v = a.take[x];
            const uint64_t upto = a.upto[x];
            if (first + upto > nfree) continue;     // the slot is refused: out of pages
            const uint32_t at = (uint32_t)(in - (upto - taken(v)));
            const uint32_t page = chunk * kChunk + order[mine - before];
            int32_t *const entry = t.table + (uint64_t)(uint32_t)a.slot[x] * t.width + a.from[x] + at;
            if (at == 0 && (v & kShared)) {
                const int32_t last = *entry;
                a.src[x] = last;
                a.dst[x] = (int32_t)page;
                atomicSub(&t.refs[last], 1);
            }
            *entry = (int32_t)page;
            t.refs[page] = 1;
        }
    }
}

// ---------------------------------------------------------------- compact ---

struct CompactArgs {
    Table t;
    int32_t *src, *dst;
    uint32_t cap;              // entries of src and dst: npages / 2
    int32_t *moves;
    uint32_t *live_count;      // [page chunks]
    uint32_t *rank;            // [npages] which mover a page is, or kNone
};

__global__ __launch_bounds__(kThreads) void k_compact_count(CompactArgs a)
{
    __shared__ uint32_t scratch[kThreads / kWave];
    const uint32_t f = page_flags(a.t, blockIdx.x, [](uint32_t, int32_t r) { return r > 0; });
    const uint32_t s = block_sum<uint32_t>(__popc(f), scratch);
    if (threadIdx.x == 0) a.live_count[blockIdx.x] = s;
}

// Movers (live pages at or past `live`, the number of live pages) and holes
// (free pages below it) in ascending order.
__global__ __launch_bounds__(kThreads) void k_compact_list(CompactArgs a)
{
    __shared__ uint32_t scratch[kThreads / kWave];
    const uint32_t chunks = gridDim.x;
    uint32_t live = 0, before = 0;
    for (uint32_t k = threadIdx.x; k < chunks; k += kThreads) {
        const uint32_t v = a.live_count[k];
        live += v;
        before += k < blockIdx.x ? v : 0u;
    }
    live = block_sum(live, scratch);
    before = block_sum(before, scratch);
    // Live pages below `live`: whole chunks and a part of one.
    const uint32_t edge = live / kChunk;
    uint32_t low = 0;
    for (uint32_t k = threadIdx.x; k < edge; k += kThreads) low += a.live_count[k];
    if (edge < chunks)
        low += __popc(page_flags(a.t, edge, [&](uint32_t p, int32_t r) { return r > 0 && p < live; }));
    low = block_sum(low, scratch);
    const uint32_t moves = live - low;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.moves = (int32_t)moves;

    const uint32_t f = page_flags(a.t, blockIdx.x, [](uint32_t, int32_t r) { return r > 0; });
    __syncthreads();                                   // scratch is read before it is reused
    uint32_t total;
    uint32_t rank = before + block_excl_scan<kThreads, uint32_t>(__popc(f), scratch, &total);
    const uint32_t p0 = blockIdx.x * kChunk + threadIdx.x * kPer;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const uint32_t p = p0 + k;
        if (p >= a.t.npages) break;
        const bool on = f >> k & 1;
        uint32_t mine = kNone;
        if (p < live) {
            if (!on && p - rank < a.cap) a.dst[p - rank] = (int32_t)p;     // hole
        } else if (on && rank - low < a.cap) {
            mine = rank - low;
            a.src[mine] = (int32_t)p;                                      // mover
        }
        a.rank[p] = mine;
        if (p >= moves && p < a.cap) a.src[p] = a.dst[p] = -1;             // past the list
        rank += on ? 1u : 0u;
    }
}

__global__ __launch_bounds__(kThreads) void k_compact_rename(CompactArgs a, uint64_t entries)
{
    const uint64_t step = (uint64_t)gridDim.x * kThreads;
    const uint32_t moves = (uint32_t)*a.moves;
    const uint64_t k0 = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
    for (uint64_t k = k0; k < entries; k += step) {
        const int32_t p = a.t.table[k];
        if (!page_ok(a.t, p)) continue;
        const uint32_t m = a.rank[p];
        if (m != kNone) a.t.table[k] = a.dst[m];
    }
    for (uint64_t k = k0; k < moves && k < a.cap; k += step) {
        const int32_t s = a.src[k], d = a.dst[k];
        a.t.refs[d] = a.t.refs[s];
        a.t.refs[s] = 0;
    }
}

// ------------------------------------------------------------------- copy ---

// Pieces of 16 KB (256 threads, four 16-byte loads in flight each), read and
// written past the caches, which the copied pages would only fill: 2,800 pages of
// 131 KB take 135 us, 5.5 TB/s, against 146 us with plain loads and stores.
constexpr uint32_t kPiece = kThreads * 64;

__global__ __launch_bounds__(kThreads) void k_kv_copy(uint8_t *pool, uint32_t npages,
                                                     uint64_t page_bytes, const int32_t *src,
                                                     const int32_t *dst, uint32_t n,
                                                     const int32_t *count, uint32_t pieces)
{
    uint32_t limit = n;
    if (count) {
        const int32_t c = *count;
        limit = c < 0 ? 0u : ((uint32_t)c < n ? (uint32_t)c : n);
    }
    const uint64_t items = (uint64_t)limit * pieces;
    for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const uint32_t k = (uint32_t)(it / pieces), piece = (uint32_t)(it % pieces);
        const int32_t s = src[k], d = dst[k];
        if (s < 0 || d < 0 || (uint32_t)s >= npages || (uint32_t)d >= npages || s == d) continue;
        const uint64_t at = (uint64_t)piece * kPiece + threadIdx.x * 16u;
        const uint8_t *const from = pool + (uint64_t)s * page_bytes;
        uint8_t *const to = pool + (uint64_t)d * page_bytes;
        u32x4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at + j * (kThreads * 16u) < page_bytes)
                x[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(from + at + j * (kThreads * 16u)));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at + j * (kThreads * 16u) < page_bytes)
                __builtin_nontemporal_store(x[j], reinterpret_cast<u32x4 *>(to + at + j * (kThreads * 16u)));
    }
}

Table table_of(const KvPageArgs &k)
{
    uint32_t sh = 0;
    while ((1u << sh) < k.page_tokens) ++sh;
    return Table{k.refs, k.table, k.lens, (uint32_t)k.npages, k.rows, k.width, sh};
}

// Chunks of n things, one at least (an empty pool still has its counts).
uint32_t chunks_of(uint64_t n, uint64_t per) { return n ? (uint32_t)((n + per - 1) / per) : 1u; }

}  // namespace

KvView kv_view(const dmadesc_kv_cache &c)
{
    uint32_t sh = 0;
    while ((1u << sh) < c.page_tokens) ++sh;
    const uint32_t code_bytes = c.kv_heads * c.page_tokens * c.dim;
    return KvView{static_cast<uint8_t *>(c.pool), c.table, c.lens,
                  kv_page_bytes(c.kv_heads, c.page_tokens, c.dim), (uint32_t)c.npages, c.rows,
                  c.width, c.kv_heads, sh, code_bytes, c.kv_heads * (c.page_tokens / kBlock)};
}

hipError_t launch_kv_check(const dmadesc_kv_cache &c, const int32_t *q_start, uint64_t total,
                           bool appending, uint8_t *status, hipStream_t s)
{
    k_kv_check<<<c.rows, kThreads, 0, s>>>(kv_view(c), q_start, (uint32_t)total, appending, status);
    return hipGetLastError();
}

hipError_t launch_kv_tree_check(const dmadesc_kv_cache &c, const int32_t *q_start,
                                const int32_t *parent, uint64_t total, uint8_t *status, hipStream_t s)
{
    k_kv_tree_check<<<c.rows, kThreads, 0, s>>>(kv_view(c), q_start, parent, (uint32_t)total, status);
    return hipGetLastError();
}

hipError_t launch_kv_free(const KvPageArgs &k, const int32_t *row, const int32_t *keep,
                          hipStream_t s)
{
    k_kv_free<<<k.n, kThreads, 0, s>>>(table_of(k), row, keep, k.status);
    return hipGetLastError();
}

hipError_t launch_kv_fork(const KvPageArgs &k, const int32_t *parent, const int32_t *child,
                          hipStream_t s)
{
    k_kv_fork<<<k.n, kThreads, 0, s>>>(table_of(k), parent, child, k.status);
    return hipGetLastError();
}

size_t ws_kv_reserve(uint64_t npages, uint64_t n)
{
    const uint32_t pc = chunks_of(npages, kChunk);
    return align256(4ull * pc) + align256((size_t)kThreads * pc) +
           align256(8ull * chunks_of(n, kThreads)) + 2 * align256(4ull * n) + align256(8ull * n);
}

hipError_t launch_kv_reserve(const KvPageArgs &k, const int32_t *slot, const int32_t *n_new,
                             int32_t *src, int32_t *dst, void *ws, hipStream_t s)
{
    const uint32_t pc = chunks_of(k.npages, kChunk), sc = chunks_of(k.n, kThreads);
    uint8_t *p = static_cast<uint8_t *>(ws);
    auto take = [&](size_t bytes) { uint8_t *const r = p; p += align256(bytes); return r; };
    ReserveArgs a{table_of(k), slot, n_new, k.n, src, dst, k.status, pc, sc,
                  nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
    a.free_count = reinterpret_cast<uint32_t *>(take(4ull * pc));
    a.free_bits = take((size_t)kThreads * pc);
    a.slot_sum = reinterpret_cast<uint64_t *>(take(8ull * sc));
    a.take = reinterpret_cast<uint32_t *>(take(4ull * k.n));
    a.upto = reinterpret_cast<uint64_t *>(take(8ull * k.n));
    a.from = reinterpret_cast<uint32_t *>(take(4ull * k.n));
    k_reserve_count<<<pc + sc, kThreads, 0, s>>>(a);
    k_reserve_give<<<pc + sc, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

size_t ws_kv_compact(uint64_t npages)
{
    return align256(4ull * chunks_of(npages, kChunk)) + align256(4ull * npages);
}

hipError_t launch_kv_compact(const KvPageArgs &k, int32_t *src, int32_t *dst, int32_t *moves,
                             void *ws, hipStream_t s)
{
    const uint32_t pc = chunks_of(k.npages, kChunk);
    uint8_t *p = static_cast<uint8_t *>(ws);
    CompactArgs a{table_of(k), src, dst, (uint32_t)(k.npages / 2), moves,
                  reinterpret_cast<uint32_t *>(p),
                  reinterpret_cast<uint32_t *>(p + align256(4ull * pc))};
    k_compact_count<<<pc, kThreads, 0, s>>>(a);
    k_compact_list<<<pc, kThreads, 0, s>>>(a);
    const uint64_t entries = (uint64_t)k.rows * k.width;
    const uint64_t most = entries > k.npages ? entries : k.npages;
    const uint64_t blocks = chunks_of(most, kThreads);
    k_compact_rename<<<(uint32_t)(blocks < 2048 ? blocks : 2048), kThreads, 0, s>>>(a, entries);
    return hipGetLastError();
}

hipError_t launch_kv_copy(void *pool, uint64_t npages, uint64_t page_bytes, const int32_t *src,
                          const int32_t *dst, uint64_t n, const int32_t *count, hipStream_t s)
{
    const uint32_t pieces = (uint32_t)((page_bytes + kPiece - 1) / kPiece);
    const uint64_t items = n * pieces;
    k_kv_copy<<<(uint32_t)(items < 65536 ? items : 65536), kThreads, 0, s>>>(
        static_cast<uint8_t *>(pool), (uint32_t)npages, page_bytes, src, dst, (uint32_t)n, count,
        pieces);
    return hipGetLastError();
}

}  // namespace dd
