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
// Bound: the launches and the dependent loads for a few rows, HBM bytes of
// the copied pages where there are many.
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

struct ReserveArgs {
    Table t;
    const int32_t *slot, *n_new;
    uint32_t n;
    int32_t *src, *dst;
    uint8_t *status;
    uint32_t *free_count;      // [page chunks] free pages
    uint64_t *slot_sum;        // [slot chunks] pages taken
    uint64_t *nfree;           // free pages of all
    uint32_t *take;            // [n] pages taken; bit 31: the last page is copied
    uint32_t *list;            // [npages] free pages by rank
};

constexpr uint32_t kShared = 1u << 31;

// What slot i needs: its pages, whether its last page is shared and partly
// filled; kNone where the slot is refused.
__device__ __forceinline__ uint32_t slot_take(const ReserveArgs &a, uint32_t i)
{
    const Table &t = a.t;
    const int32_t r = a.slot[i];
    if (r < 0 || (uint32_t)r >= t.rows) return kNone;
    const int64_t len = t.lens[r], add = a.n_new[i];
    if (add < 0 || !len_ok(t, len) || !len_ok(t, len + add)) return kNone;
    if (add == 0) return 0;
    const uint32_t have = columns(t, len), want = columns(t, len + add);
    bool shared = false;
    if (len & ((1 << t.tshift) - 1)) {
        const int32_t last = t.table[(uint64_t)r * t.width + have - 1];
        if (!page_ok(t, last)) return kNone;
        shared = t.refs[last] > 1;
    }
    return (want - have + (shared ? 1u : 0u)) | (shared ? kShared : 0u);
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

__global__ __launch_bounds__(kThreads) void k_reserve_count(ReserveArgs a, uint32_t page_chunks)
{
    __shared__ uint64_t scratch[kThreads / kWave];
    if (blockIdx.x < page_chunks) {
        const uint32_t f = page_flags(a.t, blockIdx.x, [](uint32_t, int32_t r) { return r == 0; });
        const uint64_t s = block_sum<uint64_t>(__popc(f), scratch);
        if (threadIdx.x == 0) a.free_count[blockIdx.x] = (uint32_t)s;
        return;
    }
    const uint32_t chunk = blockIdx.x - page_chunks, i = chunk * kThreads + threadIdx.x;
    uint32_t take = 0;
    if (i < a.n) {
        take = slot_take(a, i);
        a.take[i] = take;
    }
    const uint64_t s = block_sum<uint64_t>(take == kNone ? 0u : take & ~kShared, scratch);
    if (threadIdx.x == 0) a.slot_sum[chunk] = s;
}

__global__ __launch_bounds__(kThreads) void k_reserve_list(ReserveArgs a, uint32_t slot_chunks)
{
    __shared__ uint64_t scratch[kThreads / kWave];
    uint64_t before = 0, need = 0;
    for (uint32_t k = threadIdx.x; k < blockIdx.x; k += kThreads) before += a.free_count[k];
    for (uint32_t k = threadIdx.x; k < slot_chunks; k += kThreads) need += a.slot_sum[k];
    before = block_sum(before, scratch);
    need = block_sum(need, scratch);
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0)
        *a.nfree = before + a.free_count[blockIdx.x];
    if (before >= need) return;
    const uint32_t f = page_flags(a.t, blockIdx.x, [](uint32_t, int32_t r) { return r == 0; });
    __syncthreads();                                   // scratch is read before it is reused
    uint64_t total;
    uint64_t rank = before + block_excl_scan<kThreads, uint64_t>(__popc(f), scratch, &total);
    const uint32_t p0 = blockIdx.x * kChunk + threadIdx.x * kPer;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (f >> k & 1) {
            if (rank < need) a.list[rank] = p0 + k;
            ++rank;
        }
}

// One wave per slot.
__global__ __launch_bounds__(kThreads) void k_reserve_give(ReserveArgs a)
{
    const Table &t = a.t;
    const uint32_t i = blockIdx.x * (kThreads / kWave) + wave();
    if (i >= a.n) return;
    const uint32_t chunk = i / kThreads;
    uint64_t before = 0;
    for (uint32_t k = lane(); k < chunk; k += kWave) before += a.slot_sum[k];
    for (uint32_t k = chunk * kThreads + lane(); k < i; k += kWave) {
        const uint32_t v = a.take[k];
        before += v == kNone ? 0u : v & ~kShared;
    }
    before = wave_sum(before);
    const uint32_t v = a.take[i];
    const bool shared = v != kNone && (v & kShared) != 0;
    const uint32_t take = v == kNone ? 0u : v & ~kShared;
    const bool full = take > 0 && before + take > *a.nfree;
    if (v == kNone || full) {
        if (lane() == 0) {
            a.status[i] = full ? DMADESC_KV_ENOSPC : DMADESC_KV_EINVAL;
            a.src[i] = a.dst[i] = -1;
        }
        return;
    }
    const uint32_t r = (uint32_t)a.slot[i];
    const int64_t len = t.lens[r], add = a.n_new[i];
    const uint32_t from = columns(t, len) - (shared ? 1u : 0u);
    int32_t *const tab = t.table + (uint64_t)r * t.width;
    const int32_t last = shared ? tab[from] : -1;
    for (uint32_t k = lane(); k < take; k += kWave) {
        const uint32_t p = a.list[before + k];
        tab[from + k] = (int32_t)p;
        t.refs[p] = 1;
    }
    if (lane() == 0) {
        a.src[i] = last;
        a.dst[i] = shared ? (int32_t)a.list[before] : -1;
        if (shared) atomicSub(&t.refs[last], 1);
        t.lens[r] = (int32_t)(len + add);
        a.status[i] = DMADESC_KV_OK;
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

// Pieces of 16 KB (256 threads, four 16-byte loads in flight each).
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
                x[j] = *reinterpret_cast<const u32x4 *>(from + at + j * (kThreads * 16u));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at + j * (kThreads * 16u) < page_bytes)
                *reinterpret_cast<u32x4 *>(to + at + j * (kThreads * 16u)) = x[j];
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
    return align256(4ull * chunks_of(npages, kChunk)) + align256(8ull * chunks_of(n, kThreads) + 8) +
           align256(4ull * n) + align256(4ull * npages);
}

hipError_t launch_kv_reserve(const KvPageArgs &k, const int32_t *slot, const int32_t *n_new,
                             int32_t *src, int32_t *dst, void *ws, hipStream_t s)
{
    const uint32_t pc = chunks_of(k.npages, kChunk), sc = chunks_of(k.n, kThreads);
    uint8_t *p = static_cast<uint8_t *>(ws);
    ReserveArgs a{table_of(k), slot, n_new, k.n, src, dst, k.status,
                  nullptr, nullptr, nullptr, nullptr, nullptr};
    a.free_count = reinterpret_cast<uint32_t *>(p);
    p += align256(4ull * pc);
    a.nfree = reinterpret_cast<uint64_t *>(p);
    a.slot_sum = a.nfree + 1;
    p += align256(8ull * sc + 8);
    a.take = reinterpret_cast<uint32_t *>(p);
    p += align256(4ull * k.n);
    a.list = reinterpret_cast<uint32_t *>(p);
    k_reserve_count<<<pc + sc, kThreads, 0, s>>>(a, pc);
    k_reserve_list<<<pc, kThreads, 0, s>>>(a, sc);
    k_reserve_give<<<chunks_of(k.n, kThreads / kWave), kThreads, 0, s>>>(a);
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
    k_kv_copy<<<(uint32_t)(items < 4096 ? items : 4096), kThreads, 0, s>>>(
        static_cast<uint8_t *>(pool), (uint32_t)npages, page_bytes, src, dst, (uint32_t)n, count,
        pieces);
    return hipGetLastError();
}

}  // namespace dd
