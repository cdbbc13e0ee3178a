// kv_read.hip - keys and values of a paged 8-bit cache back in 16 or 32 bits,
// for gfx950.
//
// Mathematics: a value is its code times its block's scale 2^e, an exact f32
// product, rounded once to the output's type.
//
// Work split: as kv_append's, one wave to a block of 16 tokens of one head of K
// or of V. A lane stores kVals values of a token in one go; a token's row of
// one head is D / kVals lanes. V's codes lie by dimension, 16 tokens together:
// a lane takes kVals dimensions of a few tokens and turns them in registers.
// Bound: HBM. 43,000 tokens of 8 heads of 128, e4m3 to bf16: 54 us, 262 MB read and
// written, 4.8 TB/s (a large copy: 4.7); 14,000 tokens of 3 heads of 64, int8 to f32:
// 15.6 us, 5.0 TB/s. Stores past the caches: 72 us before, 64 after; six waves a SIMD
// (48 registers; the compiler took 66 to 248): 57 to 54, D = 128 to f32 106 to 73.
#include <type_traits>

#include "dd_internal.h"
#include "dd_kv.hpp"

namespace dd {
namespace {

constexpr int kThreads = 256;

struct ReadArgs {
    KvView c;
    const int32_t *first, *start;
    uint32_t total, items;
    void *k, *v;
    int64_t k_tok, k_head, v_tok, v_head;   // strides in elements
};

template <int kCodes>
__device__ __forceinline__ float code_value(uint32_t byte)
{
    if constexpr (kCodes == DMADESC_KV_E4M3) return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
    else return (float)(int8_t)byte;
}

// 16 bytes of consecutive values in one store, past the caches: nothing here reads
// them again.
template <int kType, int kVals>
__device__ __forceinline__ void put(void *out, int64_t at, const float (&x)[kVals])
{
    u32x4 w;
    if constexpr (kType == DMADESC_KV_FP32) {
        __builtin_memcpy(&w, x, sizeof w);
    } else if constexpr (kType == DMADESC_KV_BF16) {
        __bf16 y[kVals];
#pragma unroll
        for (int i = 0; i < kVals; ++i) y[i] = (__bf16)x[i];
        __builtin_memcpy(&w, y, sizeof w);
    } else {
        _Float16 y[kVals];
#pragma unroll
        for (int i = 0; i < kVals; ++i) y[i] = (_Float16)x[i];
        __builtin_memcpy(&w, y, sizeof w);
    }
    constexpr int kSize = 16 / kVals;
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4 *>(static_cast<uint8_t *>(out) + at * kSize));
}

template <int kD, int kType, int kCodes>
__global__ __launch_bounds__(kThreads, 6) void k_kv_read(ReadArgs a)
{
    constexpr int kVals = kType == DMADESC_KV_FP32 ? 4 : 8;     // values of a store
    constexpr int kLanes = kD / kVals;                          // lanes of a row
    constexpr int kRows = kWave / kLanes;                       // rows at a time
    constexpr int kRounds = kBlock / kRows;
    // Rows of whole 128-byte lines, read 8 bytes a lane, go past the caches: 57 us
    // against 60 for the prompts above, D = 256 47 against 57. Half lines (D = 64, 17.4
    // against 14.1) and 4 bytes a lane (f32, 23 against 16.7) do not.
    constexpr bool kStream = kD >= 128 && kVals == 8;
    const KvView &c = a.c;
    const uint64_t unit = (uint64_t)blockIdx.x * (kThreads / kWave) + wave();
    const uint32_t head = (uint32_t)(unit % c.kv_heads);
    const uint32_t is_v = (uint32_t)(unit / c.kv_heads) & 1u;
    const uint32_t item = (uint32_t)(unit / c.kv_heads / 2);
    if (item >= a.items) return;
    uint32_t s0, s1;
    int len;
    const uint32_t b = kv_blocks_of(c, a.start, a.total, item, s0, s1, len);
    const int64_t first = a.first ? a.first[b] : 0, count = s1 - s0;
    const int64_t nth = (int64_t)item - ((int64_t)(s0 / kBlock) + 2 * (int64_t)b);
    const int64_t block = (first >> 4) + nth;
    if (nth < 0 || block * kBlock >= first + count) return;
    const int per = (int)c.tshift - 4;
    const uint32_t sub = (uint32_t)block & ((1u << per) - 1u);
    const int ln = lane();
    const int r0 = ln / kLanes, d0 = ln % kLanes * kVals;
    const int64_t row0 = (int64_t)s0 + block * kBlock - first;  // output row of place 0
    // Places lo .. hi - 1 are asked for; from `end` on there is nothing to read.
    const int lo = first > block * kBlock ? (int)(first - block * kBlock) : 0;
    const int hi = first + count < (block + 1) * kBlock ? (int)(first + count - block * kBlock) : kBlock;
    const int64_t left = len - block * kBlock;
    int end = block < 0 || left < 0 ? 0 : left < kBlock ? (int)left : kBlock;
    uint32_t page = 0;
    if (end > 0) {                                              // inside the table, as len is
        page = (uint32_t)c.table[(uint64_t)b * c.width + ((uint32_t)block >> per)];
        if (page >= c.npages) end = 0;
    }
    const uint8_t *const base = c.pool + (uint64_t)page * c.page_bytes;
    float scale = 0.0f;
    if (end > 0)
        scale = reinterpret_cast<const float *>(base + 2ull * c.code_bytes)[(is_v ? c.scales : 0u) +
                                                                           ((head << per) + sub)];
    const uint8_t *const codes = base + (is_v ? c.code_bytes : 0u) + (uint64_t)((head << per) + sub) * (kBlock * kD);
    void *const out = is_v ? a.v : a.k;
    const int64_t tok = is_v ? a.v_tok : a.k_tok, at0 = head * (is_v ? a.v_head : a.k_head) + d0;

    if (!is_v) {
        typedef typename std::conditional<kVals == 8, u32x2, uint32_t>::type Word;
        Word w[kRounds];
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int r = r0 + i * kRows;
            w[i] = Word{};
            const Word *const from = reinterpret_cast<const Word *>(codes + r * kD + d0);
            if (r < end) w[i] = kStream ? __builtin_nontemporal_load(from) : *from;
        }
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int r = r0 + i * kRows;
            uint32_t q[2];
            __builtin_memcpy(q, &w[i], sizeof(Word));
            float x[kVals];
#pragma unroll
            for (int j = 0; j < kVals; ++j) x[j] = r < end ? code_value<kCodes>(q[j / 4] >> (8 * (j & 3)) & 0xffu) * scale : 0.0f;
            if (r >= lo && r < hi) put<kType>(out, (row0 + r) * tok + at0, x);
        }
    } else {
        // The lane's places r0 * kRounds .. + kRounds - 1 of dimensions d0 .. + kVals - 1.
        typedef typename std::conditional<kRounds == 16, u32x4,
                typename std::conditional<kRounds == 8, u32x2,
                typename std::conditional<kRounds == 4, uint32_t, uint16_t>::type>::type>::type Run;
        Run w[kVals];
#pragma unroll
        for (int j = 0; j < kVals; ++j) {
            w[j] = Run{};
            if (end > 0) w[j] = *reinterpret_cast<const Run *>(codes + (d0 + j) * kBlock + r0 * kRounds);
        }
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int r = r0 * kRounds + i;
            float x[kVals];
#pragma unroll
            for (int j = 0; j < kVals; ++j) {
                uint8_t q[sizeof(Run)];
                __builtin_memcpy(q, &w[j], sizeof(Run));
                x[j] = r < end ? code_value<kCodes>(q[i]) * scale : 0.0f;
            }
            if (r >= lo && r < hi) put<kType>(out, (row0 + r) * tok + at0, x);
        }
    }
}

template <int kD, int kType>
void launch_codes(const ReadArgs &a, uint32_t codes, uint32_t grid, hipStream_t s)
{
    if (codes == DMADESC_KV_E4M3) k_kv_read<kD, kType, DMADESC_KV_E4M3><<<grid, kThreads, 0, s>>>(a);
    else k_kv_read<kD, kType, DMADESC_KV_INT8><<<grid, kThreads, 0, s>>>(a);
}

template <int kD>
void launch_type(const ReadArgs &a, uint32_t type, uint32_t codes, uint32_t grid, hipStream_t s)
{
    if (type == DMADESC_KV_BF16) launch_codes<kD, DMADESC_KV_BF16>(a, codes, grid, s);
    else if (type == DMADESC_KV_FP16) launch_codes<kD, DMADESC_KV_FP16>(a, codes, grid, s);
    else launch_codes<kD, DMADESC_KV_FP32>(a, codes, grid, s);
}

// As k_kv_check, of what kv_read takes.
__global__ __launch_bounds__(kThreads) void k_kv_read_check(KvView c, const int32_t *first, const int32_t *start,
                                                           uint32_t total, uint8_t *status)
{
    __shared__ uint32_t bad;
    const uint32_t b = blockIdx.x;
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    const int64_t len = c.lens[b], s0 = start[b], s1 = start[b + 1], from = first ? first[b] : 0;
    const bool inval = len < 0 || len > ((int64_t)c.width << c.tshift) || s0 < 0 || s1 < s0 || s1 > total ||
                       (b == 0 && s0 != 0) || (b == c.rows - 1 && s1 != total) || from < 0 ||
                       from + (s1 - s0) > len;
    if (!inval && s1 > s0) {
        const uint32_t n = (uint32_t)((from + (s1 - s0) + (1 << c.tshift) - 1) >> c.tshift);
        for (uint32_t k = (uint32_t)(from >> c.tshift) + threadIdx.x; k < n; k += kThreads)
            if ((uint32_t)c.table[(uint64_t)b * c.width + k] >= c.npages) bad = 1;    // every writer writes 1
    }
    __syncthreads();
    if (threadIdx.x == 0) status[b] = inval ? DMADESC_KV_EINVAL : bad ? DMADESC_KV_EPAGE : DMADESC_KV_OK;
}

}  // namespace

uint64_t kv_read_groups(uint64_t total, uint32_t rows, uint32_t kv_heads)
{
    return ((total / kBlock + 2ull * rows) * 2 * kv_heads + 3) / 4;
}

hipError_t launch_kv_read(const KvReadArgs &k, hipStream_t s)
{
    ReadArgs a{kv_view(k.cache), k.first, k.start, (uint32_t)k.total,
               (uint32_t)(k.total / kBlock + 2ull * k.cache.rows), k.k, k.v, k.k_tok, k.k_head, k.v_tok, k.v_head};
    if (a.c.npages == 0) a.c.width = 0;                         // no page: every length is 0
    const uint32_t grid = (uint32_t)kv_read_groups(k.total, k.cache.rows, k.cache.kv_heads);
    if (k.cache.dim == 64) launch_type<64>(a, k.type, k.cache.codes, grid, s);
    else if (k.cache.dim == 128) launch_type<128>(a, k.type, k.cache.codes, grid, s);
    else launch_type<256>(a, k.type, k.cache.codes, grid, s);
    return hipGetLastError();
}

hipError_t launch_kv_read_check(const dmadesc_kv_cache &c, const int32_t *first, const int32_t *start,
                                uint64_t total, uint8_t *status, hipStream_t s)
{
    k_kv_read_check<<<c.rows, kThreads, 0, s>>>(kv_view(c), first, start, (uint32_t)total, status);
    return hipGetLastError();
}

}  // namespace dd
