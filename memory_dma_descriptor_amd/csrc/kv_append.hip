// kv_append.hip - quantising new keys and values into the pages of an 8-bit
// cache, for gfx950.
//
// Mathematics: a block is 16 tokens of one head of K or of V. Its scale is
// 2^e with the least e >= -64 for which every finite |x| of the block is at
// most c 2^e, c the largest code (448 or 127); a code is x 2^-e rounded once
// to the nearest, ties to even. Scales are powers of two so that products
// with them are exact: the code's rounding is the only one. A block that
// already holds earlier tokens keeps the larger of the two exponents, and
// where that grows the earlier codes are rounded again on the new grid.
// Tokens of the block past the request's length become zero.
//
// Work split: one wave owns one (block, head) of K or V, so a block's maximum
// is one wave reduction and no block is written by two waves. Blocks are
// numbered without a scan: request b's first number is q_start[b] / 16 + 2 b,
// which leaves room for the at most n / 16 + 2 blocks that n tokens touch;
// the wave finds its request by a 64-way search and waves without a block
// leave. K rows are read 8 values a lane, V two dimensions of 16 tokens a
// lane (D = 128), so that each side's codes leave in whole 8- and 16-byte
// stores in the page's own order and nothing passes through LDS.
// Bound: HBM bytes for prompts (20,000 tokens of 8 heads of 128, bf16 to e4m3:
// 34.0 us, 142 MB read and written, 4.2 TB/s; 5 prompts of f32, D = 256, to int8:
// 13.5 us, 49 MB, 3.6 TB/s), latency for single tokens (128 requests: 9.6 us, with
// the request search, then page, values and earlier block, and 16 places loaded
// where one is new).
#include <type_traits>

#include "dd_internal.h"
#include "dd_kv.hpp"
#include "dd_kv_codes.hpp"

namespace dd {
namespace {

struct AppendArgs {
    KvView c;
    const void *k, *v;
    int64_t k_tok, k_head, v_tok, v_head;   // strides in elements
    const int32_t *q_start;
    uint32_t total;
    uint32_t items;                         // block numbers
};

// kN consecutive values as they lie in memory, and as f32.
template <int kType, int kN>
struct Raw {
    typedef typename std::conditional<kType == DMADESC_KV_FP32, float, uint16_t>::type T;
    T v[kN];

    __device__ __forceinline__ void load(const void *p, int64_t at)
    {
        __builtin_memcpy(v, __builtin_assume_aligned(static_cast<const T *>(p) + at,
                                                     sizeof(v) < 16 ? sizeof(v) : 16), sizeof(v));
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (kType == DMADESC_KV_FP32) return v[i];
        else if constexpr (kType == DMADESC_KV_BF16) return __uint_as_float((uint32_t)v[i] << 16);
        else return (float)__builtin_bit_cast(_Float16, v[i]);
    }
};

template <int kD, int kType, int kCodes>
__global__ __launch_bounds__(256) void k_kv_append(AppendArgs a)
{
    const KvView &c = a.c;
    const uint64_t unit = (uint64_t)blockIdx.x * 4 + wave();
    const uint32_t head = (uint32_t)(unit % c.kv_heads);
    const uint32_t is_v = (uint32_t)(unit / c.kv_heads) & 1u;
    const uint32_t item = (uint32_t)(unit / c.kv_heads / 2);
    if (item >= a.items) return;
    uint32_t s0, s1;
    int len;
    const uint32_t b = kv_blocks_of(c, a.q_start, a.total, item, s0, s1, len);
    const int64_t nth = (int64_t)item - ((int64_t)(s0 / kBlock) + 2 * (int64_t)b);
    const int count = (int)(s1 - s0), first = len - count;
    if (nth < 0 || count <= 0 || first < 0 || nth > (len - 1) / kBlock) return;
    const int block = first / kBlock + (int)nth;
    if (block > (len - 1) / kBlock) return;
    const int per = (int)c.tshift - 4;
    const uint32_t sub = (uint32_t)block & ((1u << per) - 1u);
    const int old = first - block * kBlock;            // tokens 0..old-1 were there before
    const int end = len - block * kBlock;              // tokens end..15 are zero
    const int64_t tok0 = (int64_t)s0 + (int64_t)block * kBlock - first;   // token of place 0
    const int ln = lane();

    // The page is asked for here and waited for after the values are under way.
    const int32_t page = c.table[(uint64_t)b * c.width + ((uint32_t)block >> per)];
    auto block_of = [&](float *&scale) -> uint8_t * {
        uint8_t *const base = c.pool + (uint64_t)(uint32_t)page * c.page_bytes;
        scale = reinterpret_cast<float *>(base + 2ull * c.code_bytes) + (is_v ? c.scales : 0u) +
                ((head << per) + sub);
        return base + (is_v ? c.code_bytes : 0u) + (uint64_t)((head << per) + sub) * (kBlock * kD);
    };
    float *scale;
    int e_old = kMinExp;
    // Every place loads a new token, its own or the nearest, so that all loads
    // are in flight at once; a conditional load would be waited for where it stands.
    auto clamp = [&](int r) { return r < old ? (old < 0 ? 0 : old) : r < end ? r : end - 1; };

    if (!is_v) {
        constexpr int kLanes = kD / 8;                 // lanes of a row
        constexpr int kRows = kWave / kLanes;          // rows a round
        constexpr int kRounds = kBlock / kRows;
        const int r0 = ln / kLanes, d0 = (ln % kLanes) * 8;
        Raw<kType, 8> raw[kRounds];
        float x[kRounds][8];
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < kRounds; ++i)
            raw[i].load(a.k, (tok0 + clamp(i * kRows + r0)) * a.k_tok + head * a.k_head + d0);
        if (page < 0 || (uint32_t)page >= c.npages) return;
        uint8_t *const codes = block_of(scale);
        if (old > 0) e_old = (int)((__float_as_uint(*scale) >> 23) & 0xffu) - 127;
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int r = i * kRows + r0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[i][j] = r >= old && r < end ? raw[i].get(j) : 0.0f;
                m = fmaxf(m, finite_abs(x[i][j]));
            }
        }
        const int e_new = block_exp<kCodes>(wave_max(m));
        const int e = e_new > e_old ? e_new : e_old;
        const float up = pow2(-e), again = pow2(e_old - e);
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const int r = i * kRows + r0;
            u32x2 *const at = reinterpret_cast<u32x2 *>(codes + r * kD + d0);
            if (r < old) {
                if (e == e_old) continue;              // the earlier codes stand
                const u32x2 w = *at;
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = code_value<kCodes>(w[j / 4], j & 3) * again;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] *= up;
            }
            u32x2 o;
            o[0] = code_quad<kCodes>(x[i][0], x[i][1], x[i][2], x[i][3]);
            o[1] = code_quad<kCodes>(x[i][4], x[i][5], x[i][6], x[i][7]);
            *at = o;
        }
        if (ln == 0) *scale = pow2(e);
    } else {
        constexpr int kDims = kD / kWave;              // dimensions of a lane
        Raw<kType, kDims> raw[kBlock];
        float x[kBlock][kDims];
        float m = 0.0f;
#pragma unroll
        for (int r = 0; r < kBlock; ++r)
            raw[r].load(a.v, (tok0 + clamp(r)) * a.v_tok + head * a.v_head + ln * kDims);
        if (page < 0 || (uint32_t)page >= c.npages) return;
        uint8_t *const codes = block_of(scale);
        u32x4 *const at = reinterpret_cast<u32x4 *>(codes + ln * kDims * kBlock);
        u32x4 held[kDims];                             // earlier tokens' codes
        if (old > 0) {
#pragma unroll
            for (int j = 0; j < kDims; ++j) held[j] = at[j];
            e_old = (int)((__float_as_uint(*scale) >> 23) & 0xffu) - 127;
        } else {
#pragma unroll
            for (int j = 0; j < kDims; ++j) held[j] = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int r = 0; r < kBlock; ++r)
#pragma unroll
            for (int j = 0; j < kDims; ++j) {
                x[r][j] = r >= old && r < end ? raw[r].get(j) : 0.0f;
                m = fmaxf(m, finite_abs(x[r][j]));
            }
        const int e_new = block_exp<kCodes>(wave_max(m));
        const int e = e_new > e_old ? e_new : e_old;
        const float up = pow2(-e), again = pow2(e_old - e);
#pragma unroll
        for (int j = 0; j < kDims; ++j) {
            const u32x4 w = held[j];
            u32x4 o;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[i] = 4 * q + i < old ? code_value<kCodes>(w[q], i) * again
                                           : x[4 * q + i][j] * up;
                o[q] = code_quad<kCodes>(y[0], y[1], y[2], y[3]);
                if (e == e_old) {                      // the earlier codes stand
                    const int n = old - 4 * q;
                    const uint32_t mask = n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
                    o[q] = (o[q] & ~mask) | (w[q] & mask);
                }
            }
            at[j] = o;
        }
        if (ln == 0) *scale = pow2(e);
    }
}

template <int kD, int kType>
void launch_codes(const AppendArgs &a, uint32_t codes, uint32_t grid, hipStream_t s)
{
    if (codes == DMADESC_KV_E4M3)
        k_kv_append<kD, kType, DMADESC_KV_E4M3><<<grid, 256, 0, s>>>(a);
    else
        k_kv_append<kD, kType, DMADESC_KV_INT8><<<grid, 256, 0, s>>>(a);
}

template <int kD>
void launch_type(const AppendArgs &a, uint32_t type, uint32_t codes, uint32_t grid, hipStream_t s)
{
    if (type == DMADESC_KV_BF16) launch_codes<kD, DMADESC_KV_BF16>(a, codes, grid, s);
    else if (type == DMADESC_KV_FP16) launch_codes<kD, DMADESC_KV_FP16>(a, codes, grid, s);
    else launch_codes<kD, DMADESC_KV_FP32>(a, codes, grid, s);
}

}  // namespace

uint64_t kv_append_groups(uint64_t total, uint32_t rows, uint32_t kv_heads)
{
    return ((total / kBlock + 2ull * rows) * 2 * kv_heads + 3) / 4;
}

hipError_t launch_kv_append(const KvAppendArgs &k, hipStream_t s)
{
    AppendArgs a{kv_view(k.cache), k.k, k.v, k.k_tok, k.k_head, k.v_tok, k.v_head, k.q_start,
                 (uint32_t)k.total, (uint32_t)(k.total / kBlock + 2ull * k.cache.rows)};
    const uint32_t grid = (uint32_t)kv_append_groups(k.total, k.cache.rows, k.cache.kv_heads);
    if (k.cache.dim == 64) launch_type<64>(a, k.type, k.cache.codes, grid, s);
    else if (k.cache.dim == 128) launch_type<128>(a, k.type, k.cache.codes, grid, s);
    else launch_type<256>(a, k.type, k.cache.codes, grid, s);
    return hipGetLastError();
}

}  // namespace dd
