// dd_kv.hpp - the paged 8-bit key/value cache as the gfx950 kernels see it:
// page layout, code conversions, request search.
//
// A page holds T tokens of H heads of D values: K codes [H][T][D], V codes
// [H][T/16][D][16] (transposed by blocks of 16 tokens, so that the product
// with the probabilities reads 16 tokens of one dimension in one 16-byte
// load), K scales f32 [H][T/16], V scales [H][T/16], padded to 512 bytes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dd_device.hpp"
#include "dmadesc.h"

namespace dd {

// The cache as kernel argument.
struct KvView {
    uint8_t *pool;
    const int32_t *table;      // [rows][width]
    const int32_t *lens;       // [rows]
    uint64_t page_bytes;
    uint32_t npages, rows, width;
    uint32_t kv_heads;
    uint32_t tshift;           // log2 of the tokens of a page
    uint32_t code_bytes;       // of K (or V) in a page: H * T * D
    uint32_t scales;           // of K (or V) in a page: H * T / 16
};

namespace {

constexpr int kBlock = 16;     // tokens under one scale
constexpr int kMinExp = -64;   // least exponent of a scale

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Tokens of request b that the table can hold.
__device__ __forceinline__ int kv_len(const KvView &c, uint32_t b)
{
    const int64_t cap = (int64_t)c.width << c.tshift;
    const int64_t l = c.lens[b];
    return (int)(l < 0 ? 0 : (l > cap ? cap : l));
}

// New tokens [s0, s1) of request b, inside [0, total) whatever q_start holds.
__device__ __forceinline__ void kv_span(const int32_t *q_start, uint32_t b, uint32_t total,
                                        uint32_t &s0, uint32_t &s1)
{
    const int32_t a = q_start[b], z = q_start[b + 1];
    s0 = a < 0 ? 0u : ((uint32_t)a > total ? total : (uint32_t)a);
    s1 = z < 0 ? 0u : ((uint32_t)z > total ? total : (uint32_t)z);
    s1 = s1 < s0 ? s0 : s1;
}

// Largest request b with first(b) <= i (0 if there is none), for a
// non-decreasing first(): each round, the 64 lanes probe 64 evenly spaced
// requests with one load each, so up to 64 requests take one round and 4,096
// two, where a binary search would wait for 6 and 12 dependent loads. Called
// by a whole wave with wave-uniform i.
template <typename First>
__device__ __forceinline__ uint32_t kv_request_of(uint32_t rows, uint64_t i, First first)
{
    uint32_t lo = 0, n = rows;
    while (n > 1) {
        const uint32_t step = (n + kWave - 1) / kWave;
        const uint64_t at = (uint64_t)lane() * step;
        const bool in = at < n && first(lo + (uint32_t)at) <= i;
        const int k = __popcll(__ballot(in));
        const uint32_t skip = (uint32_t)(k > 0 ? k - 1 : 0) * step;
        lo += skip;
        n = n - skip < step ? n - skip : step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// The request of item i, where request b's items start at number
// q_start[b] / 16 + 2 b, with its span and length. As kv_request_of, but the
// last probe loads the span's end and the length beside its start, so that
// they cost no further round.
__device__ __forceinline__ uint32_t kv_blocks_of(const KvView &c, const int32_t *q_start,
                                                 uint32_t total, uint64_t i, uint32_t &s0,
                                                 uint32_t &s1, int &len)
{
    uint32_t lo = 0, n = c.rows;
    for (;;) {
        const uint32_t step = (n + kWave - 1) / kWave;
        const uint64_t at = (uint64_t)lane() * step;
        const uint32_t r = lo + (at < n ? (uint32_t)at : 0u);
        uint32_t a, z;
        kv_span(q_start, r, total, a, z);
        const int l = step == 1 ? kv_len(c, r) : 0;
        const bool in = at < n && (uint64_t)(a / kBlock) + 2ull * r <= i;
        const int k = __popcll(__ballot(in));
        const uint32_t skip = (uint32_t)(k > 0 ? k - 1 : 0);
        if (step == 1) {
            s0 = (uint32_t)__builtin_amdgcn_readlane((int)a, (int)skip);
            s1 = (uint32_t)__builtin_amdgcn_readlane((int)z, (int)skip);
            len = __builtin_amdgcn_readlane(l, (int)skip);
            return __builtin_amdgcn_readfirstlane(lo + skip);
        }
        lo += skip * step;
        n = n - skip * step < step ? n - skip * step : step;
    }
}

}  // namespace
}  // namespace dd
