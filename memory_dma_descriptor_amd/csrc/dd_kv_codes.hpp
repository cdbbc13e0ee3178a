// dd_kv_codes.hpp - the cache's codes and scales: conversions that the kernels
// writing blocks share.
#pragma once

#include "dd_kv.hpp"

namespace dd {
namespace {

// |x|, or 0 where x takes no part in the maximum (infinite or NaN).
__device__ __forceinline__ float finite_abs(float x)
{
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.0f;
}

// 2^e for e in -126..127.
__device__ __forceinline__ float pow2(int e)
{
    e = e < -126 ? -126 : e;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Least e >= kMinExp with amax 2^down <= c 2^e (c = 448 = 1.75 * 2^8,
// 127 = 1.984375 * 2^6), from the bits of amax: no logarithm that could be off by one at
// a border.
template <int kCodes>
__device__ __forceinline__ int block_exp(float amax, int down = 0)
{
    const uint32_t bits = __float_as_uint(amax);
    const int e = (int)(bits >> 23) - 127;          // amax = 1.f * 2^e
    const uint32_t frac = bits & 0x7fffffu;
    const int r = down + (kCodes == DMADESC_KV_E4M3 ? e - 8 + (frac > 0x600000u)
                                                    : e - 6 + (frac > 0x7e0000u));
    return r < kMinExp ? kMinExp : r;
}

// The nearest code of y = x 2^-e, in bits 7:0. Values past the largest code
// (only infinities) saturate; NaN is the NaN code of e4m3 and 0 in int8.
template <int kCodes>
__device__ __forceinline__ uint32_t code_pair(float y0, float y1)
{
    constexpr float top = kCodes == DMADESC_KV_E4M3 ? 448.0f : 127.0f;
    const float c0 = y0 != y0 ? y0 : fminf(fmaxf(y0, -top), top);
    const float c1 = y1 != y1 ? y1 : fminf(fmaxf(y1, -top), top);
    if constexpr (kCodes == DMADESC_KV_E4M3) {
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c0, c1, 0, false) & 0xffffu;
    } else {
        const int i0 = c0 != c0 ? 0 : (int)rintf(c0), i1 = c1 != c1 ? 0 : (int)rintf(c1);
        return ((uint32_t)i0 & 0xffu) | (((uint32_t)i1 & 0xffu) << 8);
    }
}

template <int kCodes>
__device__ __forceinline__ uint32_t code_quad(float a, float b, float c, float d)
{
    return code_pair<kCodes>(a, b) | (code_pair<kCodes>(c, d) << 16);
}

// The value of byte i of w.
template <int kCodes>
__device__ __forceinline__ float code_value(uint32_t w, int i)
{
    const uint32_t b = (w >> (8 * i)) & 0xffu;
    if constexpr (kCodes == DMADESC_KV_E4M3)
        return __builtin_amdgcn_cvt_f32_fp8((int)b, 0);
    else
        return (float)(int8_t)b;
}

__device__ __forceinline__ float wave_max(float v)
{
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, kWave));
    return v;
}

// Exponent of a block's scale (a scale of 0, of a page that was never written,
// stands for codes of 0).
__device__ __forceinline__ int scale_exp(float scale)
{
    const int e = (int)((__float_as_uint(scale) >> 23) & 0xffu) - 127;
    return e < kMinExp ? kMinExp : e;
}

// The first n bytes of a word (none for n <= 0, all for n >= 4).
__device__ __forceinline__ uint32_t first_bytes(int n)
{
    return n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
}

}  // namespace
}  // namespace dd
