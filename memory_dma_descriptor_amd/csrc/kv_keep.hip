// kv_keep.hip - bringing the accepted tokens of a drafted tree together in an
// 8-bit cache, for gfx950.
//
// Mathematics: token base + path[k] goes to base + k. From the first token that
// moves on, blocks are written as kv_append would write the tokens' cached values
// (f32 products of code, scale and 2^-kDown, exact): the least scale 2^e under which
// they fit the largest code, but no smaller one than earlier tokens of the block
// have, and codes rounded once. Places past the last kept token keep their codes.
//
// Work split: one workgroup to K or V of one head of a request, a wave to 64
// dimensions of a block of 16 tokens. path[k] >= k, so that a block's tokens come
// from itself or from behind it: a round of blocks is read by all waves before any
// writes, and nothing that a later round needs is written over. Every wave checks
// the request for itself, so that all of them write or none.
// Bound: latency. A wave waits for the request's sizes, then for path and pages
// together, then for codes and scales; the kernel's own code is kept short (one
// for all dimensions), since it is fetched anew in each launch. Six waves a SIMD
// (72 registers): 64 requests of 16 nodes, 8 heads of 128, 7.0 us; 200 requests of up
// to 60 kept tokens, 4 heads of 256, 17.4 us (before values were held smaller: six waves
// 7.5 and 17.7, five 7.7 and 18.8; eight spill: 8.3 and 19.0). Workgroups of eight waves, more blocks a round: 12.2 and 25.6 before that.
#include "dd_internal.h"
#include "dd_kv.hpp"
#include "dd_kv_codes.hpp"

namespace dd {
namespace {

constexpr int kThreads = 256;
constexpr int kMost = (int)DMADESC_TREE_MOST;

struct KeepArgs {
    KvView c;
    const int32_t *path, *count, *q_start;
    uint32_t total, dim;
    int32_t *keep;
    uint8_t *status;
};

// Values are held 2^-kDown times as large: 448 under a scale of 2^127 is past f32's
// range (kv_append gives f32's largest numbers the code 256 under 2^120).
constexpr int kDown = 24;

// The nearest codes of values in the codes' range, or e4m3's NaN.
template <int kCodes>
__device__ __forceinline__ uint32_t near_quad(const float (&y)[4])
{
    if constexpr (kCodes == DMADESC_KV_E4M3) {
        const int low = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], low, true);
    } else {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = (uint32_t)(int)rintf(y[i]);
        return __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u),
                                     __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), 0x05040100u);
    }
}

template <int kCodes>
__global__ __launch_bounds__(kThreads, 6) void k_kv_keep(KeepArgs a)
{
    __shared__ float tops[kThreads / kWave];
    const KvView &c = a.c;
    const uint32_t b = blockIdx.x / (2 * c.kv_heads), unit = blockIdx.x % (2 * c.kv_heads), head = unit / 2;
    const bool is_v = unit & 1;
    const int wv = __builtin_amdgcn_readfirstlane(wave()), ln = lane();
    const int64_t s0 = a.q_start[b], s1 = a.q_start[b + 1], len = c.lens[b], n = s1 - s0, base = len - n;
    const int64_t kept = a.count[b];
    bool inval = len < 0 || len > ((int64_t)c.width << c.tshift) || s0 < 0 || s1 < s0 || s1 > a.total || n > kMost ||
                 base < 0 || kept < 0 || kept > n;
    const int32_t *const tab = c.table + (uint64_t)b * c.width;
    const int per = (int)c.tshift - 4;
    const int64_t p0 = base >> c.tshift;                // page of the first new token
    int32_t pages = 0;                                  // lane k's is page p0 + k: a tree has 33 at most
    int mine = 0;                                       // path[ln]
    bool bad = false;
    int k0 = (int)kept;                                 // first token that moves
    if (!inval && n > 0) {
        const bool on = p0 + ln <= (len - 1) >> c.tshift;
        if (on) pages = tab[p0 + ln];
        mine = ln < (int)kept ? a.path[s0 + ln] : 0x7fffffff;
        bad = __ballot(on && (uint32_t)pages >= c.npages) != 0;
        int before = -1, p = mine;                      // before: path[k - 1] of lane 0
        bool wrong = false;
        for (int k = 0; k < (int)kept; k += kWave) {
            if (k > 0) p = k + ln < (int)kept ? a.path[s0 + k + ln] : 0x7fffffff;
            int left = __shfl_up(p, 1, kWave);          // by all lanes: an idle one gives nothing
            if (ln == 0) left = before;
            wrong |= k + ln < (int)kept && (p <= left || p >= (int)n);
            const uint64_t move = __ballot(k + ln < (int)kept && p != k + ln);
            if (move && k0 == (int)kept) k0 = k + __ffsll((unsigned long long)move) - 1;
            before = __builtin_amdgcn_readlane(p, kWave - 1);
        }
        inval = __ballot(wrong) != 0;
    }
    const bool no = inval || bad;
    if (unit == 0 && threadIdx.x == 0) {
        a.status[b] = inval ? DMADESC_KV_EINVAL : bad ? DMADESC_KV_EPAGE : DMADESC_KV_OK;
        a.keep[b] = no ? (int32_t)len : (int32_t)(base + kept);
    }
    if (no || k0 >= (int)kept) return;

    const int at0 = (int)base, first = at0 + k0, last = at0 + (int)kept - 1;
    const int slices = (int)a.dim / kWave, at_once = kThreads / kWave / slices;
    const int slice = wv % slices * kWave;              // first dimension of the wave
    // Bytes from the pool's start to a block's codes, and its scale; any lane.
    auto block_at = [&](int block, uint64_t &codes, float *&scale) {
        const uint32_t page = (uint32_t)__shfl(pages, (block >> per) - (int)p0, kWave);
        const uint32_t sub = (head << per) + ((uint32_t)block & ((1u << per) - 1u));
        const uint64_t at = (uint64_t)page * c.page_bytes;
        codes = at + ((is_v ? c.code_bytes : 0u) + sub * (kBlock * a.dim));
        scale = reinterpret_cast<float *>(c.pool + at + 2ull * c.code_bytes) + (is_v ? c.scales : 0u) + sub;
    };
    for (int round = first / kBlock; round <= last / kBlock; round += at_once) {
        const int block = round + wv / slices;
        const bool on = block <= last / kBlock;
        const int old = first > block * kBlock ? first - block * kBlock : 0;
        const int end = last < block * kBlock + kBlock - 1 ? last - block * kBlock + 1 : kBlock;
        uint64_t codes_to = 0, from_at = 0;
        float *scale_to = nullptr, *scale_from = nullptr, from_scale = 0.0f, scale_was = 0.0f;
        // Lane r < 16: where place r comes from. A place that gets no token takes the
        // nearest one's codes, times 0.
        if (on) {
            const int r = ln & 15, place = r < old ? old : r < end ? r : end - 1;
            const int k = block * kBlock + place - at0;
            int p = __shfl(mine, k & (kWave - 1), kWave);
            if (kept > kWave) p = a.path[s0 + k];
            block_at(block, codes_to, scale_to);
            block_at((at0 + p) / kBlock, from_at, scale_from);
            from_at += (uint32_t)((at0 + p) % kBlock) * (is_v ? 1u : a.dim);
            from_scale = *scale_from;
            scale_was = *scale_to;
            from_scale *= pow2(-kDown);
            if (r != place) from_scale = 0.0f;
        }
        // K: lane ln has dimensions 8 (ln % 8) .. + 7 of the slice, of places ln / 8 and
        // ln / 8 + 8. V: dimension ln of all places, and the block's own codes.
        uint8_t *const codes = c.pool + codes_to + (is_v ? (slice + ln) * kBlock : slice + ln % 8 * 8);
        uint32_t w[kBlock];
        u32x4 held = {0, 0, 0, 0};
        u32x2 row[2] = {};
        float by[kBlock], m = 0.0f;
        if (on && is_v) {
#pragma unroll
            for (int r = 0; r < kBlock; ++r) {
                const uint64_t at = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(from_at >> 32), r) << 32 |
                                    (uint32_t)__builtin_amdgcn_readlane((int)from_at, r);
                w[r] = (c.pool + at)[(slice + ln) * kBlock];
            }
            held = *reinterpret_cast<const u32x4 *>(codes);
#pragma unroll
            for (int r = 0; r < kBlock; ++r) {
                by[r] = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(from_scale), r));
                m = fmaxf(m, fabsf(code_value<kCodes>(w[r], 0) * by[r]));
            }
        } else if (on) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = i * 8 + ln / 8;
                row[i] = *reinterpret_cast<const u32x2 *>(
                    c.pool + (uint64_t)__shfl((unsigned long long)from_at, r, kWave) + slice + ln % 8 * 8);
                by[i] = __shfl(from_scale, r, kWave);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(code_value<kCodes>(row[i][j / 4], j & 3) * by[i]));
        }
        m = wave_max(m);
        if (ln == 0) tops[wv] = m;
        __builtin_amdgcn_s_waitcnt(0x0f70);             // vmcnt(0): all that the wave reads has arrived
        __syncthreads();
        for (int i = 0; i < slices; ++i) m = fmaxf(m, tops[wv / slices * slices + i]);
        __syncthreads();                                // before the next round's tops
        if (!on) continue;
        const int e_was = scale_exp(scale_was);
        int e = block_exp<kCodes>(m, kDown);
        e = e < 127 ? e : 127;                          // (-128 under 2^127 stays that code)
        if (old > 0 && e < e_was) e = e_was;
        const float up = pow2(kDown - e), again = pow2(e_was - e);
        if (is_v) {
            u32x4 o;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = code_value<kCodes>(w[4 * q + i], 0) * by[4 * q + i] * up;
                const uint32_t fresh = near_quad<kCodes>(y);
                // Earlier codes stand unless the scale grew, those past the end always.
                const uint32_t stay = first_bytes(old - 4 * q) | ~first_bytes(end - 4 * q);
                o[q] = (fresh & ~stay) | (held[q] & stay);
            }
            if (old > 0 && e != e_was) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = code_value<kCodes>(held[q], i) * again;
                    const uint32_t early = first_bytes(old - 4 * q);
                    o[q] = (near_quad<kCodes>(y) & early) | (o[q] & ~early);
                }
            }
            *reinterpret_cast<u32x4 *>(codes) = o;
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = i * 8 + ln / 8;
                u32x2 *const at = reinterpret_cast<u32x2 *>(codes + (uint32_t)r * a.dim);
                if (r >= end || (r < old && e == e_was)) continue;
                if (r < old) row[i] = *at;
                const float f = r < old ? again : up, g = r < old ? 1.0f : by[i];
                u32x2 o;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = code_value<kCodes>(row[i][q], j) * g * f;
                    o[q] = near_quad<kCodes>(y);
                }
                *at = o;
            }
        }
        if (slice == 0 && ln == 0) *scale_to = pow2(e);
    }
}

}  // namespace

uint64_t kv_keep_groups(uint32_t rows, uint32_t kv_heads)
{
    return 2ull * rows * kv_heads;
}

hipError_t launch_kv_keep(const KvKeepArgs &k, hipStream_t s)
{
    KeepArgs a{kv_view(k.cache), k.path, k.count, k.q_start, (uint32_t)k.total, k.cache.dim, k.keep, k.status};
    const uint32_t grid = (uint32_t)kv_keep_groups(k.cache.rows, k.cache.kv_heads);
    if (k.cache.codes == DMADESC_KV_E4M3) k_kv_keep<DMADESC_KV_E4M3><<<grid, kThreads, 0, s>>>(a);
    else k_kv_keep<DMADESC_KV_INT8><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace dd
