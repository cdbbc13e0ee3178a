// kv_keep.hip - bringing the accepted tokens of a drafted tree together in an
// 8-bit cache, for gfx950.
//
// Mathematics: token base + path[k] goes to base + k. From the first token that
// moves on, blocks are written as kv_append would write the tokens' cached values
// (f32 products of code and scale, exact): the least scale 2^e under which they
// fit the largest code, but no smaller one than earlier tokens of the block have,
// and codes rounded once. Places past the last kept token keep their codes.
//
// Work split: one wave to all blocks of one head of K or of V of a request,
// in ascending order. path[k] >= k, so that a block's tokens come from itself or
// from behind it, and nothing that a later block needs has been written over.
// Every wave checks the request for itself, so that all of them write or none.
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
    uint32_t total;
    int32_t *keep;
    uint8_t *status;
};

template <int kD, int kCodes>
__global__ __launch_bounds__(kThreads) void k_kv_keep(KeepArgs a)
{
    const KvView &c = a.c;
    const uint64_t unit = (uint64_t)blockIdx.x * (kThreads / kWave) + wave();
    const uint32_t head = (uint32_t)(unit % c.kv_heads);
    const uint32_t is_v = (uint32_t)(unit / c.kv_heads) & 1u;
    const uint64_t req = unit / c.kv_heads / 2;
    if (req >= c.rows) return;
    const uint32_t b = __builtin_amdgcn_readfirstlane((uint32_t)req);
    const int ln = lane();
    const int64_t s0 = a.q_start[b], s1 = a.q_start[b + 1], len = c.lens[b], n = s1 - s0, base = len - n;
    const int64_t kept = a.count[b];
    const int32_t *const tab = c.table + (uint64_t)b * c.width;
    const int per = (int)c.tshift - 4;
    bool inval = len < 0 || len > ((int64_t)c.width << c.tshift) || s0 < 0 || s1 < s0 || s1 > a.total || n > kMost ||
                 base < 0 || kept < 0 || kept > n;
    bool bad = false;
    int k0 = (int)kept;                                 // first token that moves
    if (!inval) {
        int before = -1;                                // path[k - 1] of lane 0
        bool wrong = false;
        for (int k = 0; k < (int)kept; k += kWave) {
            const int p = k + ln < (int)kept ? a.path[s0 + k + ln] : 0x7fffffff;
            int left = __shfl_up(p, 1, kWave);          // by all lanes: an idle one gives nothing
            if (ln == 0) left = before;
            wrong |= k + ln < (int)kept && (p <= left || p >= (int)n);
            const uint64_t move = __ballot(k + ln < (int)kept && p != k + ln);
            if (move && k0 == (int)kept) k0 = k + __ffsll((unsigned long long)move) - 1;
            before = __builtin_amdgcn_readlane(p, kWave - 1);
        }
        inval = __ballot(wrong) != 0;
        // The pages of all new tokens, and of the block that the first of them continues.
        if (!inval && n > 0) {
            const int64_t p0 = base >> c.tshift, p1 = (len - 1) >> c.tshift;
            for (int64_t k = p0 + ln; k <= p1; k += kWave) bad |= (uint32_t)tab[k] >= c.npages;
            bad = __ballot(bad) != 0;
        }
    }
    const bool no = inval || bad;
    if (head == 0 && is_v == 0 && ln == 0) {
        a.status[b] = inval ? DMADESC_KV_EINVAL : bad ? DMADESC_KV_EPAGE : DMADESC_KV_OK;
        a.keep[b] = no ? (int32_t)len : (int32_t)(base + kept);
    }
    if (no || k0 >= (int)kept) return;

    const int64_t first = base + k0, last = base + kept - 1;
    const uint32_t scales = is_v ? c.scales : 0u, codes_at = is_v ? c.code_bytes : 0u;
    auto block_at = [&](int64_t block) {                // page and block of one token
        const uint32_t page = (uint32_t)tab[block >> per];
        return c.pool + (uint64_t)page * c.page_bytes;
    };
    for (int64_t block = first / kBlock; block <= last / kBlock; ++block) {
        const int old = first > block * kBlock ? (int)(first - block * kBlock) : 0;
        const int end = last < block * kBlock + kBlock - 1 ? (int)(last - block * kBlock) + 1 : kBlock;
        uint8_t *const page = block_at(block);
        const uint32_t sub = (head << per) + ((uint32_t)block & ((1u << per) - 1u));
        float *const scale = reinterpret_cast<float *>(page + 2ull * c.code_bytes) + scales + sub;
        uint8_t *const codes = page + codes_at + (uint64_t)sub * (kBlock * kD);
        // Lane r < 16: where place r comes from. Places that get no token take the
        // nearest one's, and are not used.
        const int place = (ln & 15) < old ? old : (ln & 15) < end ? (ln & 15) : end - 1;
        const int64_t src = base + a.path[s0 + (block * kBlock + place - base)];
        const uint8_t *const from = block_at(src / kBlock);
        const uint32_t from_sub = (head << per) + ((uint32_t)(src / kBlock) & ((1u << per) - 1u));
        const float from_scale = reinterpret_cast<const float *>(from + 2ull * c.code_bytes)[scales + from_sub];
        const uint64_t from_at = (uint64_t)(from - c.pool) + codes_at + (uint64_t)from_sub * (kBlock * kD) +
                                 (is_v ? src % kBlock : src % kBlock * kD);
        auto at_of = [&](int r) { return (uint64_t)__shfl((unsigned long long)from_at, r, kWave); };
        auto scale_of = [&](int r) { return __shfl(from_scale, r, kWave); };
        const int e_was = scale_exp(*scale);
        float m = 0.0f;

        if (!is_v) {
            constexpr int kLanes = kD / 8, kRows = kWave / kLanes, kRounds = kBlock / kRows;
            const int r0 = ln / kLanes, d0 = ln % kLanes * 8;
            u32x2 w[kRounds];
            float by[kRounds];
#pragma unroll
            for (int i = 0; i < kRounds; ++i) {
                const int r = i * kRows + r0;
                w[i] = *reinterpret_cast<const u32x2 *>(c.pool + at_of(r) + d0);
                by[i] = scale_of(r);
            }
#pragma unroll
            for (int i = 0; i < kRounds; ++i) {
                const int r = i * kRows + r0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (r >= old && r < end) m = fmaxf(m, finite_abs(code_value<kCodes>(w[i][j / 4], j & 3) * by[i]));
            }
            int e = block_exp<kCodes>(wave_max(m));
            if (old > 0 && e < e_was) e = e_was;
            const float up = pow2(-e), again = pow2(e_was - e);
#pragma unroll
            for (int i = 0; i < kRounds; ++i) {
                const int r = i * kRows + r0;
                u32x2 *const at = reinterpret_cast<u32x2 *>(codes + r * kD + d0);
                if (r >= end || (r < old && e == e_was)) continue;
                float x[8];
                if (r < old) w[i] = *at;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = code_value<kCodes>(w[i][j / 4], j & 3);
                    x[j] = r < old ? v * again : v * by[i] * up;
                }
                u32x2 o;
                o[0] = code_quad<kCodes>(x[0], x[1], x[2], x[3]);
                o[1] = code_quad<kCodes>(x[4], x[5], x[6], x[7]);
                *at = o;
            }
            if (ln == 0) *scale = pow2(e);
        } else {
            constexpr int kDims = kD / kWave;
            uint32_t w[kBlock][kDims];
            u32x4 held[kDims];
            u32x4 *const at = reinterpret_cast<u32x4 *>(codes + ln * kDims * kBlock);
#pragma unroll
            for (int r = 0; r < kBlock; ++r)
#pragma unroll
                for (int j = 0; j < kDims; ++j) w[r][j] = c.pool[at_of(r) + (uint64_t)(ln * kDims + j) * kBlock];
#pragma unroll
            for (int j = 0; j < kDims; ++j) held[j] = at[j];
#pragma unroll
            for (int r = 0; r < kBlock; ++r)
#pragma unroll
                for (int j = 0; j < kDims; ++j)
                    if (r >= old && r < end) m = fmaxf(m, finite_abs(code_value<kCodes>(w[r][j], 0) * scale_of(r)));
            int e = block_exp<kCodes>(wave_max(m));
            if (old > 0 && e < e_was) e = e_was;
            const float up = pow2(-e), again = pow2(e_was - e);
#pragma unroll
            for (int j = 0; j < kDims; ++j) {
                u32x4 o;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 4 * q + i;
                        y[i] = r < old ? code_value<kCodes>(held[j][q], i) * again
                                       : code_value<kCodes>(w[r][j], 0) * scale_of(r) * up;
                    }
                    o[q] = code_quad<kCodes>(y[0], y[1], y[2], y[3]);
                    // Earlier codes stand unless the scale grew, those past the end always.
                    const uint32_t before = e == e_was ? first_bytes(old - 4 * q) : 0u;
                    const uint32_t stay = before | ~first_bytes(end - 4 * q);
                    o[q] = (o[q] & ~stay) | (held[j][q] & stay);
                }
                at[j] = o;
            }
            if (ln == 0) *scale = pow2(e);
        }
    }
}

template <int kD>
void launch_dim(const KeepArgs &a, uint32_t codes, uint32_t grid, hipStream_t s)
{
    if (codes == DMADESC_KV_E4M3) k_kv_keep<kD, DMADESC_KV_E4M3><<<grid, kThreads, 0, s>>>(a);
    else k_kv_keep<kD, DMADESC_KV_INT8><<<grid, kThreads, 0, s>>>(a);
}

}  // namespace

uint64_t kv_keep_groups(uint32_t rows, uint32_t kv_heads)
{
    return (2ull * rows * kv_heads + 3) / 4;
}

hipError_t launch_kv_keep(const KvKeepArgs &k, hipStream_t s)
{
    KeepArgs a{kv_view(k.cache), k.path, k.count, k.q_start, (uint32_t)k.total, k.keep, k.status};
    const uint32_t grid = (uint32_t)kv_keep_groups(k.cache.rows, k.cache.kv_heads);
    if (k.cache.dim == 64) launch_dim<64>(a, k.cache.codes, grid, s);
    else if (k.cache.dim == 128) launch_dim<128>(a, k.cache.codes, grid, s);
    else launch_dim<256>(a, k.cache.codes, grid, s);
    return hipGetLastError();
}

}  // namespace dd
