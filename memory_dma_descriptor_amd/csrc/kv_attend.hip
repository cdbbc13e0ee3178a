// kv_attend.hip - attention of new tokens over a paged 8-bit key/value cache,
// for gfx950.
//
// Mathematics. For a query row q and the cached tokens t it sees,
//   s_t = scale q.K_t,  o = sum_t 2^(s_t log2 e - m) V_t / l,  l = sum_t 2^(..)
// in one pass over the cache with a running maximum m and sum l (both f32).
// K and V are codes times 2^e per block of 16 tokens: the code products run on
// the matrix cores in the 16-bit type that holds every code exactly, the
// powers of two are applied to the f32 scores and to the probabilities. What
// the product with V gets is p_t 2^(e_t) relative to the row's running
// maximum M of (s_t + e_t), times 2^15, in f16: at most 2^15, with 11 bits
// down to 2^-29 of the largest term, so many small terms keep their weight
// and a block with a small scale keeps its precision. That rounding (2^-12 of
// each term) is the only one below f32 before the output's.
//
// Layout. Scores are computed transposed, S^T = K Q^T: the 16x16x32 product
// puts query rows on the lanes (lane % 16) and four tokens in each lane's
// registers. The K row of MFMA row 4 g + i of product j is token 4 j + i of
// block g of the 64-token tile, so lane group g = lane / 16 ends up with all
// 16 scores of block g: one K scale, one V scale and one page per lane, and
// its probabilities are, as they lie, the right operand of O^T = V^T P^T whose
// left operand is the page's own V layout (16 tokens of a dimension in 16
// bytes). Codes go from HBM to registers to the matrix cores; nothing of the
// cache passes through LDS or is shuffled.
#include "dd_internal.h"
#include "dd_kv.hpp"

namespace dd {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTile = 64;                   // tokens a wave handles at a time
constexpr uint32_t kTarget = 1024;          // workgroups that a call is split into
constexpr uint32_t kMinTiles = 16;          // least tiles of a split
constexpr uint32_t kMaxSplits = 256;
constexpr float kShift = 15.0f;             // probabilities are at most 2^15 in f16

struct AttendArgs {
    KvView c;
    const void *q;
    int64_t q_tok, q_head;
    const int32_t *q_start;
    uint32_t total, heads, group;
    int causal;
    float scale;                            // times log2 e
    void *out;
    float *lse;
    float *part;                            // [slots][rows of a tile][dim] partial outputs
    float *part_lse;                        // [slots][rows of a tile], base 2
    uint2 *plan;                            // [rows] first slot and splits of each request
    uint32_t slots;
};

// One piece of work: `count` tiles of the cache from `first`, for one row
// tile of one key head of request b.
struct Item {
    uint32_t b, split, splits, head, rt, base, first, count;
};

template <int kQ> struct QFrag;
template <> struct QFrag<DMADESC_KV_BF16> { typedef bf16x8 type; };
template <> struct QFrag<DMADESC_KV_FP16> { typedef f16x8 type; };

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Four codes as 16-bit floats, exactly.
template <int kCodes>
__device__ __forceinline__ void codes4(uint32_t w, f16x2 &a, f16x2 &b)
{
    if constexpr (kCodes == DMADESC_KV_E4M3) {
        a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
    } else {
        // The bytes, biased to 0..255, below the exponent of 1024.
        const uint32_t u = w ^ 0x80808080u;
        const f16x2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
        a = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) - bias;
        b = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) - bias;
    }
}

template <int kCodes>
__device__ __forceinline__ void codes4(uint32_t w, bf16x2 &a, bf16x2 &b)
{
    if constexpr (kCodes == DMADESC_KV_E4M3) {
        a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true);
    } else {
        const f32x2 x = {(float)(int8_t)w, (float)(int8_t)(w >> 8)};
        const f32x2 y = {(float)(int8_t)(w >> 16), (float)(int8_t)(w >> 24)};
        a = __builtin_convertvector(x, bf16x2);
        b = __builtin_convertvector(y, bf16x2);
    }
}

template <int kCodes, typename V8>
__device__ __forceinline__ V8 codes8(uint32_t lo, uint32_t hi)
{
    typedef decltype(__builtin_shufflevector(V8{}, V8{}, 0, 1)) V2;
    V2 a, b, c, d;
    codes4<kCodes>(lo, a, b);
    codes4<kCodes>(hi, c, d);
    return V8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Row tiles and cache tiles of request b.
template <int kRows>
__device__ __forceinline__ void request_size(const AttendArgs &a, uint32_t b, uint32_t &rts,
                                             uint32_t &tiles)
{
    uint32_t s0, s1;
    kv_span(a.q_start, b, a.total, s0, s1);
    rts = (uint32_t)(((uint64_t)(s1 - s0) * a.group + kRows - 1) / kRows);
    tiles = ((uint32_t)kv_len(a.c, b) + kTile - 1) / kTile;
}

__device__ __forceinline__ uint32_t splits_of(uint32_t tiles, uint32_t chunk)
{
    const uint32_t s = (tiles + chunk - 1) / chunk;
    return s < 1 ? 1u : (s > kMaxSplits ? kMaxSplits : s);
}

// The item of workgroup `id`, from the requests' lengths on the device (the
// host knows only bounds): the tiles of all requests are cut into about
// kTarget pieces of equal size. Every workgroup adds the lengths up for
// itself, one round for up to 256 requests, which costs less than a launch
// that would do it once. Returns false for workgroups past the last item.
template <int kRows>
__device__ bool find_item(const AttendArgs &a, uint32_t id, Item &it)
{
    __shared__ uint64_t sums[kWaves];
    __shared__ uint32_t scan[kWaves];
    __shared__ Item found;
    __shared__ uint32_t hit;
    const uint32_t rows = a.c.rows, heads = a.c.kv_heads;
    uint64_t work = 0;
    for (uint32_t b = threadIdx.x; b < rows; b += kThreads) {
        uint32_t rts, tiles;
        request_size<kRows>(a, b, rts, tiles);
        work += (uint64_t)rts * tiles;
    }
    work = wave_sum(work);
    if (lane() == 0) sums[wave()] = work;
    if (threadIdx.x == 0) hit = 0;
    __syncthreads();
    work = 0;
#pragma unroll
    for (int k = 0; k < kWaves; ++k) work += sums[k];
    const uint64_t even = (work * heads + kTarget - 1) / kTarget;
    const uint32_t chunk = even < kMinTiles ? kMinTiles : (uint32_t)even;

    uint64_t run = 0;
    for (uint32_t b0 = 0; b0 < rows; b0 += kThreads) {
        const uint32_t b = b0 + threadIdx.x;
        uint32_t rts = 0, tiles = 0, splits = 0;
        if (b < rows) {
            request_size<kRows>(a, b, rts, tiles);
            splits = splits_of(tiles, chunk);
        }
        const uint32_t mine = rts * splits * heads;
        uint32_t all;
        const uint64_t at = run + block_excl_scan<kThreads, uint32_t>(mine, scan, &all);
        if (id >= at && id < at + mine) {
            const uint32_t k = id - (uint32_t)at;
            const uint32_t per = (tiles + splits - 1) / splits;
            found.b = b;
            found.rt = k % rts;
            found.head = k / rts % heads;
            found.split = k / rts / heads;
            found.splits = splits;
            found.base = (uint32_t)at;
            found.first = found.split * per;
            found.count = found.first >= tiles ? 0u
                          : (tiles - found.first < per ? tiles - found.first : per);
            hit = 1;
        }
        __syncthreads();
        run += all;
        if (hit || run > id) break;
    }
    it = found;
    return hit != 0;
}

template <int kQ>
__device__ __forceinline__ void store4(void *out, uint64_t at, f32x4 v)
{
    if constexpr (kQ == DMADESC_KV_BF16) {
        const bf16x2 a = __builtin_convertvector(f32x2{v[0], v[1]}, bf16x2);
        const bf16x2 b = __builtin_convertvector(f32x2{v[2], v[3]}, bf16x2);
        *reinterpret_cast<u32x2 *>(static_cast<__bf16 *>(out) + at) =
            u32x2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
    } else {
        const f16x2 a = __builtin_convertvector(f32x2{v[0], v[1]}, f16x2);
        const f16x2 b = __builtin_convertvector(f32x2{v[2], v[3]}, f16x2);
        *reinterpret_cast<u32x2 *>(static_cast<_Float16 *>(out) + at) =
            u32x2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
    }
}

// Bytes of w that are e4m3's NaN (0x7f or 0xff), as 0x80 in each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w)
{
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

constexpr float kInf = __builtin_inff();

// 2^x for -inf..; x finite or -inf.
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

template <int kD, int kQ, int kCodes, int kNt>
__global__ __launch_bounds__(kThreads, kD <= 128 ? 2 : 1) void k_kv_attend(AttendArgs a)
{
    constexpr int kRows = 16 * kNt;
    constexpr int kC = kD / 64;             // 64-dimension pieces of a key row
    constexpr int kX = kD / 16;             // 16-dimension pieces of the output
    typedef typename QFrag<kQ>::type Q8;
    __shared__ f32x4 obuf[2][kX][kWave];
    __shared__ float stat[3][kWaves][kRows];

    Item it;
    if (!find_item<kRows>(a, blockIdx.x, it)) return;
    const KvView &c = a.c;
    const int ln = lane(), col = ln & 15, g = ln >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(wave());
    const uint32_t b = __builtin_amdgcn_readfirstlane(it.b);
    const uint32_t head = __builtin_amdgcn_readfirstlane(it.head);
    const uint32_t row0 = __builtin_amdgcn_readfirstlane(it.rt) * kRows;
    uint32_t s0, s1;
    kv_span(a.q_start, b, a.total, s0, s1);
    const int len = kv_len(c, b), news = (int)(s1 - s0);
    const uint32_t nrows = (uint32_t)news * a.group;
    const int per = (int)c.tshift - 4;
    const uint32_t sub_mask = (1u << per) - 1u;

    // The lane's query rows (operand columns) and the last token each sees.
    Q8 qf[kNt][kC][2];
    int limit[kNt];
    uint64_t orow[kNt];
    int low = len - 1, high = -1;           // least and largest limit of the tile's rows
    {
        const uint32_t jl = row0 / a.group;
        const uint32_t last = nrows - 1 < row0 + kRows - 1 ? nrows - 1 : row0 + kRows - 1;
        if (a.causal) {
            low = len - news + (int)jl;
            high = len - news + (int)(last / a.group);
        } else {
            high = len - 1;
        }
        low = low < len - 1 ? low : len - 1;
        high = high < len - 1 ? high : len - 1;
    }
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
        const uint32_t r = row0 + n * 16 + col;
        const bool on = r < nrows;
        const uint32_t rr = on ? r : 0u, j = rr / a.group, h = head * a.group + rr % a.group;
        const int lim = a.causal ? len - news + (int)j : len - 1;
        limit[n] = on ? (lim < len - 1 ? lim : len - 1) : -1;
        orow[n] = ((uint64_t)(s0 + j) * a.heads + h) * kD;
        const uint16_t *const q = static_cast<const uint16_t *>(a.q) +
                                  (int64_t)(s0 + j) * a.q_tok + (int64_t)h * a.q_head + 16 * g;
#pragma unroll
        for (int k = 0; k < kC; ++k)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                u32x4 w = {0, 0, 0, 0};
                if (on) w = *reinterpret_cast<const u32x4 *>(q + 64 * k + 8 * u);
                qf[n][k][u] = __builtin_bit_cast(Q8, w);
            }
    }

    f32x4 acc[kNt][kX];
    float m[kNt], mx[kNt], l[kNt];
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
        m[n] = mx[n] = -kInf;
        l[n] = 0.0f;
#pragma unroll
        for (int x = 0; x < kX; ++x) acc[n][x] = f32x4{0, 0, 0, 0};
    }

    const int t0 = (int)it.first;
    int t1 = (int)(it.first + it.count);
    const int see = high < 0 ? 0 : high / kTile + 1;
    t1 = t1 < see ? t1 : see;
    const int last_block = len > 0 ? (len - 1) / kBlock : 0;
    const int32_t *const tab = c.table + (uint64_t)b * c.width;
    const int kblk = col >> 2;              // block of the lane's key rows
    int32_t pk = 0, pv = 0;                 // pages of the next tile, per lane
    u32x4 kr[4][kC], vr[kX];
    float ks = 0.0f, vs = 0.0f;
    int valid = 0;                          // tokens of block g inside the request

    auto load_pages = [&](int t) {
        const int bk = t * 4 + kblk, bv = t * 4 + g;
        pk = tab[(bk < last_block ? bk : last_block) >> per];
        pv = tab[(bv < last_block ? bv : last_block) >> per];
    };
    auto load_k = [&](int t) {
        const uint32_t sub = (uint32_t)(t * 4 + kblk) & sub_mask;
        const uint32_t page = (uint32_t)pk < c.npages ? (uint32_t)pk : 0u;
        const uint8_t *const p = c.pool + (uint64_t)page * c.page_bytes +
                                 (((uint64_t)((head << per) + sub) * kBlock + (col & 3)) * kD + 16 * g);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < kC; ++k)
                kr[j][k] = *reinterpret_cast<const u32x4 *>(p + 4 * j * kD + 64 * k);
    };
    auto load_v = [&](int t) {
        const int bv = t * 4 + g;
        const uint32_t sub = (uint32_t)bv & sub_mask;
        const bool ok = (uint32_t)pv < c.npages;
        const uint32_t page = ok ? (uint32_t)pv : 0u;
        const uint8_t *const p = c.pool + (uint64_t)page * c.page_bytes;
        const uint8_t *const pvv = p + c.code_bytes + (uint64_t)((head << per) + sub) * (kBlock * kD) +
                                   col * 16;
        const float *const sc = reinterpret_cast<const float *>(p + 2ull * c.code_bytes) +
                                ((head << per) + sub);
        ks = sc[0];
        vs = sc[c.scales];
        const int left = len - bv * kBlock;
        valid = ok ? (left < 0 ? 0 : (left < kBlock ? left : kBlock)) : 0;
#pragma unroll
        for (int x = 0; x < kX; ++x) vr[x] = *reinterpret_cast<const u32x4 *>(pvv + 256 * x);
    };

    int t = t0 + wv;
    if (t < t1) {
        load_pages(t);
        load_k(t);
        load_v(t);
        load_pages(t + kWaves);
    }
    for (; t < t1; t += kWaves) {
        const bool more = t + kWaves < t1;
        f32x4 s[kNt][4];
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[n][j] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < kC; ++k)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const Q8 kf = codes8<kCodes, Q8>(kr[j][k][2 * u], kr[j][k][2 * u + 1]);
#pragma unroll
                    for (int n = 0; n < kNt; ++n) s[n][j] = mfma(kf, qf[n][k][u], s[n][j]);
                }
        const float kscale = ks * a.scale, vscale = vs;
        const int nvalid = valid;
        if (more) load_k(t + kWaves);

        const int tok = t * kTile + g * kBlock;       // first token of the lane's block
        const bool edge = t * kTile + kTile - 1 > low;   // some row does not see the whole tile
        const float ve = (float)((int)(__float_as_uint(vscale) >> 23 & 0xffu) - 126);
        f16x8 pf[kNt][2];
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
            const int lim = nvalid == 0 ? -1 : limit[n];
            float top = -kInf;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float v = s[n][j][i] * kscale;
                    s[n][j][i] = tok + 4 * j + i <= lim ? v : -kInf;
                    top = fmaxf(top, s[n][j][i]);
                }
            float topv = top == -kInf ? -kInf : top + ve;
            top = fmaxf(top, __shfl_xor(top, 16, kWave));
            topv = fmaxf(topv, __shfl_xor(topv, 16, kWave));
            top = fmaxf(top, __shfl_xor(top, 32, kWave));
            topv = fmaxf(topv, __shfl_xor(topv, 32, kWave));
            const float mn = fmaxf(m[n], top), mxn = fmaxf(mx[n], topv);
            const float ms = mn == -kInf ? 0.0f : mn, mxs = mxn == -kInf ? 0.0f : mxn;
            const float f = nvalid == 0 ? 0.0f : vscale * exp2_(ms - mxs + kShift);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = exp2_(s[n][j][i] - ms);
                    sum += p;
                    pf[n][j >> 1][(j & 1) * 4 + i] = (_Float16)(p * f);
                }
            l[n] = l[n] * exp2_(m[n] - ms) + sum;
            const float back = exp2_(mx[n] - mxs);
            m[n] = mn;
            mx[n] = mxn;
#pragma unroll
            for (int x = 0; x < kX; ++x) acc[n][x] *= back;
        }

        if constexpr (kCodes == DMADESC_KV_E4M3) {
            // A NaN code that a row does not see must not reach it (0 * NaN):
            // codes past the length are cleared; other NaN codes are found by
            // a product of indicators and then cleared.
            if (edge) {
                uint32_t found = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int keep = nvalid - 4 * q;
                    const uint32_t mask = keep >= 4 ? 0xffffffffu : keep <= 0 ? 0u : (1u << (8 * keep)) - 1u;
#pragma unroll
                    for (int x = 0; x < kX; ++x) {
                        vr[x][q] &= mask;
                        found |= nan_bytes(vr[x][q]);
                    }
                }
                if (__ballot(found != 0)) {
#pragma unroll
                    for (int x = 0; x < kX; ++x)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            f16x8 is_nan;
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                is_nan[i] = (_Float16)(float)(nan_bytes(vr[x][2 * u + i / 4]) >>
                                                              (8 * (i & 3) + 7) & 1u);
#pragma unroll
                            for (int n = 0; n < kNt; ++n) {
                                f16x8 seen;
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    seen[i] = (_Float16)(tok + 8 * u + i <= limit[n] ? 1.0f : 0.0f);
                                const f32x4 cnt = mfma(is_nan, seen, f32x4{0, 0, 0, 0});
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (cnt[i] > 0.0f) acc[n][x][i] = __builtin_nanf("");
                            }
                        }
#pragma unroll
                    for (int x = 0; x < kX; ++x)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t z = nan_bytes(vr[x][q]);
                            vr[x][q] &= ~(z | (z - (z >> 7)));
                        }
                }
            }
        }
#pragma unroll
        for (int x = 0; x < kX; ++x)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const f16x8 vf = codes8<kCodes, f16x8>(vr[x][2 * u], vr[x][2 * u + 1]);
#pragma unroll
                for (int n = 0; n < kNt; ++n) acc[n][x] = mfma(vf, pf[n][u], acc[n][x]);
            }
        if (more) {
            load_v(t + kWaves);
            load_pages(t + 2 * kWaves);
        }
    }

    // Join the waves: common maxima first, then the sums, two waves at a time.
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
        l[n] += __shfl_xor(l[n], 16, kWave);
        l[n] += __shfl_xor(l[n], 32, kWave);
        if (g == 0) {
            stat[0][wv][n * 16 + col] = m[n];
            stat[1][wv][n * 16 + col] = mx[n];
            stat[2][wv][n * 16 + col] = l[n];
        }
    }
    __syncthreads();
    const bool whole = it.splits == 1;
    const uint32_t slot = blockIdx.x;       // the item's number is its partial result's
    if (slot == it.base && threadIdx.x == 0) a.plan[b] = make_uint2(it.base, it.splits);
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
        float ma = -kInf, mxa = -kInf, la = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            ma = fmaxf(ma, stat[0][w][n * 16 + col]);
            mxa = fmaxf(mxa, stat[1][w][n * 16 + col]);
        }
        const float ms = ma == -kInf ? 0.0f : ma, mxs = mxa == -kInf ? 0.0f : mxa;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            la += stat[2][w][n * 16 + col] * exp2_(stat[0][w][n * 16 + col] - ms);
        const float mine = exp2_(mx[n] - mxs);
#pragma unroll
        for (int x = 0; x < kX; ++x) acc[n][x] *= mine;
        if (wv >= 2)
#pragma unroll
            for (int x = 0; x < kX; ++x) obuf[wv - 2][x][ln] = acc[n][x];
        __syncthreads();
        if (wv < 2)
#pragma unroll
            for (int x = 0; x < kX; ++x) acc[n][x] += obuf[wv][x][ln];
        __syncthreads();
        if (wv == 1)
#pragma unroll
            for (int x = 0; x < kX; ++x) obuf[0][x][ln] = acc[n][x];
        __syncthreads();
        if (wv == 0) {
            const uint32_t r = row0 + n * 16 + col;
            // A row that sees nothing: zero, and no mass (la = 0).
            const float norm = la == 0.0f ? 0.0f : exp2_(mxs - ms - kShift) / la;
            const float lse2 = la == 0.0f ? -kInf : ms + __builtin_log2f(la);
            if (r < nrows) {
#pragma unroll
                for (int x = 0; x < kX; ++x) {
                    const f32x4 o = (acc[n][x] + obuf[0][x][ln]) * norm;
                    if (whole)
                        store4<kQ>(a.out, orow[n] + 16 * x + 4 * g, o);
                    else
                        *reinterpret_cast<f32x4 *>(
                            a.part + ((uint64_t)slot * kRows + n * 16 + col) * kD + 16 * x + 4 * g) = o;
                }
                if (g == 0) {
                    if (!whole) a.part_lse[(uint64_t)slot * kRows + n * 16 + col] = lse2;
                    else if (a.lse) a.lse[orow[n] / kD] = lse2 * 0.69314718055994531f;
                }
            }
        }
        __syncthreads();
    }
}

// Joins the splits of one output row (token, head): a workgroup's waves take
// every fourth split each.
template <int kD, int kQ>
__global__ __launch_bounds__(kThreads) void k_kv_join(AttendArgs a, uint32_t tile_rows)
{
    constexpr int kE = kD / kWave;          // values of a lane
    __shared__ float part[kWaves][kD];
    __shared__ float mass[kWaves];
    const uint32_t tokn = blockIdx.x / a.heads, h = blockIdx.x % a.heads;
    const uint32_t b = kv_request_of(a.c.rows, tokn, [&](uint32_t r) {
        const int32_t s = a.q_start[r];
        return (uint64_t)(s < 0 ? 0 : s);
    });
    uint32_t s0, s1;
    kv_span(a.q_start, b, a.total, s0, s1);
    if (tokn < s0 || tokn >= s1) return;
    const uint2 plan = a.plan[b];
    if (plan.y <= 1 || plan.y > kMaxSplits) return;
    const uint32_t kvh = h / a.group;
    const uint32_t r = (tokn - s0) * a.group + h % a.group;
    const uint32_t rts = ((s1 - s0) * a.group + tile_rows - 1) / tile_rows;
    const uint32_t first = plan.x + kvh * rts + r / tile_rows, step = a.c.kv_heads * rts;
    if ((uint64_t)first + (uint64_t)(plan.y - 1) * step >= a.slots) return;   // q_start out of order
    const uint64_t in = r % tile_rows;
    float top = -kInf;
    for (uint32_t s = lane(); s < plan.y; s += kWave)
        top = fmaxf(top, a.part_lse[(uint64_t)(first + s * step) * tile_rows + in]);
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
    if (top == -kInf) top = 0.0f;
    float o[kE] = {}, w = 0.0f;
#pragma unroll 4
    for (uint32_t s = wave(); s < plan.y; s += kWaves) {
        const uint64_t at = (uint64_t)(first + s * step) * tile_rows + in;
        const float v = exp2_(a.part_lse[at] - top);
        w += v;
#pragma unroll
        for (int k = 0; k < kE; ++k) o[k] += v * a.part[at * kD + k * kWave + lane()];
    }
#pragma unroll
    for (int k = 0; k < kE; ++k) part[wave()][k * kWave + lane()] = o[k];
    if (lane() == 0) mass[wave()] = w;
    __syncthreads();
    const float all = mass[0] + mass[1] + mass[2] + mass[3];
    for (uint32_t d = threadIdx.x; d < kD; d += kThreads) {
        const float v = part[0][d] + part[1][d] + part[2][d] + part[3][d];
        const float y = all == 0.0f ? 0.0f : v / all;
        const uint64_t at = (uint64_t)blockIdx.x * kD + d;
        if constexpr (kQ == DMADESC_KV_BF16) static_cast<__bf16 *>(a.out)[at] = (__bf16)y;
        else static_cast<_Float16 *>(a.out)[at] = (_Float16)y;
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[blockIdx.x] = all == 0.0f ? -kInf : (top + __builtin_log2f(all)) * 0.69314718055994531f;
}

// Rows of a tile: one product's 16 where a request's rows fit it, else 32.
uint32_t tile_rows_of(uint64_t total, uint32_t rows, uint32_t group)
{
    return (total + rows - 1) / rows * group <= 16 ? 16u : 32u;
}

// Workgroups (= partial results) that a call may need: the even pieces, and
// one more for each row tile of each key head.
uint64_t slots_of(uint64_t total, uint32_t rows, uint32_t heads, uint32_t kv_heads)
{
    const uint32_t group = heads / kv_heads, tr = tile_rows_of(total, rows, group);
    return kTarget + kv_heads * (total * group / tr + rows);
}

template <int kD, int kQ, int kCodes>
void launch_rows(const AttendArgs &a, uint32_t tile_rows, uint32_t grid, hipStream_t s)
{
    if (tile_rows == 16) k_kv_attend<kD, kQ, kCodes, 1><<<grid, kThreads, 0, s>>>(a);
    else k_kv_attend<kD, kQ, kCodes, 2><<<grid, kThreads, 0, s>>>(a);
}

template <int kD, int kQ>
void launch_codes(const AttendArgs &a, uint32_t codes, uint32_t tile_rows, uint32_t grid,
                  bool join, hipStream_t s)
{
    if (codes == DMADESC_KV_E4M3) launch_rows<kD, kQ, DMADESC_KV_E4M3>(a, tile_rows, grid, s);
    else launch_rows<kD, kQ, DMADESC_KV_INT8>(a, tile_rows, grid, s);
    if (join) k_kv_join<kD, kQ><<<a.total * a.heads, kThreads, 0, s>>>(a, tile_rows);
}

template <int kD>
void launch_type(const AttendArgs &a, uint32_t type, uint32_t codes, uint32_t tile_rows,
                 uint32_t grid, bool join, hipStream_t s)
{
    if (type == DMADESC_KV_BF16)
        launch_codes<kD, DMADESC_KV_BF16>(a, codes, tile_rows, grid, join, s);
    else
        launch_codes<kD, DMADESC_KV_FP16>(a, codes, tile_rows, grid, join, s);
}

}  // namespace

size_t ws_kv_attend(uint64_t total, uint32_t rows, uint32_t heads, uint32_t kv_heads,
                    uint32_t dim, uint64_t)
{
    if (total == 0 || rows == 0) return 0;
    const uint64_t slots = slots_of(total, rows, heads, kv_heads);
    const uint32_t tr = tile_rows_of(total, rows, heads / kv_heads);
    return align256(8ull * rows) + align256(4 * slots * tr) + align256(4 * slots * tr * dim);
}

hipError_t launch_kv_attend(const KvAttendArgs &k, hipStream_t s)
{
    AttendArgs a{};
    a.c = kv_view(k.cache);
    if (a.c.npages == 0) a.c.width = 0;                 // no page: every length is 0
    a.q = k.q;
    a.q_tok = k.q_tok;
    a.q_head = k.q_head;
    a.q_start = k.q_start;
    a.total = (uint32_t)k.total;
    a.heads = k.heads;
    a.group = k.heads / k.cache.kv_heads;
    a.causal = k.causal;
    const float scale = k.scale != 0.0f ? k.scale : 1.0f / sqrtf((float)k.cache.dim);
    a.scale = scale * 1.44269504088896341f;
    a.out = k.out;
    a.lse = k.lse;
    const uint32_t tr = tile_rows_of(k.total, k.cache.rows, a.group);
    a.slots = (uint32_t)slots_of(k.total, k.cache.rows, k.heads, k.cache.kv_heads);
    uint8_t *p = static_cast<uint8_t *>(k.ws);
    a.plan = reinterpret_cast<uint2 *>(p);
    p += align256(8ull * k.cache.rows);
    a.part_lse = reinterpret_cast<float *>(p);
    p += align256(4ull * a.slots * tr);
    a.part = reinterpret_cast<float *>(p);
    const bool join = ((uint64_t)a.c.width << a.c.tshift) > (uint64_t)kMinTiles * kTile;
    if (k.cache.dim == 64) launch_type<64>(a, k.type, k.cache.codes, tr, a.slots, join, s);
    else if (k.cache.dim == 128) launch_type<128>(a, k.type, k.cache.codes, tr, a.slots, join, s);
    else launch_type<256>(a, k.type, k.cache.codes, tr, a.slots, join, s);
    return hipGetLastError();
}

}  // namespace dd
