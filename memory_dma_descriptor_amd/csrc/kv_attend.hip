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
// maximum M of (s_t + e_t), in f16, where the largest stands at 2^14 (few rows)
// or 2^13 to 2^15 (many): 11 bits down to 2^-27 of the largest term, fewer to
// 2^-37, so many small terms keep their weight and a block with a small scale
// keeps its precision. That rounding (2^-11 of each term at most) is the only
// one below f32 before the output's. In two bf16 parts, which would keep more,
// the second product would run twice.
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
// Waves a SIMD of the kernel of few rows, by the registers of its accumulators,
// and workgroups of each kernel that fit the 256 compute units at once.
constexpr int few_occupancy(int dim, int nt)
{
    return dim * nt <= 64 ? 3 : dim * nt <= 128 ? 2 : 1;
}
constexpr uint32_t slots_few(int dim, int nt) { return 256u * few_occupancy(dim, nt); }
constexpr uint32_t slots_many(int dim) { return dim == 64 ? 768 : dim == 128 ? 512 : 256; }
constexpr uint32_t kLongFew = 32, kLongMany = ~0u;      // tiles of a piece past which two rounds run
constexpr uint32_t kWholeFew = 20, kWholeMany = 4;      // tiles up to which nothing is split
constexpr uint32_t kMaxSplits = 256;
constexpr uint32_t kRowsMany = 128;         // query rows of a workgroup of the kernel of many
constexpr uint32_t kMostFew = 64;           // rows up to which a request is the first's, if both run
constexpr float kShift = 15.0f;             // probabilities are at most 2^14 in f16, see ve
// Log of the largest factor of an exponential: what f32 loses of one below 2^-126
// is then below f16's least step.
constexpr float kFar = 100.0f;

struct AttendArgs {
    KvView c;
    const void *q;
    int64_t q_tok, q_head;
    const int32_t *q_start;
    uint32_t total, heads, group;
    int causal;
    float scale;                            // times log2 e
    float most_scale;                       // of K under which the product with scale is finite
    void *out;
    float *lse;
    float *part;                            // [slots][rows of a tile][dim] partial outputs
    float *part_lse;                        // [slots][rows of a tile], base 2
    uint2 *plan;                            // [rows] first slot and splits of each request
    uint32_t slots;
    uint32_t least, most;                   // requests of least..most query rows are this kernel's
};

// One piece of work: the split-th of `splits` even parts of the cache that one
// row tile of one key head of request b sees. The request's new tokens are
// s0 .. s0 + news - 1, its length is len.
struct Item {
    uint32_t b, split, splits, head, rt, base, s0;
    int news, len;
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

// Most pieces of `base` unsplit ones when `aim` are aimed at.
__host__ __device__ constexpr uint32_t most_pieces(uint32_t base, uint32_t aim)
{
    return base < aim ? aim + aim / 8 : base + aim / 2;
}

// What a call's requests are cut into: about as many pieces as workgroups fit
// the card at once (kSlots), so that they run in one round of equal pieces, or
// in two where they are longer than kLong tiles (32 for few rows: 64 requests of
// 200 to 9,000 tokens take 130 us in two rounds and 155 in one, 4 of 100,000 and
// more 159 either way), but no piece below kLeast tiles, and nothing where no
// request has more than kWhole, which saves the join (a request alone, 32 heads
// on 8, split / whole: 2,040 tokens 13 / 22 us, 1,500 tokens 12 / 14 us, 900
// tokens, by its launch, 16 / 12 us). The host knows only bounds, so every
// workgroup adds the lengths up for itself and finds its own piece, which costs
// less than a launch that would do it once: up to 64 requests are one load and a
// few lane exchanges of each wave.
template <int kRows, int kThreads, uint32_t kSlots, uint32_t kLeast, uint32_t kWhole, uint32_t kLong>
struct Plan {
    static constexpr int kWaves = kThreads / kWave;

    struct Size {
        uint32_t rts, tiles, s0;      // row tiles (0: not this kernel's request), cache tiles
        int news, len;
    };

    static __device__ __forceinline__ Size size(const AttendArgs &a, uint32_t b)
    {
        Size z{};
        if (b >= a.c.rows) return z;
        uint32_t s1;
        kv_span(a.q_start, b, a.total, z.s0, s1);
        z.news = (int)(s1 - z.s0);
        z.len = kv_len(a.c, b);
        const uint32_t n = (uint32_t)z.news * a.group;      // total * heads < 2^31
        z.rts = n < a.least || n > a.most ? 0u : (n + kRows - 1) / kRows;
        z.tiles = ((uint32_t)z.len + kTile - 1) / kTile;
        return z;
    }

    static __device__ __forceinline__ uint32_t splits(const Size &z, uint32_t chunk)
    {
        const uint32_t s = (z.tiles + chunk - 1) / chunk;
        return s < 1 ? 1u : (s > kMaxSplits ? kMaxSplits : s);
    }

    // Tiles of a piece for `work` tiles in `base` unsplit pieces (a request's last
    // piece is half full on the average), and how many pieces are aimed at.
    static __device__ __forceinline__ uint32_t first_chunk(float work, float base, bool whole, uint32_t &aim)
    {
        aim = kSlots;
        if (whole) return kWhole;
        float c = ceilf(work / fmaxf((float)kSlots - 0.5f * base, 0.25f * kSlots));
        if (c > (float)kLong) {
            aim = 2 * kSlots;
            c = ceilf(work / fmaxf(2.0f * kSlots - 0.5f * base, 0.5f * kSlots));
        }
        return c < (float)kLeast ? kLeast : (uint32_t)c;
    }

    // Round `round` of looking for a piece length: a little longer each time until
    // the pieces are no more than aimed at. Where that does not come out (requests
    // of one length double their pieces at once), an eighth more will do, and where
    // that does not either, nothing is split. The host sizes the grid by most_pieces.
    static constexpr int kStrict = 4, kRounds = 12;
    static __device__ __forceinline__ bool fits(uint32_t pieces, float base, uint32_t aim, int round)
    {
        return pieces <= (round <= kStrict && base < (float)aim ? aim : most_pieces((uint32_t)base, aim));
    }
    static __device__ __forceinline__ uint32_t larger(uint32_t chunk, uint32_t first, int round)
    {
        return round == kStrict ? first : round < kRounds ? chunk + chunk / 16 + 1 : 1u << 30;
    }

    static __device__ __forceinline__ Item item(const Size &z, uint32_t b, uint32_t at, uint32_t k,
                                                uint32_t parts, uint32_t heads)
    {
        // Heads first: workgroups go round the 8 XCDs, so a head's meet in few caches.
        return Item{b, k / heads / z.rts, parts, k % heads, k / heads % z.rts, at, z.s0, z.news, z.len};
    }

    // The piece of workgroup `id`; false past the last. Every wave of the
    // workgroup calls it (with more than 64 requests it has barriers).
    static __device__ bool find(const AttendArgs &a, uint32_t id, Item &it)
    {
        const uint32_t rows = a.c.rows, heads = a.c.kv_heads;
        if (rows <= (uint32_t)kWave) {
            const Size z = size(a, (uint32_t)lane());
            const float work = wave_sum((float)z.rts * (float)z.tiles) * (float)heads;
            const float base = wave_sum((float)z.rts) * (float)heads;
            uint32_t aim;
            uint32_t chunk = first_chunk(work, base, __ballot(z.rts > 0 && z.tiles > kWhole) == 0, aim);
            const uint32_t first = chunk;
            uint32_t mine = z.rts * splits(z, chunk) * heads, upto = wave_incl_scan(mine);
            for (int k = 0; k <= kRounds && !fits(__builtin_amdgcn_readlane(upto, kWave - 1), base, aim, k); ++k) {
                chunk = larger(chunk, first, k);
                mine = z.rts * splits(z, chunk) * heads;
                upto = wave_incl_scan(mine);
            }
            const uint64_t hit = __ballot(id < upto && id >= upto - mine);
            if (hit == 0) return false;
            const int b = __ffsll((unsigned long long)hit) - 1;
            const auto get = [b](uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, b); };
            const Size w{get(z.rts), get(z.tiles), get(z.s0), (int)get((uint32_t)z.news),
                         (int)get((uint32_t)z.len)};
            const uint32_t at = get(upto - mine);
            it = item(w, (uint32_t)b, at, id - at, splits(w, chunk), heads);
            return true;
        }
        __shared__ float fsum[2][kWaves];
        __shared__ uint32_t scan[kWaves];
        __shared__ Item found;
        __shared__ uint32_t hit, large;
        if (threadIdx.x == 0) hit = large = 0;
        __syncthreads();
        float work = 0.0f, base = 0.0f;
        for (uint32_t b = threadIdx.x; b < rows; b += kThreads) {
            const Size z = size(a, b);
            work += (float)z.rts * (float)z.tiles;
            base += (float)z.rts;
            if (z.rts > 0 && z.tiles > kWhole) large = 1;         // every writer writes 1
        }
        work = wave_sum(work);
        base = wave_sum(base);
        if (lane() == 0) {
            fsum[0][wave()] = work;
            fsum[1][wave()] = base;
        }
        __syncthreads();
        work = base = 0.0f;
#pragma unroll
        for (int k = 0; k < kWaves; ++k) {
            work += fsum[0][k];
            base += fsum[1][k];
        }
        work *= (float)heads;
        base *= (float)heads;
        uint32_t aim;
        uint32_t chunk = first_chunk(work, base, large == 0, aim);
        const uint32_t first = chunk;
        for (int k = 0; k <= kRounds; ++k) {
            uint32_t n = 0;
            for (uint32_t b = threadIdx.x; b < rows; b += kThreads) {
                const Size z = size(a, b);
                n += z.rts * splits(z, chunk) * heads;
            }
            n = wave_sum(n);
            __syncthreads();
            if (lane() == 0) scan[wave()] = n;
            __syncthreads();
            n = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) n += scan[w];
            if (fits(n, base, aim, k)) break;
            chunk = larger(chunk, first, k);
        }
        uint64_t run = 0;
        for (uint32_t b0 = 0; b0 < rows; b0 += kThreads) {
            const uint32_t b = b0 + threadIdx.x;
            const Size z = size(a, b);
            const uint32_t parts = splits(z, chunk), mine = z.rts * parts * heads;
            uint32_t all;
            __syncthreads();
            const uint64_t at = run + block_excl_scan<kThreads, uint32_t>(mine, scan, &all);
            if (id >= at && id < at + mine) {
                found = item(z, b, (uint32_t)at, id - (uint32_t)at, parts, heads);
                hit = 1;
            }
            __syncthreads();
            run += all;
            if (hit || run > id) break;
        }
        it = found;
        return hit != 0;
    }
};

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

// w without the bytes that nan_bytes found.
__device__ __forceinline__ uint32_t without(uint32_t w, uint32_t nans)
{
    return w & ~(nans | (nans - (nans >> 7)));
}

// The first `keep` bytes of word q of a run of 16.
__device__ __forceinline__ uint32_t keep_mask(int keep, int q)
{
    const int n = keep - 4 * q;
    return n >= 4 ? ~0u : n <= 0 ? 0u : (1u << (8 * n)) - 1u;
}

// A NaN code of V must reach the rows that see its token and no other, but in
// a product 0 * NaN is NaN. In the tiles that some row sees only in part it is
// therefore replaced by 0 and its token noted per dimension, the first one:
// rows see the tokens up to their limit, so a row whose limit reaches that
// token has NaN in that dimension in the end.
constexpr int kNoNan = 0x7fffffff;
__device__ __forceinline__ void note_nan(int *first_nan, uint32_t nans, int dim, int tok)
{
    if (nans) atomicMin(&first_nan[dim], tok + (__builtin_ctz(nans) >> 3));
}

constexpr float kInf = __builtin_inff();

// 2^x for -inf..; x finite or -inf.
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// Attention for single tokens and drafts, where reading the cache is the bound:
// 16 or 32 query rows of one key head a workgroup, its four waves taking every
// fourth tile of a piece of the cache, 16 KB (D = 128) each in flight while the
// tile before is multiplied. Two waves a SIMD keep 128 KB of a compute unit's reads
// outstanding. 64 requests of 200 to 9,000 tokens, 32 heads on 8, D = 128, e4m3:
// 130 us, 730 MB read and written, 5.6 TB/s (a large copy: 4.9); 4 of 100,000 to
// 131,072 tokens: 159 us, 6.2 TB/s. One tile alone takes 6 us, most of it the launch and
// fetching 14 KB of code for the first time; each further one of a wave 1.3 us.
template <int kD, int kQ, int kCodes, int kNt>
__global__ __launch_bounds__(kThreads, few_occupancy(kD, kNt)) void k_kv_attend(AttendArgs a)
{
    constexpr int kRows = 16 * kNt;
    constexpr int kC = kD / 64;             // 64-dimension pieces of a key row
    constexpr int kX = kD / 16;             // 16-dimension pieces of the output
    typedef typename QFrag<kQ>::type Q8;
    __shared__ f32x4 obuf[kWaves][kNt * kX][kWave];
    __shared__ float stat[3][kWaves][kRows];
    __shared__ int first_nan[kD];

    Item it;
    if (!Plan<kRows, kThreads, slots_few(kD, kNt), 4, kWholeFew, kLongFew>::find(a, blockIdx.x, it)) return;
    for (int d = (int)threadIdx.x; d < kD; d += kThreads) first_nan[d] = kNoNan;
    __syncthreads();
    const KvView &c = a.c;
    const int ln = lane(), col = ln & 15, g = ln >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(wave());
    const uint32_t b = __builtin_amdgcn_readfirstlane(it.b);
    const uint32_t head = __builtin_amdgcn_readfirstlane(it.head);
    const uint32_t s0 = __builtin_amdgcn_readfirstlane(it.s0);
    const int len = __builtin_amdgcn_readfirstlane(it.len), news = __builtin_amdgcn_readfirstlane(it.news);
    const uint32_t nrows = (uint32_t)news * a.group;
    const uint32_t row0 = __builtin_amdgcn_readfirstlane(it.rt) * kRows;
    const int per = (int)c.tshift - 4;
    const uint32_t sub_mask = (1u << per) - 1u;

    // The lane's query rows (operand columns) and the last token each sees; a
    // column past the last row computes row 0 with nothing seen.
    Q8 qf[kNt][kC][2];
    int limit[kNt];
    int low = len - 1, high = len - 1;      // least and largest limit of the tile's rows
    if (a.causal) {
        const uint32_t last = nrows - 1 < row0 + kRows - 1 ? nrows - 1 : row0 + kRows - 1;
        low = len - news + (int)(row0 / a.group);
        high = len - news + (int)(last / a.group);
    }
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
        const uint32_t r = row0 + n * 16 + col;
        const bool on = r < nrows;
        const uint32_t rr = on ? r : 0u, j = rr / a.group, h = head * a.group + rr % a.group;
        limit[n] = !on ? -1 : a.causal ? len - news + (int)j : len - 1;
        const uint16_t *const q = static_cast<const uint16_t *>(a.q) +
                                  (int64_t)(s0 + j) * a.q_tok + (int64_t)h * a.q_head + 16 * g;
#pragma unroll
        for (int k = 0; k < kC; ++k)
#pragma unroll
            for (int u = 0; u < 2; ++u)
                qf[n][k][u] = __builtin_bit_cast(Q8, *reinterpret_cast<const u32x4 *>(q + 64 * k + 8 * u));
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

    // The tiles that some row sees, in even parts.
    const int see = high < 0 ? 0 : high / kTile + 1;
    const int part = (see + (int)it.splits - 1) / (int)it.splits;
    const int t0 = (int)it.split * part;
    const int t1 = t0 + part < see ? t0 + part : see;
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
    // Codes are read once and past the caches (read like this, 5.8 TB/s; plainly,
    // 5.4). `on` false: no tile follows; the same few bytes for all lanes instead.
    auto load_k = [&](int t, bool on) {
        const uint32_t sub = (uint32_t)(t * 4 + kblk) & sub_mask;
        const uint32_t page = (uint32_t)pk < c.npages ? (uint32_t)pk : 0u;
        const uint64_t at = (uint64_t)page * c.page_bytes +
                            (((uint64_t)((head << per) + sub) * kBlock + (col & 3)) * kD + 16 * g);
        const uint8_t *const p = c.pool + (on ? at : 0u);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < kC; ++k)
                kr[j][k] = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4 *>(p + 4 * j * kD + 64 * k));
    };
    auto load_v = [&](int t, bool on) {
        const int bv = t * 4 + g;
        const uint32_t sub = (uint32_t)bv & sub_mask;
        const bool ok = (uint32_t)pv < c.npages;
        const uint32_t page = ok ? (uint32_t)pv : 0u;
        const uint8_t *const p = c.pool + (uint64_t)page * c.page_bytes;
        const uint8_t *const pvv = on ? p + c.code_bytes + (uint64_t)((head << per) + sub) * (kBlock * kD) +
                                            col * 16
                                      : c.pool;
        const float *const sc = reinterpret_cast<const float *>(p + 2ull * c.code_bytes) +
                                ((head << per) + sub);
        ks = sc[0];
        vs = sc[c.scales];
        const int left = len - bv * kBlock;
        valid = ok ? (left < 0 ? 0 : (left < kBlock ? left : kBlock)) : 0;
#pragma unroll
        for (int x = 0; x < kX; ++x)
            vr[x] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(pvv + 256 * x));
    };

    int t = t0 + wv;
    if (t < t1) {
        load_pages(t);
        // Wait for the queries here, with the pages: left to their first use, the
        // wait would stand in the loop and be one for all loads.
        __builtin_amdgcn_s_waitcnt(0x0f70);         // vmcnt(0)
        load_k(t, true);
        load_v(t, true);
        load_pages(t + kWaves < t1 ? t + kWaves : t);
        // The loads of the wave's next tile are in flight under the products of this
        // one. They are made in the last round too: were they conditional, the wait
        // for K at the top would have to be one for all loads.
        do {
            const bool more = t + kWaves < t1;
            const int after = more ? t + kWaves : t;
            const int later = t + 2 * kWaves < t1 ? t + 2 * kWaves : after;
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
            const int nvalid = valid;
            load_k(after, more);
            // With one wave a SIMD the products with the scales stand here, after the loads
            // of K: 32 requests of 500 to 8,000 tokens, D = 256, 56 us against 59 where the
            // compiler places them. With D = 128 it loses (a long cache 161 against 157 us),
            // with two row tiles of D = 256 registers spill.
            if constexpr (kD == 256 && kNt == 1) asm volatile("" : "+v"(ks), "+v"(vs));
            // Finite, so that a score of 0 stays one. (Taken before the loads of K, the
            // compiler waits for the scale between them.)
            const float kscale = fminf(ks, a.most_scale) * a.scale, vscale = vs;

            const int tok = t * kTile + g * kBlock;       // first token of the lane's block
            const bool edge = t * kTile + kTile - 1 > low;   // some row does not see the whole tile
            // (A scale of 0, of a page that was never written, stands for codes of 0.)
            const float ve = fmaxf((float)((int)(__float_as_uint(vscale) >> 23 & 0xffu) - 126), kMinExp + 1.0f);
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
                // The probability in f16 is p f. Where f would be large (a V scale far above
                // that of the row's largest score) part of it, 2^h, goes into the
                // exponential, so that neither factor leaves f32's range. f is written with
                // the scale itself: from its exponent alone the compiler takes the scale
                // earlier and waits for it before the loads of V (3 % of a long cache's time).
                const float rise = ms - mxs + kShift, h = fmaxf(rise + ve - kFar, 0.0f);
                const float f = nvalid == 0 ? 0.0f : vscale * exp2_(rise - h), from = ms - h;
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = exp2_(s[n][j][i] - from);
                        sum += p;
                        pf[n][j >> 1][(j & 1) * 4 + i] = (_Float16)(p * f);
                    }
                l[n] = __builtin_fmaf(sum, exp2_(-h), l[n] * exp2_(m[n] - ms));
                const float back = exp2_(mx[n] - mxs);
                m[n] = mn;
                mx[n] = mxn;
#pragma unroll
                for (int x = 0; x < kX; ++x) acc[n][x] *= back;
            }

            if (kCodes == DMADESC_KV_E4M3 && edge) {
                uint32_t found = 0;
#pragma unroll
                for (int x = 0; x < kX; ++x)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        vr[x][q] &= keep_mask(nvalid, q);
                        found |= nan_bytes(vr[x][q]);
                    }
                if (__ballot(found != 0)) {
#pragma unroll
                    for (int x = 0; x < kX; ++x)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t z = nan_bytes(vr[x][q]);
                            note_nan(first_nan, z, 16 * x + col, tok + 4 * q);
                            vr[x][q] = without(vr[x][q], z);
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
            load_v(after, more);
            load_pages(later);
            t += kWaves;
        } while (t < t1);
    }

    // Join the waves: common references first, then the sums through LDS, each
    // wave adding up its share of the 16-dimension pieces.
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
    if (a.plan && blockIdx.x == it.base && threadIdx.x == 0) a.plan[b] = make_uint2(it.base, it.splits);
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
        float mxa = -kInf;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) mxa = fmaxf(mxa, stat[1][w][n * 16 + col]);
        const float mine = exp2_(mx[n] - (mxa == -kInf ? 0.0f : mxa));
#pragma unroll
        for (int x = 0; x < kX; ++x) obuf[wv][n * kX + x][ln] = acc[n][x] * mine;
    }
    __syncthreads();
    const bool whole = it.splits == 1;
#pragma unroll 1
    for (int n = 0; n < kNt; ++n) {
        const uint32_t r = row0 + n * 16 + col;
        if (r >= nrows) break;                      // the lane's rows ascend
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
        // A row that sees nothing: zero, and no mass (la = 0).
        const float norm = la == 0.0f ? 0.0f : exp2_(mxs - ms - kShift) / la;
        const float lse2 = la == 0.0f ? -kInf : ms + __builtin_log2f(la);
        const uint64_t prow = (uint64_t)blockIdx.x * kRows + n * 16 + col;   // of the partial results
        const uint32_t j = r / a.group;
        const uint64_t orow = (uint64_t)(s0 + j) * a.heads + head * a.group + r % a.group;
        const int lim = a.causal ? len - news + (int)j : len - 1;
#pragma unroll 1
        for (int x = wv; x < kX; x += kWaves) {
            f32x4 o = obuf[0][n * kX + x][ln];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) o += obuf[w][n * kX + x][ln];
            o *= norm;
            if (kCodes == DMADESC_KV_E4M3) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (first_nan[16 * x + 4 * g + i] <= lim) o[i] = __builtin_nanf("");
            }
            if (whole) store4<kQ>(a.out, orow * kD + 16 * x + 4 * g, o);
            else *reinterpret_cast<f32x4 *>(a.part + prow * kD + 16 * x + 4 * g) = o;
        }
        if (wv == 0 && g == 0) {
            if (!whole) a.part_lse[prow] = lse2;
            else if (a.lse) a.lse[orow] = lse2 * 0.69314718055994531f;
        }
    }
}

// ------------------------------------------------------------- many rows ---

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mfma32(f16x8 a, f16x8 b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// The larger of x in this lane and in the lane 32 away.
__device__ __forceinline__ float half_max(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Attention for chunks of prompts, where the matrix cores are the bound: a
// workgroup takes 128 query rows of one key head, 32 a wave, and all of its
// waves walk the same tiles of 64 tokens. A tile's codes are turned into 16-bit
// floats once, on the way into LDS (two buffers each, one barrier a tile, the
// loads of later tiles in flight meanwhile). As above S^T = K Q^T and
// O^T = V^T P^T, here with the 32x32x16 product, which reads half the operand
// bytes per operation that the 16x16x32 one reads. K's tokens are laid in LDS
// with bits 2 and 3 of their number exchanged: then each lane's scores 8 c ..
// 8 c + 7 are tokens 8 h .. 8 h + 7 of block c (h = lane / 32), which is the
// order in which the second product takes them.
//
// Here the vector unit has more to do than the matrix unit (D = 128, a tile of a
// wave: 1,024 cycles of products, some 260 vector instructions of 4 cycles, 32 of
// them exponentials of 16), so that three things are done differently. The softmax takes one
// reference per row, the running maximum M of s + e: 2^(s + e - M + 13) is both the
// f16 probability and, times 2^-e once per block, the term of the sum; it moves
// only when a row passes it by 2^2, so that the accumulators are seldom rescaled
// (by 2^8, with terms that much nearer f16's end, took the same time): 11 bits
// down to 2^-27 of the row's largest term, fewer to 2^-37, nothing below.
// (Where scales lie beyond 2^-40..2^40 a term could vanish in the one and matter
// in the other; from the first such tile on the sum is taken from exponentials of
// its own.) The next codes are converted between the first product's
// instructions and a block's exponentials taken between the second's. And a wave
// in a product goes before the other wave of its SIMD. 2,048 tokens over 16,384,
// 32 heads on 8, D = 128, e4m3: 540 to 555 us by the card, 930 to 950 TFLOP/s (a
// library product of 8192^3: 1,217). By counters of that launch the matrix unit is busy 45 % of the cycles, the
// vector unit 63 %, LDS 42 %.
template <int kD, int kQ, int kCodes>
__global__ __launch_bounds__(kThreads, kD <= 64 ? 3 : kD <= 128 ? 2 : 1) void k_kv_attend_many(AttendArgs a)
{
    constexpr int kK = kD / 16;                     // steps of the first product
    constexpr int kX = kD / 32;                     // 32-dimension pieces of the output
    constexpr int kRows = (int)kRowsMany;
    constexpr int kChunkStride = kTile * 16 + 16;   // 8 dimensions of 64 tokens, and a bank step
    constexpr int kLoads = kTile * kD / 16 / kThreads;   // 16-byte loads of a thread, K and V each
    constexpr int kPieces = kD;                     // 16-byte pieces of a block
    constexpr float kRise = 2.0f, kLift = 13.0f;
    // The sum l stands 2^kSum above its terms relative to M. They may lie as far from M
    // as V scales lie from 1: with scales of 2^-64 to 2^127 and 2^29 tokens l stays
    // inside f32's range, and so does what matters of it 2^-30 further down.
    constexpr float kSum = 32.0f;
    typedef typename QFrag<kQ>::type Q8;
    __shared__ __align__(16) uint8_t kbuf[2][kD / 8 * kChunkStride];
    __shared__ __align__(16) uint8_t vbuf[2][kTile * kD * 2];
    __shared__ float scales[2][3][4];   // [buffer][scale of K, exponent of V, 2^(kSum - kLift - that)][block]
    __shared__ int first_nan[kD];

    Item it;
    if (!Plan<kRows, kThreads, slots_many(kD), 4, kWholeMany, kLongMany>::find(a, blockIdx.x, it)) return;
    for (int d = (int)threadIdx.x; d < kD; d += kThreads) first_nan[d] = kNoNan;
    __syncthreads();
    const KvView &c = a.c;
    const int ln = lane(), col = ln & 31, h = ln >> 5, tid = (int)threadIdx.x;
    const int wv = __builtin_amdgcn_readfirstlane(wave());
    const uint32_t b = __builtin_amdgcn_readfirstlane(it.b);
    const uint32_t head = __builtin_amdgcn_readfirstlane(it.head);
    const uint32_t row0 = __builtin_amdgcn_readfirstlane(it.rt) * kRows;
    const uint32_t wrow0 = row0 + wv * 32;   // first row of the wave
    const uint32_t s0 = __builtin_amdgcn_readfirstlane(it.s0);
    const int len = __builtin_amdgcn_readfirstlane(it.len), news = __builtin_amdgcn_readfirstlane(it.news);
    const uint32_t nrows = (uint32_t)news * a.group;
    const int per = (int)c.tshift - 4;
    const uint32_t sub_mask = (1u << per) - 1u;

    // Least and largest limit of the workgroup's rows, least of the wave's.
    int low = len - 1, high = len - 1, wlow = len - 1;
    if (a.causal) {
        const uint32_t last = nrows - 1 < row0 + kRows - 1 ? nrows - 1 : row0 + kRows - 1;
        low = len - news + (int)(row0 / a.group);
        high = len - news + (int)(last / a.group);
        wlow = len - news + (int)(wrow0 / a.group);
    }
    const int see = high < 0 ? 0 : high / kTile + 1;
    const int part = (see + (int)it.splits - 1) / (int)it.splits;
    const int t0 = (int)it.split * part;
    const int t1 = t0 + part < see ? t0 + part : see;

    Q8 qf[kK];
    const uint32_t r = wrow0 + col;
    const bool on = r < nrows;
    const uint32_t jq = on ? r / a.group : 0u, hq = head * a.group + (on ? r % a.group : 0u);
    const int limit = !on ? -1 : a.causal ? len - news + (int)jq : len - 1;
    {
        const uint16_t *const q = static_cast<const uint16_t *>(a.q) +
                                  (int64_t)(s0 + jq) * a.q_tok + (int64_t)hq * a.q_head + 8 * h;
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;   // a negative scale turns q round
#pragma unroll
        for (int k = 0; k < kK; ++k)
            qf[k] = __builtin_bit_cast(Q8, *reinterpret_cast<const u32x4 *>(q + 16 * k) ^ flip);
    }
    const float scale = fabsf(a.scale);

    f32x16 acc[kX];
#pragma unroll
    for (int x = 0; x < kX; ++x)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[x][i] = 0.0f;
    float mx = -kInf, l = 0.0f;

    // Staging: thread tid loads 16-byte pieces tid, tid + 256, .. of the tile's K
    // and V; a piece of K is 16 dimensions of a token, of V 16 tokens of a
    // dimension. A wave's 64 pieces lie in one block, so its page and address are
    // scalars, read from the lanes of a register that holds the pages of 64 blocks;
    // the next 64 are loaded 16 tiles ahead. Tiles past the last are staged too
    // (from addresses inside a page) and not used.
    const int32_t *const tab = c.table + (uint64_t)b * c.width;
    const int last_block = len > 0 ? (len - 1) / kBlock : 0;
    u32x4 kr[kLoads], vr[kLoads];
    float sc = 0.0f;
    int group = t0;                                 // tile of lane 0 of `here`; `ahead` follows it
    int32_t here, ahead;
    auto load_pages = [&](int t) -> int32_t {
        const int blk = t * 4 + ln;
        const uint32_t p = (uint32_t)tab[(blk < last_block ? blk : last_block) >> per];
        return (int32_t)(p < c.npages ? p : 0u);
    };
    auto piece_at = [&](int t, int i) -> const uint8_t * {
        const int first = wv * kWave + i * kThreads, blk = first / kPieces;
        const int32_t p = __builtin_amdgcn_readlane(here, (t - group) * 4 + blk);
        const uint32_t sub = (head << per) + ((uint32_t)(t * 4 + blk) & sub_mask);
        return c.pool + (uint64_t)(uint32_t)p * c.page_bytes + (uint64_t)sub * (kBlock * kD) +
               first % kPieces * 16;
    };
    auto load_k = [&](int t) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            kr[i] = *reinterpret_cast<const u32x4 *>(piece_at(t, i) + ln * 16);
    };
    auto load_v = [&](int t) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            vr[i] = *reinterpret_cast<const u32x4 *>(piece_at(t, i) + c.code_bytes + ln * 16);
        if (wv == 0) {                              // lanes 0..7: K's and V's scales of the 4 blocks
            const uint32_t p = (uint32_t)__shfl(here, (t - group) * 4 + (ln & 3), kWave);
            const uint32_t sub = (head << per) + ((uint32_t)(t * 4 + (ln & 3)) & sub_mask);
            if (ln < 8)
                sc = reinterpret_cast<const float *>(c.pool + (uint64_t)p * c.page_bytes +
                                                     2ull * c.code_bytes)[(ln >> 2) * c.scales + sub];
        }
    };
    auto clean_v = [&](int t) {                     // the tile's codes that must not count
        if (kCodes == DMADESC_KV_E4M3 && t * kTile + kTile - 1 > low) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int piece = tid + i * kThreads, in = piece % kPieces;
                const int tok0 = t * kTile + piece / kPieces * kBlock;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    vr[i][q] &= keep_mask(len - tok0, q);
                    const uint32_t z = nan_bytes(vr[i][q]);
                    note_nan(first_nan, z, in, tok0 + 4 * q);
                    vr[i][q] = without(vr[i][q], z);
                }
            }
        }
    };
    // Half n of the thread's pieces (8 codes each): K's, then V's.
    constexpr int kOps = 4 * kLoads;
    auto stage = [&](int buf, int n) {
        const int i = n >> 1 & (kLoads - 1), piece = tid + i * kThreads;
        const int blk = piece / kPieces, in = piece % kPieces;
        if (n < kOps / 2) {
            const int tok = in / (kD / 16), x = in % (kD / 16);
            const int pos = blk * 16 + ((tok & 3) | (tok >> 1 & 4) | (tok << 1 & 8));
            *reinterpret_cast<Q8 *>(kbuf[buf] + (2 * x + (n & 1)) * kChunkStride + pos * 16) =
                codes8<kCodes, Q8>(kr[i][2 * (n & 1)], kr[i][2 * (n & 1) + 1]);
        } else {
            reinterpret_cast<f16x8 *>(vbuf[buf])[(blk * 2 + (n & 1)) * kD + in] =
                codes8<kCodes, f16x8>(vr[i][2 * (n & 1)], vr[i][2 * (n & 1) + 1]);
        }
    };
    auto stage_scales = [&](int t, int buf) {
        if (tid < 8) {                              // K: scale; V: exponent and 2^-exponent
            const float s = (t * 4 + (tid & 3)) * kBlock < len ? sc : 1.0f;
            // (A scale of 0, of a page that was never written, stands for codes of 0.)
            const int eb = (int)(__float_as_uint(s) >> 23 & 0xffu) - 127, e = eb < kMinExp ? kMinExp : eb;
            if (tid < 4) {
                // Never 0, so that a masked -inf stays one, and finite, so that a 0 does.
                scales[buf][0][tid] = fmaxf(fminf(s, a.most_scale) * scale, 1.4e-45f);
            } else {
                scales[buf][1][tid - 4] = (float)e;
                scales[buf][2][tid - 4] = __uint_as_float((uint32_t)(127 + (int)(kSum - kLift) - e) << 23);
            }
        }
    };
    auto k_operand = [&](int buf, int k) -> Q8 {
        return *reinterpret_cast<const Q8 *>(kbuf[buf] + (2 * (k >> 1) + h) * kChunkStride +
                                             ((k & 1) * 32 + col) * 16);
    };
    auto v_operand = [&](int buf, int k) -> f16x8 {
        return reinterpret_cast<const f16x8 *>(vbuf[buf])[(k / kX * 2 + h) * kD + k % kX * 32 + col];
    };
    auto fetch = [&](int t) {                       // tile t's codes, of this group of 16 or the next
        if (t >= group + 16) {
            group += 16;
            here = ahead;
            ahead = load_pages(group + 16);
        }
        load_k(t);
        load_v(t);
    };

    bool wide = false;                              // scales too far apart for one exponential
    if (t0 < t1) {
        here = load_pages(t0);
        ahead = load_pages(t0 + 16);
        load_k(t0);
        load_v(t0);
        clean_v(t0);
#pragma unroll
        for (int n = 0; n < kOps; ++n) stage(0, n);
        stage_scales(t0, 0);
        fetch(t0 + 1);
    }
    if (wrow0 >= nrows) {                           // a wave past the last row only stages
        for (int t = t0; t < t1; ++t) {
            const int buf = (t - t0) & 1;
            __syncthreads();
            clean_v(t + 1);
#pragma unroll
            for (int n = 0; n < kOps; ++n) stage(buf ^ 1, n);
            stage_scales(t + 1, buf ^ 1);
            fetch(t + 2);
        }
        return;
    }
    // In LDS as tile t begins: its codes; in registers: those of t + 1.
    for (int t = t0; t < t1; ++t) {
        const int buf = (t - t0) & 1;
        Q8 kf[4];
        f16x8 vf[4];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) kf[k] = k_operand(buf, k);
        clean_v(t + 1);
        // The scores, the next codes' conversion under them.
        f32x16 s[2];
#pragma unroll
        for (int i = 0; i < 16; ++i) s[0][i] = s[1][i] = 0.0f;
        __builtin_amdgcn_sched_barrier(0);
        constexpr int kSteps = 2 * kK;
        __builtin_amdgcn_s_setprio(1);              // the matrix unit before the other wave's vector work
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
            if (k + 3 < kSteps) kf[(k + 3) & 3] = k_operand(buf, k + 3);
            else vf[k + 3 - kSteps] = v_operand(buf, k + 3 - kSteps);
            s[k & 1] = mfma32(kf[k & 3], qf[k >> 1], s[k & 1]);
#pragma unroll
            for (int m = k * kOps / kSteps; m < (k + 1) * kOps / kSteps; ++m) stage(buf ^ 1, m);
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_setprio(0);
        stage_scales(t + 1, buf ^ 1);
        fetch(t + 2);
        float ks[4], ve[4], back[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ks[i] = scales[buf][0][i];
            ve[i] = scales[buf][1][i];
            back[i] = scales[buf][2][i];
            wide |= fabsf(ve[i]) > 40.0f;
        }
        if (t * kTile + kTile - 1 > wlow) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int tok = t * kTile + u * 32 + (i >> 3) * 16 + 8 * h + (i & 7);
                    s[u][i] = tok <= limit ? s[u][i] : -kInf;
                }
        }
        // The reference moves where a row's maximum has risen far enough.
        float tv = -kInf;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = -kInf;
#pragma unroll
            for (int k = 0; k < 8; ++k) top = fmaxf(top, s[i >> 1][(i & 1) * 8 + k]);
            tv = fmaxf(tv, __builtin_fmaf(top, ks[i], ve[i]));
        }
        tv = half_max(tv);
        if (__ballot(tv > mx + kRise)) {
            const float mxn = fmaxf(mx, tv);
            // In two factors: where M rises over the whole range of scales, one alone
            // would lie below f32's range and l, which need not be small then, be lost.
            const float half = mxn == -kInf ? 1.0f : exp2_(0.5f * (mx - mxn)), by = half * half;
            l = l * half * half;
            mx = mxn;
#pragma unroll
            for (int x = 0; x < kX; ++x) acc[x] *= by;
        }
        const float ref = (mx == -kInf ? 0.0f : mx) - kLift;
        if (__builtin_amdgcn_readfirstlane(wide)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    l += exp2_(__builtin_fmaf(s[i >> 1][(i & 1) * 8 + k], ks[i], kSum - kLift - ref));
                back[i] = 0.0f;
            }
        }
        // The exponentials of block i + 1 under block i's product with V.
        f16x8 pf[2];
        float sum = 0.0f;
        auto take = [&](int i, int k) {
            const float p = exp2_(__builtin_fmaf(s[i >> 1][(i & 1) * 8 + k], ks[i], ve[i] - ref));
            sum += p;
            pf[i & 1][k] = (_Float16)p;
        };
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < 8; ++k) take(0, k);
        __builtin_amdgcn_s_setprio(1);
        l = __builtin_fmaf(sum, back[0], l);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sum = 0.0f;
#pragma unroll
            for (int x = 0; x < kX; ++x) {
                const int k = i * kX + x;
                if (k + 3 < 4 * kX) vf[(k + 3) & 3] = v_operand(buf, k + 3);
                acc[x] = mfma32(vf[k & 3], pf[i & 1], acc[x]);
                if (i < 3)
#pragma unroll
                    for (int e = x * 8 / kX; e < (x + 1) * 8 / kX; ++e) take(i + 1, e);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (i < 3) l = __builtin_fmaf(sum, back[i + 1], l);
        }
        __builtin_amdgcn_s_setprio(0);
    }

    if (a.plan && blockIdx.x == it.base && tid == 0) a.plan[b] = make_uint2(it.base, it.splits);
    l += __shfl_xor(l, 32, kWave);
    if (!on) return;
    const uint64_t orow = (uint64_t)(s0 + jq) * a.heads + hq;
    const uint64_t prow = (uint64_t)blockIdx.x * kRows + (r - row0);
    const float norm = l == 0.0f ? 0.0f : exp2_(kSum - kLift) / l;
    const float lse2 = l == 0.0f ? -kInf : mx - kSum + __builtin_log2f(l);
#pragma unroll
    for (int x = 0; x < kX; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4 o = f32x4{acc[x][4 * i], acc[x][4 * i + 1], acc[x][4 * i + 2],
                            acc[x][4 * i + 3]} * norm;
            const int d = 32 * x + 8 * i + 4 * h;
            if (kCodes == DMADESC_KV_E4M3) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (first_nan[d + k] <= limit) o[k] = __builtin_nanf("");
            }
            if (it.splits == 1) store4<kQ>(a.out, orow * kD + d, o);
            else *reinterpret_cast<f32x4 *>(a.part + prow * kD + d) = o;
        }
    if (h == 0) {
        if (it.splits != 1) a.part_lse[prow] = lse2;
        else if (a.lse) a.lse[orow] = lse2 * 0.69314718055994531f;
    }
}

// Joins the splits of 16 query rows of one key head. Groups of kD / 4 lanes take
// a row each, or several groups a row where the rows are fewer, every group
// some of the splits. The chunks of 16 are numbered without a scan: request b's
// first is q_start[b] * group / 16 + b.
constexpr uint32_t kJoinRows = 16;
// Threads of its workgroups: 512 where they all run at once (420 of them: 5.3 us,
// with 256 threads 6.2), 256 where they are many and most find nothing to join
// (4,000: 5.3 us, with 512 threads 9.6).
constexpr uint32_t kJoinWide = 512, kJoinNarrow = 256, kJoinOnce = 1024;

template <int kD, int kQ, int kJoinThreads>
__global__ __launch_bounds__(kJoinThreads) void k_kv_join(AttendArgs few, AttendArgs many,
                                                     uint32_t tile_rows)
{
    constexpr uint32_t kLanes = kD / 4, kGroups = kJoinThreads / kLanes;
    __shared__ f32x4 osum[kGroups][kLanes];
    const uint32_t head = blockIdx.x % few.c.kv_heads, chunk = blockIdx.x / few.c.kv_heads;
    const uint32_t b = kv_request_of(few.c.rows, chunk, [&](uint32_t r) {
        const int32_t s = few.q_start[r];
        const uint64_t u = s < 0 ? 0u : ((uint32_t)s > few.total ? few.total : (uint32_t)s);
        return u * few.group / kJoinRows + r;
    });
    uint32_t s0, s1;
    kv_span(few.q_start, b, few.total, s0, s1);
    const uint32_t nrows = (s1 - s0) * few.group;
    const int64_t r0 = ((int64_t)chunk - (int64_t)((uint64_t)s0 * few.group / kJoinRows + b)) * kJoinRows;
    if (r0 < 0 || r0 >= nrows) return;
    const bool is_many = nrows > few.most;
    const AttendArgs &a = is_many ? many : few;
    if (is_many) tile_rows = kRowsMany;
    const uint2 plan = a.plan[b];
    if (plan.y <= 1 || plan.y > kMaxSplits) return;
    const uint32_t rts = (nrows + tile_rows - 1) / tile_rows;
    const uint32_t first = plan.x + (uint32_t)r0 / tile_rows * a.c.kv_heads + head;
    const uint32_t step = a.c.kv_heads * rts;
    if ((uint64_t)first + (uint64_t)(plan.y - 1) * step >= a.slots) return;   // q_start out of order

    const uint32_t rows = nrows - (uint32_t)r0 < kJoinRows ? nrows - (uint32_t)r0 : kJoinRows;
    const uint32_t width = rows < kGroups ? rows : kGroups;       // rows at a time
    const uint32_t share = kGroups / width;                       // groups of a row
    const uint32_t grp = threadIdx.x / kLanes, at = threadIdx.x % kLanes;
    const uint32_t phase = grp / width;
    for (uint32_t base = 0; base < rows; base += width) {
        const uint32_t row = base + grp % width;
        const bool on = phase < share && row < rows;
        const uint64_t in = (uint32_t)r0 % tile_rows + row;
        float top = -kInf, all = 0.0f;
        f32x4 o = {0, 0, 0, 0};
        if (on) {
            float mine = -kInf;
            for (uint32_t s = at; s < plan.y; s += kLanes) {
                const float x = a.part_lse[(uint64_t)(first + s * step) * tile_rows + in];
                top = fmaxf(mine, x);
                const float ref = top == -kInf ? 0.0f : top;
                all = all * exp2_(mine - ref) + exp2_(x - ref);
                mine = top;
            }
#pragma unroll
            for (int d = (int)kLanes / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, kLanes));
            if (top == -kInf) top = 0.0f;
            all *= exp2_(mine - top);
#pragma unroll
            for (int d = (int)kLanes / 2; d > 0; d >>= 1) all += __shfl_xor(all, d, kLanes);
            // A part's weight in two factors: alone it may lie below f32's range where its
            // part's values are large; and over kMaxSplits, so that no sum passes the
            // range that its parts lie in.
#pragma unroll 4
            for (uint32_t s = phase; s < plan.y; s += share) {
                const uint64_t p = (uint64_t)(first + s * step) * tile_rows + in;
                const float v = exp2_(0.5f * (a.part_lse[p] - top));
                o += *reinterpret_cast<const f32x4 *>(a.part + p * kD + at * 4) * v * (v * (1.0f / kMaxSplits));
            }
        }
        osum[grp][at] = o;
        __syncthreads();
        if (on && phase == 0) {
            for (uint32_t k = 1; k < share; ++k) o += osum[grp + k * width][at];
            const uint32_t r = (uint32_t)r0 + row;
            const uint64_t orow = (uint64_t)(s0 + r / a.group) * a.heads + head * a.group + r % a.group;
            const float norm = all == 0.0f ? 0.0f : (float)kMaxSplits / all;
            store4<kQ>(a.out, orow * kD + at * 4, o * norm);
            if (a.lse && at == 0)
                a.lse[orow] = all == 0.0f ? -kInf : (top + __builtin_log2f(all)) * 0.69314718055994531f;
        }
        __syncthreads();
    }
}

// How a call's memory and launches follow from what the host knows, which is
// not the requests' own sizes. Up to 32 query rows per key head on the average
// of all table rows the kernel of few rows takes all requests, past that the
// kernel of many rows (35 rows, 33 requests: 43 us by three row tiles of the
// first, 38 by the second; 28 rows: 32 and 34; D = 256, 32 rows: 27 and 41). Both
// are launched and share the requests where that average is at most 32 and one
// request could have more than 1,024 rows if each other table row brought a
// token: an idle launch costs 4 us. The average is no rule for uneven batches:
// 63 requests of a token (123 us alone) and a chunk of 2,048 over 4,096 (134) take
// 281 us together, the chunk of 512 tokens of one request 24 us alone and 49 in a
// table of 512 rows that bring nothing.
struct Launch {
    uint32_t tile_rows;          // of the kernel of few rows: one product's 16, or 32
    uint32_t few, many;          // workgroups (= partial results) of each kernel
    uint32_t most;               // rows of a request up to which it is the first kernel's
    uint32_t join;               // workgroups of the join, 0: nothing can be split
    size_t plan_at, few_lse, few_part, many_lse, many_part, bytes;
    bool fits;                   // false: too many workgroups for a launch, the rest is not set
};

Launch launch_of(uint64_t total, uint32_t rows, uint32_t heads, uint32_t kv_heads, uint32_t dim,
                 uint64_t tokens)
{
    Launch p{};
    const uint64_t group = heads / kv_heads, all = total * group;
    const uint64_t mean = (total + rows - 1) / rows * group;
    const uint64_t tiles = (tokens + kTile - 1) / kTile;
    const bool split_few = tiles > kWholeFew, split_many = tiles > kWholeMany;
    const bool few = mean <= 32u, both = few && total > rows && (total - rows) * group > 1024;
    p.most = !few ? 0u : both ? kMostFew : ~0u;
    p.tile_rows = mean <= 16 ? 16u : 32u;
    // Unsplit pieces: a row tile of a key head each; all rows' whole tiles and one
    // more of each request at most.
    const uint64_t few_rows = both && all > rows * (uint64_t)kMostFew ? rows * (uint64_t)kMostFew : all;
    const uint64_t big = both ? all / (kMostFew + 1) : rows;      // requests that have many
    auto grid = [&](uint64_t base, bool split, uint32_t slots, uint32_t long_) -> uint64_t {
        if (!split || base > kKvMaxGroups) return base;
        const uint32_t one = most_pieces((uint32_t)base, slots), two = most_pieces((uint32_t)base, 2 * slots);
        return base * tiles > (uint64_t)long_ * slots / 4 && two > one ? two : one;
    };
    uint64_t n_few = 0, n_many = 0, n_join = 0;
    if (few)
        n_few = grid(kv_heads * (few_rows / p.tile_rows + rows), split_few,
                     slots_few((int)dim, (int)p.tile_rows / 16), kLongFew);
    if (!few || both)
        n_many = grid(kv_heads * (all / kRowsMany + (big < rows ? big : rows)), split_many,
                      slots_many((int)dim), kLongMany);
    if ((n_few && split_few) || (n_many && split_many)) n_join = kv_heads * (all / kJoinRows + rows);
    p.fits = n_few <= kKvMaxGroups && n_many <= kKvMaxGroups && n_join <= kKvMaxGroups;
    if (!p.fits) return p;
    p.few = (uint32_t)n_few;
    p.many = (uint32_t)n_many;
    p.join = (uint32_t)n_join;
    size_t at = align256(8ull * rows);
    auto take = [&](size_t bytes) { const size_t r = at; at += align256(bytes); return r; };
    const size_t f = split_few ? p.few : 0, n = split_many ? p.many : 0;
    p.few_lse = take(4 * f * p.tile_rows);
    p.few_part = take(4 * f * p.tile_rows * dim);
    p.many_lse = take(4 * n * kRowsMany);
    p.many_part = take(4 * n * kRowsMany * dim);
    p.bytes = p.join ? at : 0;                       // nothing to join: no partial results, no plan
    return p;
}

template <int kD, int kQ, int kCodes>
void launch_all(const AttendArgs &few, const AttendArgs &many, const Launch &p, hipStream_t s)
{
    if (p.many) k_kv_attend_many<kD, kQ, kCodes><<<p.many, kThreads, 0, s>>>(many);
    if (p.few) {
        if (p.tile_rows == 16) k_kv_attend<kD, kQ, kCodes, 1><<<p.few, kThreads, 0, s>>>(few);
        else k_kv_attend<kD, kQ, kCodes, 2><<<p.few, kThreads, 0, s>>>(few);
    }
    if (p.join && p.join <= kJoinOnce)
        k_kv_join<kD, kQ, kJoinWide><<<p.join, kJoinWide, 0, s>>>(few, many, p.tile_rows);
    else if (p.join)
        k_kv_join<kD, kQ, kJoinNarrow><<<p.join, kJoinNarrow, 0, s>>>(few, many, p.tile_rows);
}

template <int kD>
void launch_dim(const KvAttendArgs &k, const AttendArgs &few, const AttendArgs &many,
                const Launch &p, hipStream_t s)
{
    const bool e4m3 = k.cache.codes == DMADESC_KV_E4M3;
    if (k.type == DMADESC_KV_BF16) {
        if (e4m3) launch_all<kD, DMADESC_KV_BF16, DMADESC_KV_E4M3>(few, many, p, s);
        else launch_all<kD, DMADESC_KV_BF16, DMADESC_KV_INT8>(few, many, p, s);
    } else {
        if (e4m3) launch_all<kD, DMADESC_KV_FP16, DMADESC_KV_E4M3>(few, many, p, s);
        else launch_all<kD, DMADESC_KV_FP16, DMADESC_KV_INT8>(few, many, p, s);
    }
}

}  // namespace

bool kv_attend_fits(uint64_t total, uint32_t rows, uint32_t heads, uint32_t kv_heads, uint32_t dim,
                    uint64_t tokens)
{
    return launch_of(total, rows, heads, kv_heads, dim, tokens).fits;
}

size_t ws_kv_attend(uint64_t total, uint32_t rows, uint32_t heads, uint32_t kv_heads,
                    uint32_t dim, uint64_t tokens)
{
    if (total == 0 || rows == 0) return 0;
    return launch_of(total, rows, heads, kv_heads, dim, tokens).bytes;
}

hipError_t launch_kv_attend(const KvAttendArgs &k, hipStream_t s)
{
    const dmadesc_kv_cache &c = k.cache;
    const Launch p = launch_of(k.total, c.rows, k.heads, c.kv_heads, c.dim,
                               (uint64_t)c.width * c.page_tokens);
    AttendArgs few{};
    few.c = kv_view(c);
    if (few.c.npages == 0) few.c.width = 0;             // no page: every length is 0
    few.q = k.q;
    few.q_tok = k.q_tok;
    few.q_head = k.q_head;
    few.q_start = k.q_start;
    few.total = (uint32_t)k.total;
    few.heads = k.heads;
    few.group = k.heads / c.kv_heads;
    few.causal = k.causal;
    const float scale = k.scale != 0.0f ? k.scale : 1.0f / sqrtf((float)c.dim);
    few.scale = scale * 1.44269504088896341f;
    few.most_scale = 0x1p127f / fabsf(few.scale);
    few.out = k.out;
    few.lse = k.lse;
    uint8_t *const ws = static_cast<uint8_t *>(k.ws);
    few.plan = p.join ? reinterpret_cast<uint2 *>(ws + p.plan_at) : nullptr;
    AttendArgs many = few;
    few.part = reinterpret_cast<float *>(ws + p.few_part);
    few.part_lse = reinterpret_cast<float *>(ws + p.few_lse);
    few.slots = p.few;
    few.least = 1;
    few.most = p.most;
    many.part = reinterpret_cast<float *>(ws + p.many_part);
    many.part_lse = reinterpret_cast<float *>(ws + p.many_lse);
    many.slots = p.many;
    many.least = p.most + 1;
    many.most = ~0u;
    if (c.dim == 64) launch_dim<64>(k, few, many, p, s);
    else if (c.dim == 128) launch_dim<128>(k, few, many, p, s);
    else launch_dim<256>(k, few, many, p, s);
    return hipGetLastError();
}

}  // namespace dd
