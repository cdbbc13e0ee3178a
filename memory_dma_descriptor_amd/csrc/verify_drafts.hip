// verify_drafts.hip - which tokens of a drafted tree the target accepts, and the
// token after them, from given random numbers, for gfx950.
//
// Mathematics: sampling without replacement against the target. At a node with
// target row p and draft row d its children are tried in order. The remainder
// before any is refused is p; after a token is refused it is the positive part of
// w / W - d / Q, w the remainder, W its mass and Q the mass of d without the
// tokens refused. A refused token has none of it left (it was refused because
// u d(x) / Q >= w(x) / W with u < 1), and so w = max(p - c d, 0) for one number c:
// c = 0 at first, and c + W / Q after a refusal. The rows count as having mass 1
// before any refusal. Without a draft row the drafts are certain, and the
// remainder is p without the tokens refused. Everything is f64 and summed in one fixed
// order, so that a call answers the same every time; a sum in another order could answer
// otherwise only where u stands within the last bits of a border.
//
// One workgroup a request, one launch. The walk's tests read two numbers each,
// gathered for all nodes at once, and a first child's test depends on nothing
// else; one wave walks, and all sum a mass W where a child follows a refused one.
// Then the weights of the last node are summed in 64 even parts, four of a wave,
// and one wave looks for the place where the running sum passes u W: for the
// part, for the 64th of it, for the weight.
//
// Bound: one compute unit's stream over a row, and steps that wait for one another.
// 64 requests of 6 rows, 131,072 f32 numbers, draft rows: 25 us, 67 MB read, 20 of them
// in the sums (13 where the rows are in the caches); without draft rows 14; 24 trees of
// 32, 50,257 bf16: 36 us, 6 for each refused child of all requests with another behind
// it; one request of 25, 32,000, certain: 6.8. Several workgroups to a row for the draw,
// in a second launch, took 7 + 64, 29 + 19 and 4 + 12.
#include <type_traits>

#include "dd_internal.h"
#include "dd_kv.hpp"

namespace dd {
namespace {

constexpr int kMost = (int)DMADESC_TREE_MOST;
constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / kWave;
constexpr int kOwn = 4;                                 // parts of a wave
constexpr int kParts = kOwn * kWaves;
constexpr uint32_t kLongPart = kWave * kWave;           // weights of a part that a wave finishes alone
constexpr int kBits = 1 << 14;                          // of the refused tokens, by runs of a load

struct Args {
    const void *probs, *draft;
    int64_t probs_row, draft_row;
    uint32_t vocab;                                     // < 2^31, so that places past it still fit
    const int32_t *tokens, *parent, *q_start;
    uint32_t rows, total;
    const float *u;
    int32_t *path, *count, *next;
    uint8_t *status;
};

// The tokens refused at a node; without a draft row, also a bit for each run of
// numbers that a load takes, which says where to look the list up.
struct Refused {
    int32_t token[kMost];
    uint32_t bits[kBits / 32];
};

constexpr int kN = 4;                                   // numbers that a thread loads at once

// What is negative or NaN counts as 0, infinity as the largest number. (The median
// is the least of the three where one is NaN, and 0 of a quiet one; a signalling one,
// which a minimum hands on, is made quiet first.)
__device__ __forceinline__ float sound(float x)
{
    return __builtin_amdgcn_fmed3f(__builtin_canonicalizef(x), 0.0f, 3.402823466e38f);
}

template <int kType>
__device__ __forceinline__ float number(const void *p, int64_t at)
{
    float x;
    if constexpr (kType == DMADESC_KV_FP32) x = static_cast<const float *>(p)[at];
    else if constexpr (kType == DMADESC_KV_BF16) x = __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[at] << 16);
    else x = (float)static_cast<const _Float16 *>(p)[at];
    return sound(x);
}

// kN numbers as they lie in memory, at any place.
template <int kType>
struct Raw {
    typedef typename std::conditional<kType == DMADESC_KV_FP32, uint32_t, uint16_t>::type Bits;
    uint32_t w[kN * sizeof(Bits) / 4];

    __device__ __forceinline__ void load(const void *p, int64_t at)
    {
        __builtin_memcpy(w, static_cast<const Bits *>(p) + at, sizeof w);
    }
    // Number i as it counts (kSound), or as it is.
    template <bool kSound>
    __device__ __forceinline__ float get(int i) const
    {
        float x;
        if constexpr (kType == DMADESC_KV_FP32) x = __uint_as_float(w[i]);
        else if constexpr (kType == DMADESC_KV_BF16)
            x = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        else x = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i / 2] >> (16 * (i & 1))));
        return kSound ? sound(x) : x;
    }
    // `bits` and all bits of the numbers.
    __device__ __forceinline__ uint32_t all_bits(uint32_t bits) const
    {
#pragma unroll
        for (uint32_t x : w) bits |= x;
        return bits;
    }
    // Whether the numbers that `bits` come from are 0 or more and less than 2, and so
    // count as they are: neither the sign nor the first bit of the exponent is set.
    static __device__ __forceinline__ bool all_sound(uint32_t bits)
    {
        return (bits & (kType == DMADESC_KV_FP32 ? 0xc0000000u : 0xc000c000u)) == 0;
    }
};

// Sums across lanes through the vector unit's own lane moves (a step takes some
// 30 cycles; the shuffles of dd_device.hpp, which pass through LDS, 150).
template <int kCtrl, int kRowMask = 0xf>
__device__ __forceinline__ double moved(double x)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, kCtrl, kRowMask, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), kCtrl, kRowMask, 0xf, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Inclusive running sum across the wave: rows of 16 lanes, then their ends.
__device__ __forceinline__ double running_sum(double x)
{
    x += moved<0x111>(x);               // from 1, 2, 4 and 8 lanes to the left in the row
    x += moved<0x112>(x);
    x += moved<0x114>(x);
    x += moved<0x118>(x);
    x += moved<0x142, 0xa>(x);          // lane 15 to row 1, 47 to row 3
    x += moved<0x143, 0xc>(x);          // lane 31 to rows 2 and 3
    return x;
}

// The sum of a row of 16 lanes, in all of them.
__device__ __forceinline__ double row_sum(double x)
{
    x += moved<0x128>(x);               // turned by 8, 4, 2, 1
    x += moved<0x124>(x);
    x += moved<0x122>(x);
    x += moved<0x121>(x);
    return x;
}

__device__ __forceinline__ double lane_value(double x, int from)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, from);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), from);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Whether a lane's condition holds, where it is the same in all lanes.
__device__ __forceinline__ bool uniform(bool x) { return __ballot(x) != 0; }

__device__ __forceinline__ double remains(float p, float d, double c)
{
    return __builtin_fmax((double)p - c * (double)d, 0.0);      // (all finite)
}

// What is drawn from: a row of probs and of draft, c, and the refused tokens.
struct Row {
    int64_t p, d;
    double c;
    int refused;                                        // of the list; without a draft row
};

// A run of kN weights.
template <int kType, bool kDraft>
struct Run {
    Raw<kType> p, d;

    __device__ __forceinline__ void load(const Args &a, const Row &w, int64_t at)
    {
        p.load(a.probs, w.p + at);
        if constexpr (kDraft) d.load(a.draft, w.d + at);
    }
    __device__ __forceinline__ uint32_t all_bits(uint32_t bits) const
    {
        bits = p.all_bits(bits);
        if constexpr (kDraft) bits = d.all_bits(bits);
        return bits;
    }
    // Their sum, of places lo .. hi - 1 of the row if `part`; the run starts at `at`.
    template <bool kSound>
    __device__ __forceinline__ double sum(const Row &w, const Refused &no, uint32_t at, bool part, uint32_t lo,
                                          uint32_t hi) const
    {
        double x[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const float pi = p.template get<kSound>(i);
            if constexpr (kDraft) x[i] = remains(pi, d.template get<kSound>(i), w.c);
            else x[i] = (double)pi;
        }
        if (part) {
#pragma unroll
            for (int i = 0; i < kN; ++i) x[i] = at + i >= lo && at + i < hi ? x[i] : 0.0;
        }
        if constexpr (!kDraft) {
            if (w.refused > 0) {
                const uint32_t bit = lo / kN & (kBits - 1);
                if (no.bits[bit / 32] >> (bit & 31) & 1u)
                    for (int k = 0; k < w.refused; ++k) {
                        const uint32_t y = (uint32_t)no.token[k] - at;
#pragma unroll
                        for (int i = 0; i < kN; ++i) x[i] = y == (uint32_t)i ? 0.0 : x[i];
                    }
            }
        }
        return (x[0] + x[1]) + (x[2] + x[3]);
    }
};

// One weight, of any row length.
template <int kType, bool kDraft>
__device__ __forceinline__ double weight(const Args &a, const Row &w, const Refused &no, uint32_t at)
{
    const float p = number<kType>(a.probs, w.p + at);
    if constexpr (kDraft) return remains(p, number<kType>(a.draft, w.d + at), w.c);
    bool out = false;
    for (int k = 0; k < w.refused; ++k) out |= (uint32_t)no.token[k] == at;
    return out ? 0.0 : (double)p;
}

// Masses of the kParts parts of [from, end), `part` weights each (a multiple of a
// wave's loads), in masses[]. Called by the whole workgroup.
template <int kType, bool kDraft>
__device__ __forceinline__ void sum_parts(const Args &a, const Row &w, const Refused &no, uint32_t from, uint32_t end,
                                          uint32_t part, double *masses)
{
    const int ln = lane();
    double sum[kOwn] = {};
    const uint32_t start = from + (uint32_t)__builtin_amdgcn_readfirstlane(wave()) * kOwn * part;
    typedef Run<kType, kDraft> R;
    // Numbers are summed as they are, and once more as they count if some are not
    // ordinary: made sound one by one, the listed trees take 40.3 us, so 35.8.
    uint32_t bits = 0;
    // The wave's parts, any of which may hold the row's end: a run that would pass it is
    // moved back, and counts from its own place on (`end` is the row's or a multiple of
    // kN).
    auto by_runs = [&](auto as_they_count) {
        constexpr bool kSound = decltype(as_they_count)::value;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) sum[i] = 0.0;
        for (uint32_t k = 0; k < part; k += kWave * kN) {
            R run[kOwn];
            uint32_t at[kOwn];
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                at[i] = start + i * part + k + (uint32_t)ln * kN;
                run[i].load(a, w, at[i] < a.vocab - kN ? at[i] : a.vocab - kN);
            }
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                const uint32_t place = at[i] < a.vocab - kN ? at[i] : a.vocab - kN;
                sum[i] += run[i].template sum<kSound>(w, no, place, true, at[i], end);
                if (!kSound) bits = run[i].all_bits(bits);
            }
        }
    };
    if (a.vocab < (uint32_t)kN) {
        if (start + ln < end) sum[0] = weight<kType, kDraft>(a, w, no, start + ln);
    } else if (start + kOwn * part <= end) {
        // The next loads are in flight under this round's sums.
        R now[kOwn], next[kOwn];
        const uint32_t own = (uint32_t)ln * kN;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) now[i].load(a, w, (int64_t)(start + i * part) + own);
        for (uint32_t k = 0; k < part; k += kWave * kN) {
            const uint32_t after = k + kWave * kN < part ? k + kWave * kN : k;
#pragma unroll
            for (int i = 0; i < kOwn; ++i) next[i].load(a, w, (int64_t)(start + i * part + after) + own);
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                const uint32_t at = start + i * part + k + own;
                sum[i] += now[i].template sum<false>(w, no, at, false, at, end);
                bits = now[i].all_bits(bits);
                now[i] = next[i];
            }
        }
    } else if (start < end) {
        by_runs(std::false_type{});
    }
    if (uniform(!Raw<kType>::all_sound(bits))) by_runs(std::true_type{});
    // Lane 16 i ends up with the sum of part i.
    static_assert(kOwn == 4);
    const bool up = ln & 32, odd = ln & 16;
    const double s0 = (up ? sum[2] : sum[0]) + __shfl_xor(up ? sum[0] : sum[2], 32, kWave);
    const double s1 = (up ? sum[3] : sum[1]) + __shfl_xor(up ? sum[1] : sum[3], 32, kWave);
    const double s = row_sum((odd ? s1 : s0) + __shfl_xor(odd ? s0 : s1, 16, kWave));
    __syncthreads();
    if ((ln & 15) == 0) masses[wave() * kOwn + ln / 16] = s;
    __syncthreads();
}

// Weights of a part when kParts of them hold n.
__device__ __forceinline__ uint32_t part_of(uint32_t n)
{
    constexpr uint32_t kStep = kWave * kN;
    return ((n + kParts - 1) / kParts + kStep - 1) / kStep * kStep;
}

// The walk, of one wave: where it stands between two masses.
struct Walk {
    int v, kids_at, cnt, refused;       // node, its next child to look at, accepted rows, refused children
    double c, c_before, W, Q;
    bool pending;                       // c is new, its mass not summed yet

    __device__ __forceinline__ void start()
    {
        c = c_before = 0.0;
        W = Q = 1.0;
        pending = false;
    }
};

constexpr uint32_t kFirst = 1u << 16, kFit = 1u << 17;  // of a node: accepted if tried first; can be tried

// Goes on until a mass is wanted (true) or no child is accepted. The whole numbers
// are scalars: what they come from is the same in all lanes, which the compiler
// does not see everywhere.
template <bool kDraft>
__device__ __forceinline__ bool walk(Walk &s, int n, const uint32_t *node, const int32_t *tok, const float *px,
                                     const float *dx, const float *ux, int32_t *path, int32_t *gone)
{
    const int ln = lane();
    int v = __builtin_amdgcn_readfirstlane(s.v), kids_at = __builtin_amdgcn_readfirstlane(s.kids_at);
    int cnt = __builtin_amdgcn_readfirstlane(s.cnt), refused = __builtin_amdgcn_readfirstlane(s.refused);
    bool wants = false;
    for (;;) {
        int taken = -1;
        for (int k = kids_at & -kWave; k < n; k += kWave) {
            const uint32_t me = k + ln < n ? node[k + ln] : 0u;
            const uint64_t first = __ballot((me & kFirst) != 0);
            const uint32_t up = (me & kFit) && k + ln >= kids_at ? me & 0xffffu : 0xfffeu;
            uint64_t kids = __ballot(up == (uint32_t)v);
            if (refused == 0 && n <= kWave) {
                // As long as first children are accepted, a look at the lanes takes each.
                while (kids != 0 && (first >> (__ffsll((unsigned long long)kids) - 1) & 1)) {
                    v = __ffsll((unsigned long long)kids) - 1;
                    if (ln == 0) path[cnt] = v;
                    ++cnt;
                    kids = __ballot(up == (uint32_t)v);
                }
            }
            while (kids != 0) {
                const int at = __ffsll((unsigned long long)kids) - 1, j = k + at;
                kids &= kids - 1;
                bool yes;
                if (refused == 0) {
                    yes = first >> at & 1;
                } else {
                    const int x = tok[j];
                    bool again = false;
                    for (int i = 0; i < refused; i += kWave) again |= i + ln < refused && gone[i + ln] == x;
                    if (uniform(again)) continue;
                    if constexpr (kDraft) {
                        if (uniform(!(s.Q > 0.0))) continue;
                        if (uniform(s.pending)) {
                            kids_at = j;
                            wants = true;
                            break;
                        }
                        yes = uniform((double)ux[j] * (double)dx[j] * s.W < remains(px[j], dx[j], s.c) * s.Q);
                    } else {
                        yes = uniform((double)ux[j] * s.W < (double)px[j]);
                    }
                }
                if (yes) {
                    taken = j;
                    break;
                }
                if (ln == 0) gone[refused] = tok[j];
                ++refused;
                if constexpr (kDraft) {
                    s.c_before = s.c;
                    s.c += s.W / s.Q;
                    s.Q -= (double)dx[j];
                    s.pending = true;
                } else {
                    s.W -= (double)px[j];
                }
            }
            if (wants || taken >= 0) break;
        }
        if (wants || taken < 0) break;
        v = taken;
        kids_at = v + 1;
        if (ln == 0) path[cnt] = v;
        ++cnt;
        refused = 0;
        s.start();
    }
    s.v = v;
    s.kids_at = kids_at;
    s.cnt = cnt;
    s.refused = refused;
    return wants;
}

template <int kType, bool kDraft>
__global__ __launch_bounds__(kThreads) void k_verify(Args a)
{
    static_assert(kParts == kWave);
    __shared__ uint32_t node[kMost];
    __shared__ int32_t tok[kMost], path[kMost];
    __shared__ float px[kMost], dx[kMost], ux[kMost];
    __shared__ double masses[kParts];
    __shared__ uint32_t wrong;
    __shared__ Refused gone;
    __shared__ int shared_v, shared_cnt, shared_refused;
    __shared__ double shared_c[2];                      // the remainder's c, and the one before
    __shared__ bool more;
    const uint32_t b = blockIdx.x;
    const int tid = (int)threadIdx.x, ln = lane();
    uint32_t s0, s1;
    kv_span(a.q_start, b, a.total, s0, s1);
    const int64_t raw0 = a.q_start[b], raw1 = a.q_start[b + 1];
    bool inval = raw0 < 0 || raw1 < raw0 || raw1 > a.total || (b == 0 && raw0 != 0) ||
                 (b == a.rows - 1 && raw1 != a.total) || s1 - s0 > (uint32_t)kMost;
    const int n = inval ? 0 : (int)(s1 - s0);
    if (tid == 0) wrong = 0;
    if (!kDraft && tid < kBits / 32) gone.bits[tid] = 0;
    __syncthreads();
    if (tid < n) {
        const int64_t row = (int64_t)s0 + tid;
        int p = tid == 0 ? -1 : a.parent[row];
        const int t = a.tokens[row];
        const float u = a.u[row];
        if (p < -1 || p >= tid) {
            if (tid > 0) wrong = 1;                     // every writer writes 1
            p = -1;
        }
        const bool on = p >= 0 && t >= 0 && (uint32_t)t < a.vocab;
        const float pv = on ? number<kType>(a.probs, (int64_t)(s0 + p) * a.probs_row + t) : 0.0f;
        const float dv = kDraft && on ? number<kType>(a.draft, (int64_t)(s0 + p) * a.draft_row + t) : 0.0f;
        const bool fit = kDraft ? dv > 0.0f : pv > 0.0f;
        const bool first = kDraft ? (double)u * (double)dv < (double)pv : u < pv;
        node[tid] = ((uint32_t)p & 0xffffu) | (first ? kFirst : 0u) | (fit ? kFit : 0u);
        tok[tid] = t;
        px[tid] = pv;
        dx[tid] = dv;
        ux[tid] = u;
        if (tid == 0) path[0] = 0;
    }
    __syncthreads();
    inval = inval || wrong;
    if (inval || n == 0) {
        for (uint32_t i = tid; i < s1 - s0; i += kThreads) a.path[s0 + i] = -1;
        if (tid == 0) {
            a.count[b] = 0;
            a.status[b] = inval ? DMADESC_KV_EINVAL : DMADESC_KV_OK;
            a.next[b] = -1;
        }
        return;
    }

    // (The walk's state field by field: copied whole, the compiler puts it into LDS by
    // thread number, which it reads from the dispatch packet in host memory: 3 to 7 us.)
    Walk s;
    s.v = s.refused = 0;
    s.kids_at = s.cnt = 1;
    s.start();
    auto row_of = [&](int refused) {                    // the row that the walk has come to
        const int64_t row = (int64_t)s0 + __builtin_amdgcn_readfirstlane(shared_v);
        return Row{row * a.probs_row, row * a.draft_row, lane_value(shared_c[0], 0), refused};
    };
    for (;;) {
        if (__builtin_amdgcn_readfirstlane(wave()) == 0) {
            const bool wants = walk<kDraft>(s, n, node, tok, px, dx, ux, path, gone.token);
            if (ln == 0) {
                shared_v = s.v;
                shared_cnt = s.cnt;
                shared_refused = s.refused;
                shared_c[0] = s.c;
                shared_c[1] = s.c_before;
                more = wants;
            }
            if (!kDraft && !wants)
                for (int i = ln; i < s.refused; i += kWave) {
                    const uint32_t bit = (uint32_t)gone.token[i] / kN & (kBits - 1);
                    atomicOr(&gone.bits[bit / 32], 1u << (bit & 31));
                }
        }
        __syncthreads();
        if (!kDraft || !__builtin_amdgcn_readfirstlane(more)) break;
        const Row w = row_of(0);
        sum_parts<kType, kDraft>(a, w, gone, 0, a.vocab, part_of(a.vocab), masses);
        const double mass = lane_value(running_sum(masses[ln]), kWave - 1);
        s.pending = false;
        if (uniform(mass > 0.0)) s.W = mass;
        else s.c = s.c_before;                          // nothing would be left: it stays as it was
    }
    const int refused = __builtin_amdgcn_readfirstlane(shared_refused);
    for (int i = tid; i < n; i += kThreads) a.path[s0 + i] = i < shared_cnt ? path[i] : -1;
    if (tid == 0) {
        a.count[b] = shared_cnt;
        a.status[b] = DMADESC_KV_OK;
    }

    // The next token, from what remains of row v.
    Row w = row_of(refused);
    uint32_t from = 0, end = a.vocab, part = part_of(end);
    double aim = 0.0, ahead = 0.0;                      // u times the mass; mass before `from`
    bool whole = true, past = false;                    // past: no running sum passes the aim, so the last weight
    for (;;) {
        double mine = 0.0;                              // of the lane's 64th of [from, end)
        if (part > 1) {
            if (whole || part * kParts > kLongPart) {   // by the whole workgroup, until a part is short
                sum_parts<kType, kDraft>(a, w, gone, from, end, part, masses);
                mine = masses[ln];
            } else {
                const uint32_t at = from + (uint32_t)ln * part, to = at + part < end ? at + part : end;
                if (a.vocab < (uint32_t)kN) {
                    for (uint32_t k = at; k < to; ++k) mine += weight<kType, kDraft>(a, w, gone, k);
                } else {                                // (from and part are multiples of kN)
#pragma unroll 4
                    for (uint32_t k = at; k < to; k += kN) {
                        Run<kType, kDraft> run;
                        const uint32_t place = k < a.vocab - kN ? k : a.vocab - kN;
                        run.load(a, w, place);
                        mine += run.template sum<true>(w, gone, place, true, k, to);
                    }
                }
            }
        } else if (from + ln < end) {
            mine = weight<kType, kDraft>(a, w, gone, from + ln);
        }
        const double upto = running_sum(mine);
        if (whole) {
            const double all = lane_value(upto, kWave - 1);
            if (uniform(!(all > 0.0))) {
                if (w.refused < refused || refused == 0) {      // nothing to draw from
                    if (tid == 0) a.next[b] = -1;
                    return;
                }
                w.c = lane_value(shared_c[1], 0);                      // nothing remains: the remainder before
                w.refused = refused - 1;
                continue;
            }
            aim = (double)ux[0] * all;
            whole = false;
        }
        // The first part whose running sum passes the aim. Where none does (the sums'
        // last bits, or u of 1 or more, or NaN) it is the last with any mass.
        const uint64_t some = __ballot(mine > 0.0), pass = __ballot(mine > 0.0 && ahead + upto > aim);
        past = past || pass == 0;
        const int k = past ? 63 - __clzll((unsigned long long)some) : __ffsll((unsigned long long)pass) - 1;
        ahead += lane_value(upto - mine, k);
        from += (uint32_t)k * part;
        if (part == 1) break;
        end = from + part < end ? from + part : end;
        if (part > kLongPart) {
            part = part_of(part);
        } else {                                        // one wave finishes
            if (__builtin_amdgcn_readfirstlane(wave()) != 0) return;
            part = part > kWave ? (part + kWave - 1) / kWave : 1;
        }
    }
    if (tid == 0) a.next[b] = (int32_t)from;
}

template <int kType>
void launch_type(const Args &a, hipStream_t s)
{
    if (a.draft) k_verify<kType, true><<<a.rows, kThreads, 0, s>>>(a);
    else k_verify<kType, false><<<a.rows, kThreads, 0, s>>>(a);
}

}  // namespace

hipError_t launch_verify(const VerifyArgs &v, hipStream_t s)
{
    const Args a{v.probs, v.draft, v.probs_row, v.draft_row, (uint32_t)v.vocab, v.tokens, v.parent, v.q_start, v.rows,
                 (uint32_t)v.total, v.u, v.path, v.count, v.next, v.status};
    if (v.type == DMADESC_KV_BF16) launch_type<DMADESC_KV_BF16>(a, s);
    else if (v.type == DMADESC_KV_FP16) launch_type<DMADESC_KV_FP16>(a, s);
    else launch_type<DMADESC_KV_FP32>(a, s);
    return hipGetLastError();
}

}  // namespace dd
