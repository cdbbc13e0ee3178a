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
// remainder is p without the tokens refused. Everything is f64: the answers are
// whole numbers, so that what is summed in another order must not change them.
//
// Two launches. The first walks the tree, one workgroup a request: a test reads
// two numbers, all of them gathered beforehand, and a mass W is summed only where
// a child follows a refused one. The second draws the token after the last
// accepted one: workgroups sum 4,096 weights each, and a request's last one to
// finish looks for the place where the running sum passes u W. The sums are added
// in one order whoever is last.
#include "dd_internal.h"
#include "dd_kv.hpp"

namespace dd {
namespace {

constexpr int kMost = (int)DMADESC_TREE_MOST;
constexpr int kWalkThreads = 1024;
constexpr int kDrawThreads = 256;
constexpr int kPer = 16;                                // weights of a thread
constexpr uint32_t kTile = kDrawThreads * kPer;

// What the draw of a request needs from its walk.
struct Draw {
    double c, c_before;         // the remainder, and the one before the last refusal
    int64_t row;                // of probs and draft; -1: nothing is drawn
    int32_t refused, last;      // tokens refused there; the last one of them
    float u;
    uint32_t done;              // workgroups that have summed their part
};

struct Args {
    const void *probs, *draft;
    int64_t probs_row, draft_row;
    uint64_t vocab;
    const int32_t *tokens, *parent, *q_start;
    uint32_t rows, total, tiles;
    const float *u;
    int32_t *path, *count, *next;
    uint8_t *status;
    Draw *draw;                 // [rows]
    int32_t *refused;           // [total] refused tokens of the last node, from q_start on
    double2 *part;              // [rows][tiles] mass of the remainder and of the one before
};

// The numbers of a row; what is not positive and finite counts as 0.
template <int kType>
__device__ __forceinline__ float sound(const void *p, int64_t at)
{
    float x;
    if constexpr (kType == DMADESC_KV_FP32) x = static_cast<const float *>(p)[at];
    else if constexpr (kType == DMADESC_KV_BF16) x = __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[at] << 16);
    else x = (float)static_cast<const _Float16 *>(p)[at];
    return x > 0.0f && x < __builtin_inff() ? x : 0.0f;
}

// kN consecutive numbers from `at` on, zeros past `end`.
template <int kType, int kN>
__device__ __forceinline__ void sound_run(const void *p, int64_t row, uint64_t at, uint64_t end, float (&x)[kN])
{
    if (at + kN <= end) {
        if constexpr (kType == DMADESC_KV_FP32) {
            float y[kN];
            __builtin_memcpy(y, static_cast<const float *>(p) + row + at, sizeof y);
#pragma unroll
            for (int i = 0; i < kN; ++i) x[i] = y[i];
        } else {
            uint16_t y[kN];
            __builtin_memcpy(y, static_cast<const uint16_t *>(p) + row + at, sizeof y);
#pragma unroll
            for (int i = 0; i < kN; ++i)
                x[i] = kType == DMADESC_KV_BF16 ? __uint_as_float((uint32_t)y[i] << 16) : (float)__builtin_bit_cast(_Float16, y[i]);
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = x[i] > 0.0f && x[i] < __builtin_inff() ? x[i] : 0.0f;
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = at + i < end ? sound<kType>(p, row + (int64_t)(at + i)) : 0.0f;
    }
}

template <int kThreads>
__device__ __forceinline__ double block_sum(double v, double *scratch)
{
    v = wave_sum(v);
    __syncthreads();
    if (lane() == 0) scratch[wave()] = v;
    __syncthreads();
    double all = 0.0;
#pragma unroll
    for (int k = 0; k < kThreads / kWave; ++k) all += scratch[k];
    return all;
}

__device__ __forceinline__ double remains(float p, float d, double c)
{
    const double w = (double)p - c * (double)d;
    return w > 0.0 ? w : 0.0;
}

template <int kType, bool kDraft>
__global__ __launch_bounds__(kWalkThreads) void k_verify_walk(Args a)
{
    __shared__ int16_t up[kMost];
    __shared__ int32_t tok[kMost], path[kMost], gone[kMost];
    __shared__ float px[kMost], dx[kMost], ux[kMost];
    __shared__ double scratch[kWalkThreads / kWave];
    __shared__ uint32_t wrong;
    const uint32_t b = blockIdx.x;
    const int tid = (int)threadIdx.x, ln = lane();
    uint32_t s0, s1;
    kv_span(a.q_start, b, a.total, s0, s1);
    const int64_t raw0 = a.q_start[b], raw1 = a.q_start[b + 1];
    bool inval = raw0 < 0 || raw1 < raw0 || raw1 > a.total || (b == 0 && raw0 != 0) ||
                 (b == a.rows - 1 && raw1 != a.total) || s1 - s0 > (uint32_t)kMost;
    const int n = inval ? 0 : (int)(s1 - s0);
    if (tid == 0) wrong = 0;
    __syncthreads();
    if (tid < n) {
        const int64_t row = (int64_t)s0 + tid;
        int p = tid == 0 ? -1 : a.parent[row];
        if (p < -1 || p >= tid) {
            if (tid > 0) wrong = 1;                     // every writer writes 1
            p = -1;
        }
        const int t = a.tokens[row];
        up[tid] = (int16_t)p;
        tok[tid] = t;
        ux[tid] = a.u[row];
        const bool on = p >= 0 && t >= 0 && (uint64_t)t < a.vocab;
        px[tid] = on ? sound<kType>(a.probs, (int64_t)(s0 + p) * a.probs_row + t) : 0.0f;
        dx[tid] = kDraft && on ? sound<kType>(a.draft, (int64_t)(s0 + p) * a.draft_row + t) : 0.0f;
    }
    __syncthreads();
    inval = inval || wrong;

    int cnt = 0;
    int64_t row = -1;
    double c = 0.0, c_before = 0.0;
    int refused = 0, last = -1;
    if (!inval && n > 0) {
        int v = 0;
        if (tid == 0) path[0] = 0;
        cnt = 1;
        for (;;) {                                      // down the tree: a child comes after its parent
            double W = 1.0, Q = 1.0;
            bool pending = false;                       // c is new, its mass not summed yet
            int taken = -1;
            c = c_before = 0.0;
            refused = 0;
            last = -1;
            for (int k = v / kWave * kWave; k < n && taken < 0; k += kWave) {
                uint64_t kids = __ballot(k + ln < n && k + ln > v && up[k + ln < n ? k + ln : 0] == v);
                while (kids && taken < 0) {
                    const int j = k + __ffsll((unsigned long long)kids) - 1;
                    kids &= kids - 1;
                    const int x = tok[j];
                    const double u = ux[j], p = px[j], d = dx[j];
                    bool again = false;
                    for (int i = 0; i < refused; i += kWave) again |= i + ln < refused && gone[i + ln] == x;
                    if (__ballot(again)) continue;
                    if constexpr (kDraft) {
                        if (!(d > 0.0 && Q > 0.0)) continue;
                        if (pending) {                  // the mass that the last refusal left
                            double sum = 0.0;
                            for (uint64_t at = (uint64_t)tid * 4; at < a.vocab; at += kWalkThreads * 4) {
                                float pv[4], dv[4];
                                sound_run<kType>(a.probs, (int64_t)(s0 + v) * a.probs_row, at, a.vocab, pv);
                                sound_run<kType>(a.draft, (int64_t)(s0 + v) * a.draft_row, at, a.vocab, dv);
#pragma unroll
                                for (int i = 0; i < 4; ++i) sum += remains(pv[i], dv[i], c);
                            }
                            sum = block_sum<kWalkThreads>(sum, scratch);
                            pending = false;
                            if (sum > 0.0) W = sum;
                            else c = c_before;          // nothing would be left: it stays as it was
                        }
                        if (u * d * W < remains((float)p, (float)d, c) * Q) {
                            taken = j;
                            break;
                        }
                        c_before = c;
                        c += W / Q;
                        Q -= d;
                        pending = true;
                    } else {
                        if (!(p > 0.0)) continue;
                        if (u * W < p) {
                            taken = j;
                            break;
                        }
                        W -= p;
                        last = x;
                    }
                    __syncthreads();                    // every wave has read the list
                    if (tid == 0) gone[refused] = x;
                    ++refused;
                    __syncthreads();
                }
            }
            row = (int64_t)s0 + v;
            if (taken < 0) break;
            v = taken;
            if (tid == 0) path[cnt] = v;
            ++cnt;
        }
    }
    __syncthreads();
    for (uint32_t i = tid; i < s1 - s0; i += kWalkThreads) a.path[s0 + i] = (int)i < cnt ? path[i] : -1;
    if (!kDraft)
        for (int i = tid; i < refused; i += kWalkThreads) a.refused[s0 + i] = gone[i];
    if (tid == 0) {
        a.count[b] = cnt;
        a.status[b] = inval ? DMADESC_KV_EINVAL : DMADESC_KV_OK;
        if (row < 0) a.next[b] = -1;
        a.draw[b] = Draw{c, c_before, row, refused, last, row < 0 ? 0.0f : ux[0], 0u};
    }
}

// The weights of kN tokens from `at` on: of the remainder and of the one before.
template <int kType, bool kDraft, int kN>
__device__ __forceinline__ void weights(const Args &a, const Draw &w, const int32_t *gone, uint64_t at, uint64_t end,
                                        double (&now)[kN], double (&before)[kN])
{
    float p[kN], d[kN];
    sound_run<kType>(a.probs, w.row * a.probs_row, at, end, p);
    if constexpr (kDraft) {
        sound_run<kType>(a.draft, w.row * a.draft_row, at, end, d);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            now[i] = remains(p[i], d[i], w.c);
            before[i] = remains(p[i], d[i], w.c_before);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) now[i] = before[i] = p[i];
        for (int k = 0; k < w.refused; ++k) {
            const uint64_t x = (uint64_t)gone[k] - at;
#pragma unroll
            for (int i = 0; i < kN; ++i)
                if (x == (uint64_t)i) {
                    now[i] = 0.0;
                    if (gone[k] != w.last) before[i] = 0.0;
                }
        }
    }
}

template <int kType, bool kDraft>
__global__ __launch_bounds__(kDrawThreads) void k_verify_draw(Args a)
{
    __shared__ double scratch[kDrawThreads / kWave];
    __shared__ uint32_t is_last, tile_at, token_at, some_at;
    __shared__ int32_t gone[kDraft ? 1 : kMost];
    const uint32_t b = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
    const int tid = (int)threadIdx.x;
    const Draw w = a.draw[b];
    if (w.row < 0) return;
    if (!kDraft) {
        const uint32_t s0 = (uint32_t)a.q_start[b];
        for (int i = tid; i < w.refused; i += kDrawThreads) gone[i] = a.refused[s0 + i];
        __syncthreads();
    }
    {
        const uint64_t from = (uint64_t)tile * kTile, end = from + kTile < a.vocab ? from + kTile : a.vocab;
        double now = 0.0, before = 0.0;
#pragma unroll
        for (int k = 0; k < kPer / 4; ++k) {
            const uint64_t at = from + (uint64_t)(k * kDrawThreads + tid) * 4;
            if (at >= end) break;
            double x[4], y[4];
            weights<kType, kDraft>(a, w, gone, at, end, x, y);
            now += (x[0] + x[1]) + (x[2] + x[3]);
            before += (y[0] + y[1]) + (y[2] + y[3]);
        }
        now = block_sum<kDrawThreads>(now, scratch);
        before = block_sum<kDrawThreads>(before, scratch);
        if (tid == 0) {
            double2 *const p = &a.part[(uint64_t)b * a.tiles + tile];
            __hip_atomic_store(&p->x, now, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(&p->y, before, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            is_last = __hip_atomic_fetch_add(&a.draw[b].done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                      a.tiles - 1;
            tile_at = token_at = some_at = 0xffffffffu;
        }
        __syncthreads();
        if (!is_last) return;
    }
    // The request's last workgroup: all parts are there. Their running sum first.
    const double2 *const part = a.part + (uint64_t)b * a.tiles;
    auto part_of = [&](uint32_t t, bool use_before) {
        const double *const p = use_before ? &part[t].y : &part[t].x;
        return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    };
    double all = 0.0, all_before = 0.0;
    for (uint32_t t = tid; t < a.tiles; t += kDrawThreads) {
        all += part_of(t, false);
        all_before += part_of(t, true);
    }
    all = block_sum<kDrawThreads>(all, scratch);
    all_before = block_sum<kDrawThreads>(all_before, scratch);
    const bool use_before = !(all > 0.0);                   // nothing is left: the remainder before
    if (use_before) all = all_before;
    if (!(all > 0.0)) {
        if (tid == 0) a.next[b] = -1;
        return;
    }
    const double aim = (double)w.u * all;
    // The first part whose running sum passes the aim; else the last that has any mass.
    double run = 0.0;
    uint32_t some = 0;
    double some_run = 0.0;
    for (uint32_t t0 = 0; t0 < a.tiles && tile_at == 0xffffffffu; t0 += kDrawThreads) {
        const uint32_t t = t0 + tid;
        const double mine = t < a.tiles ? part_of(t, use_before) : 0.0;
        double sum;
        const double at = run + block_excl_scan<kDrawThreads, double>(mine, scratch, &sum);
        if (mine > 0.0 && at + mine > aim) atomicMin(&tile_at, t);
        if (mine > 0.0) {
            some = t;
            some_run = at;
        }
        run += sum;
        __syncthreads();
    }
    // (A u of 1 or more, or NaN, or the sums' last bits: no part passes.)
    const bool none = tile_at == 0xffffffffu;
    if (none) {
        if (tid == 0) tile_at = 0;
        __syncthreads();
        atomicMax(&tile_at, some);
        __syncthreads();
    }
    const uint32_t at_tile = tile_at;
    {
        const uint64_t from = (uint64_t)at_tile * kTile, end = from + kTile < a.vocab ? from + kTile : a.vocab;
        // The mass before this part, in the same order as above.
        double ahead = 0.0;
        for (uint32_t t = tid; t < at_tile; t += kDrawThreads) ahead += part_of(t, use_before);
        ahead = block_sum<kDrawThreads>(ahead, scratch);
        (void)some_run;
        double x[kPer], y[kPer];
        const uint64_t at = from + (uint64_t)tid * kPer;
        if (at < end) {
            weights<kType, kDraft>(a, w, gone, at, end, x, y);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i) x[i] = y[i] = 0.0;
        }
        double mine = 0.0, sum;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (use_before) x[i] = y[i];
            mine += x[i];
        }
        double upto = ahead + block_excl_scan<kDrawThreads, double>(mine, scratch, &sum);
        int hit = -1, any = -1;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            upto += x[i];
            if (x[i] > 0.0) {
                if (hit < 0 && upto > aim) hit = i;
                any = i;
            }
        }
        if (tid == 0) some_at = 0;
        __syncthreads();
        if (hit >= 0 && !none) atomicMin(&token_at, (uint32_t)(tid * kPer + hit));
        if (any >= 0) atomicMax(&some_at, (uint32_t)(tid * kPer + any));
        __syncthreads();
        if (tid == 0) a.next[b] = (int32_t)(from + (token_at != 0xffffffffu ? token_at : some_at));
    }
}

template <int kType, bool kDraft>
void launch_both(const Args &a, hipStream_t s)
{
    k_verify_walk<kType, kDraft><<<a.rows, kWalkThreads, 0, s>>>(a);
    k_verify_draw<kType, kDraft><<<a.rows * a.tiles, kDrawThreads, 0, s>>>(a);
}

template <int kType>
void launch_type(const Args &a, hipStream_t s)
{
    if (a.draft) launch_both<kType, true>(a, s);
    else launch_both<kType, false>(a, s);
}

struct Layout {
    size_t refused, part, bytes;
    uint64_t tiles;
};

Layout layout_of(uint64_t total, uint32_t rows, uint64_t vocab)
{
    Layout l{};
    l.tiles = (vocab + kTile - 1) / kTile;
    l.refused = align256(sizeof(Draw) * (size_t)rows);
    l.part = l.refused + align256(4 * total);
    l.bytes = l.part + align256(sizeof(double2) * (size_t)rows * l.tiles);
    return l;
}

}  // namespace

uint64_t verify_groups(uint32_t rows, uint64_t vocab)
{
    return rows * layout_of(0, rows, vocab).tiles;
}

size_t ws_verify(uint64_t total, uint32_t rows, uint64_t vocab)
{
    return layout_of(total, rows, vocab).bytes;
}

hipError_t launch_verify(const VerifyArgs &v, hipStream_t s)
{
    const Layout l = layout_of(v.total, v.rows, v.vocab);
    uint8_t *const ws = static_cast<uint8_t *>(v.ws);
    Args a{v.probs, v.draft, v.probs_row, v.draft_row, v.vocab, v.tokens, v.parent, v.q_start, v.rows,
           (uint32_t)v.total, (uint32_t)l.tiles, v.u, v.path, v.count, v.next, v.status,
           reinterpret_cast<Draw *>(ws), reinterpret_cast<int32_t *>(ws + l.refused),
           reinterpret_cast<double2 *>(ws + l.part)};
    if (v.type == DMADESC_KV_BF16) launch_type<DMADESC_KV_BF16>(a, s);
    else if (v.type == DMADESC_KV_FP16) launch_type<DMADESC_KV_FP16>(a, s);
    else launch_type<DMADESC_KV_FP32>(a, s);
    return hipGetLastError();
}

}  // namespace dd
