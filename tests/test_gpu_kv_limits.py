"""The cache's attention at the ends of its ranges, on the GPU against the
definition in 64 bits: block scales and score factors far apart, in the kernel
of few rows, the kernel of many rows and the join of split requests."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import memory_dma_descriptor_amd as dd
from tests import kv_cases as kc
from tests.gpu_cases import say
from tests.test_gpu_kv import i32, make_table, random_pool, starts

pytestmark = pytest.mark.gpu


def reference(pool, table, lens, news, q, kv, tokens, codes, causal, scale):
    """kc.attend's outputs, and for the bound: `top`, the row's largest probability
    times V scale, and `codes`, the sum of |V code| over the tokens it sees."""
    total, heads, dim = q.shape
    group = heads // kv
    zero = lambda *s: np.zeros((total, heads) + s)                           # noqa: E731
    r = dict(out=zero(dim), mass=zero(dim), codes=zero(dim), top=zero(), size=zero(),
             lse=zero() - math.inf)
    at = 0
    for b, (length, n) in enumerate(zip(lens, news)):
        if length and n:
            k, v = kc.request_cache(pool, table[b], length, kv, tokens, dim, codes)
            _, vc, _, vs = kc.split_page(np.ascontiguousarray(pool[table[b, :kc.columns(length, tokens)]]),
                                         kv, tokens, dim)
            vc = np.abs(kc.TABLE[codes][vc]).transpose(0, 2, 4, 1, 3).reshape(-1, kv, dim)[:length]
            vs = np.repeat(vs.astype(np.float64).transpose(0, 2, 1), kc.BLOCK, axis=1)
            vs = vs.reshape(-1, kv)[:length]
            limit = (length - n + np.arange(n)) if causal else np.full(n, length - 1)
            seen = np.arange(length) <= limit[:, None]
            some = seen.any(1)
            for h in range(heads):
                g, rows = h // group, np.arange(at, at + n)[some]
                see = seen[some]
                s = np.where(see, q[rows, h] @ k[:, g].T * scale, -math.inf)
                top = s.max(1)
                lse = top + np.log(np.exp(s - top[:, None]).sum(1))
                p = np.exp(s - lse[:, None])
                r["out"][rows, h], r["mass"][rows, h] = p @ v[:, g], p @ np.abs(v[:, g])
                r["codes"][rows, h] = see @ vc[:, g]
                r["top"][rows, h] = (p * vs[:, g]).max(1)
                size = np.abs(q[rows, h]) @ np.abs(k[:, g]).T * abs(scale)
                r["size"][rows, h] = np.where(see, size, 0).max(1)
                r["lse"][rows, h] = lse
        at += n
    return r


def bounds(ref, dim, longest, dtype, exps):
    """kc.attend_bounds with what far scales add. A probability is rounded in f16
    relative to the row's largest probability times V scale, which stands at 2^13
    or more there: half of f16's least step, 2^-25, is 2^-38 of it for each unit
    of a code. The exponentials' arguments hold scores and exponents together: at
    most eight roundings of half a step of (|score| + |exponent|) each, where 16
    more cover the offsets 13, 15 and 32."""
    out, lse = kc.attend_bounds(ref, dim, longest, dtype)
    arg = 8 * 2.0 ** -24 * (ref["size"] + max(abs(e) for e in exps) + 16)
    err = arg[..., None] * ref["mass"] + 2.0 ** -38 * ref["top"][..., None] * ref["codes"]
    return out + err * (1 + torch.finfo(dtype).eps / 2), lse + arg


def check(pool, table, lens, news, q, kv, tokens, codes, exps, causal=True, scale=None):
    """q: numpy float32 [total, heads, dim], cast to bf16 (whose range holds the values)."""
    dim = q.shape[2]
    q = torch.from_numpy(q).bfloat16()
    ref = reference(pool, table, lens, news, q.double().numpy(), kv, tokens, codes, causal,
                    1 / math.sqrt(dim) if scale is None else scale)
    args = (q.cuda(), i32(starts(news)), torch.from_numpy(pool).cuda(), i32(table), i32(lens), kv, tokens)
    r = dd.kv_attend(*args, codes=codes, causal=causal, scale=scale)
    out, lse = r["out"].double().cpu().numpy(), r["lse"].double().cpu().numpy()
    bound, lse_bound = bounds(ref, dim, max(lens), q.dtype, exps)
    empty = np.isneginf(ref["lse"])
    assert np.isfinite(out).all() and np.array_equal(np.isneginf(lse), empty)
    assert (out[empty] == 0).all()
    d = np.abs(out - ref["out"]) / bound
    with np.errstate(invalid="ignore"):
        dl = np.abs(lse - ref["lse"]) / lse_bound
    say(f"  worst out {d.max():.3f}, lse {np.nanmax(dl, initial=0):.3f} of the bound")
    assert d.max() <= 1 and np.nanmax(dl, initial=0) <= 1
    again = dd.kv_attend(*args, codes=codes, causal=causal, scale=scale)
    assert torch.equal(again["out"], r["out"]) and torch.equal(again["lse"], r["lse"])


def far_cache(rng, lens, kv, tokens, dim, codes, far, gap, first_far, spare=1, extra=1):
    """A cache whose tokens before first_far have zero values (scale 2^-64, as
    kv_append writes them) and score 0 under one_hot queries, and whose later ones
    have values under 2^far and score -gap."""
    npages = sum(kc.columns(n, tokens) for n in lens) + spare
    pool = random_pool(rng, npages, kv, tokens, dim, codes)
    table = make_table(rng, lens, tokens, npages, extra)
    kcodes, vcodes, ks, vs = kc.split_page(pool, kv, tokens, dim)
    ks[:], kcodes[:], vs[:] = 1.0, 0, 2.0 ** far
    for b, n in enumerate(lens):
        for t in range(n):
            p = table[b, t // tokens]
            if t < first_far:
                vcodes[p, :, t % tokens // 16, :, t % 16] = 0
                vs[p, :, t % tokens // 16] = 2.0 ** -64
            else:
                kcodes[p, :, t % tokens, 0] = kc.nearest([-float(gap)], codes)[0]
    return pool, table


def one_hot(total, heads, dim):
    q = np.zeros((total, heads, dim), np.float32)
    q[:, :, 0] = 1
    return q


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("far", [-20, 50, 80, 119])
@pytest.mark.parametrize("gap", [0, 40, 88, 112])
def test_few_rows_zero_values_beside_large_ones(codes, causal, far, gap):
    # Rows that see the zero values alone, with the large ones hidden in the same
    # tile, and rows that see both, in one tile and in several.
    say(f"few far {codes} {causal} 2^{far} gap {gap}")
    rng = np.random.default_rng(1000 + far + gap)
    for dim, lens, news, first in ((64, [36], [8], 32), (128, [400, 52], [3, 6], 48), (256, [67], [5], 64)):
        pool, table = far_cache(rng, lens, 2, 16, dim, codes, far, gap, first)
        check(pool, table, lens, news, one_hot(sum(news), 4, dim), 2, 16, codes, (-64, far), causal, 1.0)


def test_few_rows_that_see_nothing_beside_large_values():
    rng = np.random.default_rng(0)
    pool, table = far_cache(rng, [5, 20], 1, 16, 64, kc.INT8, 119, 0, 0)
    check(pool, table, [5, 20], [9, 4], one_hot(13, 2, 64), 1, 16, kc.INT8, (-64, 119), True, 1.0)


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("far,gap", [(50, 0), (50, 88), (61, 0), (80, 0), (119, 0), (119, 40), (119, 112)])
def test_join_of_far_scales(codes, far, gap):
    # The zero values in one piece of a split request, the large ones in another,
    # whose weight alone is below f32's range.
    say(f"join far {codes} 2^{far} gap {gap}")
    rng = np.random.default_rng(1000 + far + gap)
    for lens, first in (([6000, 30], 3008), ([6000, 30], 5920)):
        pool, table = far_cache(rng, lens, 1, 64, 64, codes, far, gap, first)
        check(pool, table, lens, [1, 1], one_hot(2, 2, 64), 1, 64, codes, (-64, far), True, 1.0)


def test_join_of_the_largest_values():
    # Partial outputs that are all near f32's largest number.
    rng = np.random.default_rng(1)
    pool, table = far_cache(rng, [6000], 1, 64, 64, kc.INT8, 120, 0, 0)
    _, vcodes, _, _ = kc.split_page(pool, 1, 64, 64)
    vcodes[:] = 127
    check(pool, table, [6000], [1], one_hot(1, 2, 64), 1, 64, kc.INT8, (120, 120), True, 1.0)


# Requests of this size, two heads on one, run in the kernel of many rows: the
# first pair with its cache cut into pieces, the second whole.
MANY = [([700, 500], [90, 120], 2), ([200, 150], [90, 120], 1)]


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("far,gap", [(-20, 40), (50, 0), (50, 88), (61, 0), (63, 0), (80, 0), (119, 0),
                                     (119, 40), (119, 112)])
def test_many_rows_zero_values_beside_large_ones(codes, causal, far, gap):
    say(f"many far {codes} {causal} 2^{far} gap {gap}")
    rng = np.random.default_rng(1000 + far + gap)
    for (lens, news, extra), dim in zip(MANY, (64, 128)):
        pool, table = far_cache(rng, lens, 1, 64, dim, codes, far, gap, 128, extra=extra)
        check(pool, table, lens, news, one_hot(sum(news), 2, dim), 1, 64, codes, (-64, far), causal, 1.0)


def test_many_rows_of_the_largest_values():
    rng = np.random.default_rng(1)
    for lens, news, extra in MANY:
        pool, table = far_cache(rng, lens, 1, 64, 64, kc.INT8, 120, 0, 0, extra=extra)
        _, vcodes, _, _ = kc.split_page(pool, 1, 64, 64)
        vcodes[:] = 127
        check(pool, table, lens, news, one_hot(sum(news), 2, 64), 1, 64, kc.INT8, (120, 120), True, 1.0)


def random_case(rng, lens, news, tokens, dim, codes, exps, q_scale, extra=1):
    npages = sum(kc.columns(n, tokens) for n in lens) + 1
    pool = random_pool(rng, npages, 1, tokens, dim, codes, exps)
    table = make_table(rng, lens, tokens, npages, extra)
    return pool, table, rng.standard_normal((sum(news), 2, dim)).astype(np.float32) * np.float32(q_scale)


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("lens,news,extra", MANY + [([700, 500], [3, 2], 2)])
def test_keys_and_factors_at_their_ends(codes, lens, news, extra):
    # K scale times factor past f32's largest number, under queries of zero; and
    # below its least normal one, under queries that would make the difference count.
    rng = np.random.default_rng(9)
    pool, table, q = random_case(rng, lens, news, 32, 64, codes, (-7, -4), 0.0, extra)
    ks = kc.split_page(pool, 1, 32, 64)[2]
    ks[:] = 2.0 ** 119
    check(pool, table, lens, news, q, 1, 32, codes, (-7, -4), True, 2.0 ** 10)
    q = q + rng.standard_normal(q.shape).astype(np.float32) * np.float32(2.0 ** 108)
    ks[:] = 2.0 ** -64
    check(pool, table, lens, news, q, 1, 32, codes, (-7, -4), True, 2.0 ** -80)


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("lens,news,extra", MANY + [([700, 500], [3, 2], 2)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scales_far_apart(codes, lens, news, extra, dim):
    # Scales over 2^-64..2^3 under flat and peaked scores, all small, all large;
    # and scales that lie far apart from some tile on only.
    say(f"far apart {codes} {news} {dim}")
    rng = np.random.default_rng(dim)
    for exps, q_scale in (((-64, 3), 0.05), ((-64, 3), 1.0), ((-64, -50), 1.0), ((41, 60), 2.0 ** -56)):
        pool, table, q = random_case(rng, lens, news, 32, dim, codes, exps, q_scale, extra)
        check(pool, table, lens, news, q, 1, 32, codes, exps)
    pool, table, q = random_case(rng, lens, news, 32, dim, codes, (-8, -4), 1.0, extra)
    _, _, ks, vs = kc.split_page(pool, 1, 32, dim)
    for b, n in enumerate(lens):
        for t in range(n * 2 // 3 // 16 * 16, n, 16):
            vs[table[b, t // 32], 0, t % 32 // 16] = 2.0 ** rng.integers(-64, 60)
    check(pool, table, lens, news, q, 1, 32, codes, (-64, 60))


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("lens,news,extra", MANY + [([700, 500], [3, 2], 2)])
@pytest.mark.parametrize("scale", [-0.3, -1e-5, 1e-6, 2.0])
def test_factors(codes, lens, news, extra, scale):
    say(f"factor {scale} {codes} {news}")
    rng = np.random.default_rng(7)
    for dim, causal in ((64, True), (128, False), (256, True)):
        pool, table, q = random_case(rng, lens, news, 32, dim, codes, (-7, -4), 1.0, extra)
        check(pool, table, lens, news, q, 1, 32, codes, (-7, -4), causal, scale)


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("lens,news,extra", MANY + [([700, 500], [3, 2], 2), ([100, 5], [3, 9], 2)])
def test_pages_never_written(codes, lens, news, extra):
    # Scales of 0 under codes of 0, as a zeroed pool has them, alone and beside others.
    rng = np.random.default_rng(11)
    pool, table, q = random_case(rng, lens, news, 32, 64, codes, (-7, -4), 1.0, extra)
    _, vcodes, ks, vs = kc.split_page(pool, 1, 32, 64)
    for p in range(0, len(pool), 3):
        ks[p], vs[p], vcodes[p] = 0, 0, 0
    check(pool, table, lens, news, q, 1, 32, codes, (-127, -4))
    pool[:] = 0
    check(pool, table, lens, news, q, 1, 32, codes, (-127, -4))


def test_reserve_more_pages_than_32_bits_count():
    # 128 slots of one call ask for 2^25 pages each, 2^32 with the single pages of the
    # first and the last one: only the first can have its page.
    rows, width, tokens = 130, 1 << 25, 16
    table = torch.empty((rows, width), dtype=torch.int32, device="cuda")     # 17 GiB, not read
    table[:, 0] = -1
    refs, lens = torch.zeros(300, dtype=torch.int32, device="cuda"), i32([0] * rows)
    news = [16] + [width * tokens] * 128 + [16]
    r = dd.kv_reserve(refs, table, lens, i32(range(rows)), i32(news), tokens, check=False)
    assert r["status"].tolist() == [dd.KV_OK] + [dd.KV_ENOSPC] * 129
    assert lens.tolist() == [16] + [0] * 129 and refs.tolist() == [1] + [0] * 299
    assert table[:, 0].tolist() == [0] + [-1] * 129
    assert (r["src"] == -1).all() and (r["dst"] == -1).all()


def test_reserve_names_bad_pages():
    # A partly filled last page outside the pool; the same entry under a full page
    # and in a row that takes nothing is not looked at.
    state = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (
        [1, 0, 0, 0], [[9, -1], [-1, -1], [-7, -1], [5, -1], [9, -1], [0, -1]], [3, 16, 1, 16, 3, 4])]
    r = dd.kv_reserve(*state, i32(range(6)), i32([1, 1, 40, 1, 0, 13]), 16, check=False)
    assert r["status"].tolist() == [dd.KV_EPAGE, dd.KV_OK, dd.KV_EINVAL, dd.KV_OK, dd.KV_OK, dd.KV_OK]
    assert state[2].tolist() == [3, 17, 1, 17, 3, 17] and state[0].tolist() == [1, 1, 1, 1]
    assert state[1].tolist() == [[9, -1], [-1, 1], [-7, -1], [5, 2], [9, -1], [0, 3]]


def test_strides_of_single_tokens_and_heads():
    # A view of one token, or of one head, may have any stride there.
    rng = np.random.default_rng(3)
    pool, table, _ = random_case(rng, [40], [1], 16, 64, kc.E4M3, (-7, -4), 1.0)
    x = torch.randn((4, 2, 64 + 3), device="cuda").bfloat16()
    one = x.flatten()[:2 * 64].view(1, 2, 64)
    odd = one.as_strided((1, 2, 64), (131, 64, 1))
    head = one.as_strided((2, 1, 64), (64, 5, 1))
    pools, outs = [], []
    for k in (one, odd):
        p = torch.zeros((8, dd.kv_page_bytes(2, 16, 64)), dtype=torch.uint8, device="cuda")
        dd.kv_append(k, k, i32([0, 1]), p, i32([[0, 3, 5]]), i32([40]), 16)
        pools.append(p)
        outs.append(dd.kv_attend(k, i32([0, 1]), p, i32([[0, 3, 5]]), i32([40]), 2, 16)["out"])
    assert pools[0].any() and torch.equal(*pools) and torch.equal(*outs)
    outs = [dd.kv_attend(q, i32([0, 2]), torch.from_numpy(pool).cuda(), i32(table), i32([40]), 1, 16)["out"]
            for q in (one.view(2, 1, 64), head)]
    assert torch.equal(*outs)


def test_attend_without_the_log_sum_exp():
    rng = np.random.default_rng(4)
    pool, table, q = random_case(rng, [700, 500], [3, 2], 32, 64, kc.E4M3, (-7, -4), 1.0)
    q = torch.from_numpy(q).bfloat16().cuda()
    args = (q, i32([0, 3, 5]), torch.from_numpy(pool).cuda(), i32(table), i32([700, 500]), 1, 32)
    want, out = dd.kv_attend(*args), dict(out=torch.empty_like(q))
    assert dd.kv_attend(*args, out=out) is out and torch.equal(out["out"], want["out"])
    many = torch.randn((300, 2, 64), device="cuda").bfloat16()
    args = (many, i32([0, 100, 300])) + args[2:]
    want, out = dd.kv_attend(*args), dict(out=torch.empty_like(many), lse=None)
    assert torch.equal(dd.kv_attend(*args, out=out)["out"], want["out"]) and out["lse"] is None
