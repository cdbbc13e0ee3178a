"""Keeping accepted tokens and reading the paged 8-bit cache back on the GPU, against
their definitions in 64 bits: codes, scales and values exactly."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import memory_dma_descriptor_amd as dd
from tests import kv_cases as kc
from tests import tree_cases as tc
from tests.gpu_cases import say
from tests.test_gpu_kv import TYPES, i32, make_table, random_pool, starts

pytestmark = pytest.mark.gpu


def appended_pool(rng, lens, table, npages, heads, tokens, dim, codes, spread):
    """A pool that append wrote (so that scales hold their blocks), blocks far apart in size."""
    pool = np.zeros((npages, kc.page_bytes(heads, tokens, dim)), np.uint8)
    total = int(sum(lens))
    def values():
        x = rng.standard_normal((total, heads, dim))
        return x * np.exp2(rng.integers(-spread, spread + 1, (total, 1, 1)))
    return kc.append(pool, table, lens, starts(lens), values(), values(), tokens, codes)


def check_keep(lens, news, paths, heads, tokens, dim, codes, seed=0, spread=3, edit=None):
    rng = np.random.default_rng(seed)
    npages = sum(kc.columns(n, tokens) for n in lens) + 2
    table = make_table(rng, lens, tokens, npages)
    pool = appended_pool(rng, lens, table, npages, heads, tokens, dim, codes, spread)
    if edit:
        edit(pool, table)
    want = tc.keep(pool, table, lens, paths, news, heads, dim, tokens, codes)
    flat = np.full(sum(news), -1, np.int32)
    for s0, p in zip(starts(news), paths):
        flat[s0:s0 + len(p)] = p
    dev = torch.from_numpy(pool).cuda()
    r = dd.kv_keep(i32(flat), i32([len(p) for p in paths]), i32(starts(news)), dev, i32(table), i32(lens), heads,
                   tokens, dim, codes=codes)
    assert r["keep"].tolist() == [l - n + len(p) for l, n, p in zip(lens, news, paths)]
    assert tc.same_codes(dev.cpu().numpy(), want, heads, tokens, dim, codes)


def some_paths(rng, news):
    return [sorted(rng.choice(n, rng.integers(1, n + 1), replace=False).tolist()) if n else [] for n in news]


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("dim,heads,tokens", [(64, 3, 16), (128, 2, 32), (256, 1, 64), (128, 5, 128), (64, 1, 1024)])
def test_keep(codes, dim, heads, tokens):
    say(f"keep {codes} {dim} {heads} {tokens}")
    rng = np.random.default_rng(dim)
    news = [1, 16, 0, 33, 7, 64, 20, 5]
    lens = [1, 20, 30, 33, 100, 70, 35, 21]
    check_keep(lens, news, some_paths(rng, news), heads, tokens, dim, codes)
    check_keep(lens, news, [[0]] + [[n - 1] if n else [] for n in news[1:]], heads, tokens, dim, codes, seed=1)


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
def test_keep_long_paths(codes):
    rng = np.random.default_rng(5)
    news = [512, 300, 512]
    paths = some_paths(rng, news)
    paths[0] = list(range(1, 512))                     # all but the first: every token moves by one
    check_keep([515, 333, 512], news, paths, 1, 16, 64, codes)


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
def test_keep_leaves_what_does_not_move(codes):
    # Whole paths and empty ones: nothing is written, whatever the blocks hold.
    check_keep([40, 25, 16], [17, 9, 16], [list(range(17)), [], list(range(5))], 2, 16, 64, codes)
    # The first ones stand, the rest moves.
    check_keep([40, 90], [17, 60], [[0, 1, 2, 3, 9], list(range(30)) + [40, 41, 59]], 2, 16, 64, codes, seed=2)


@pytest.mark.parametrize("spread", [0, 20])
def test_keep_blocks_of_very_different_scales(spread):
    rng = np.random.default_rng(6)
    news = [40, 60, 100]
    for codes in (kc.E4M3, kc.INT8):
        check_keep([50, 60, 130], news, some_paths(rng, news), 2, 16, 64, codes, seed=spread, spread=spread)


def test_keep_zeros_and_nan_codes():
    def edit(pool, table):
        k, v, ks, vs = kc.split_page(pool, 1, 16, 64)
        k[table[0, 1], 0, 3, 7] = 0x7f
        v[table[0, 1], 0, 0, 9, 5] = 0xff
        k[table[0, 2]] = 0                              # a page of zeros, its scales the least
        v[table[0, 2]] = 0
        ks[table[0, 2]] = vs[table[0, 2]] = 2.0 ** -64
    check_keep([60], [55], [[0, 14, 16, 30, 31, 35, 40]], 1, 16, 64, kc.E4M3, edit=edit)
    check_keep([60], [55], [[30, 31, 32]], 1, 16, 64, kc.E4M3, edit=edit)


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_keep_values_past_the_range_of_float32(codes, dim):
    """Scales up to 2^127: code times scale is past float32, and the least scale that
    holds it is still a number. Among blocks of ordinary scales and earlier tokens."""
    for seed in range(3):
        rng = np.random.default_rng(seed)
        def edit(pool, table):
            for s in kc.split_page(pool, 2, 32, dim)[2:]:
                far = rng.random(s.shape) < (0.3, 0.7, 1.0)[seed]
                s[far] = np.exp2(rng.integers(110, 128, s.shape))[far]
        news = [40, 60, 100, 9]
        check_keep([50, 63, 130, 30], news, some_paths(rng, news), 2, 32, dim, codes, seed=seed, edit=edit)


@pytest.mark.parametrize("codes", [dd.KV_E4M3, dd.KV_INT8])
def test_keep_what_append_wrote_of_the_largest_numbers(codes):
    """float32's largest numbers go to a code whose value is past them (256 x 2^120 in
    e4m3); moved beside small ones they are what they were."""
    heads, tokens, dim, n = 1, 16, 64, 40
    top = float(np.finfo(np.float32).max)
    k = torch.full((n, heads, dim), 1.0, device="cuda")
    k[20:] = top
    k[20:, :, ::2] = -top
    pool = torch.zeros((3, dd.kv_page_bytes(heads, tokens, dim)), dtype=torch.uint8, device="cuda")
    table, lens = i32([[2, 0, 1]]), i32([n])
    dd.kv_append(k, k, i32([0, n]), pool, table, lens, tokens, codes=codes)
    host = pool.cpu().numpy()
    want = tc.keep(host, np.array([[2, 0, 1]]), [n], [[0, 1, 25, 39]], [n], heads, dim, tokens, codes)
    dd.kv_keep(i32([0, 1, 25, 39] + [-1] * 36), i32([4]), i32([0, n]), pool, table, lens, heads, tokens, dim, codes=codes)
    assert tc.same_codes(pool.cpu().numpy(), want, heads, tokens, dim, codes)
    r = dd.kv_read(None, i32([0, 4]), 4, pool, table, i32([4]), heads, tokens, dim, codes=codes, dtype=torch.float32)
    assert (r["k"][2:].abs() > 3e38).all() and (r["v"][2:].abs() > 3e38).all()


def test_keep_refuses():
    heads, tokens, dim = 2, 16, 64
    rng = np.random.default_rng(1)
    pool = torch.from_numpy(random_pool(rng, 8, heads, tokens, dim, kc.INT8)).cuda()
    before = pool.clone()
    def run(path, count, start, lens, table):
        with pytest.raises(dd.DmadescRefused) as e:
            dd.kv_keep(i32(path), i32(count), i32(start), pool, i32(table), i32(lens), heads, tokens, dim,
                       codes=dd.KV_INT8)
        torch.cuda.synchronize()
        assert torch.equal(pool, before)
        assert e.value.out["keep"].tolist() == lens
        return e.value.out["status"].tolist()
    good = [[0, 1, 2]]
    for path in ([3, 1, 2, 4], [0, 0, 1, 2], [-1, 1, 2, 3], [1, 2, 3, 10], [1, 2, 3, 1 << 30]):
        assert run(path + [0] * 6, [4], [0, 10], [20], good) == [dd.KV_EINVAL]
    path = [1, 3, 5] + [-1] * 7
    assert run(path, [11], [0, 10], [20], good) == [dd.KV_EINVAL]
    assert run(path, [-1], [0, 10], [20], good) == [dd.KV_EINVAL]
    assert run(path, [3], [0, 10], [9], good) == [dd.KV_EINVAL]            # more new tokens than length
    assert run(path, [3], [0, 10], [49], good) == [dd.KV_EINVAL]           # past the table
    assert run(path, [3], [0, 10], [-1], good) == [dd.KV_EINVAL]
    assert run(path, [3], [0, 11], [20], good) == [dd.KV_EINVAL]
    assert run(path, [3], [0, 10], [20], [[0, 8, 2]]) == [dd.KV_EPAGE]
    assert run(path, [3], [0, 10], [20], [[-1, 1, 2]]) == [dd.KV_EPAGE]
    long = list(range(1, 514))
    assert run(long, [500], [0, 513], [600], [list(np.arange(40) % 8)]) == [dd.KV_EINVAL]


# -------------------------------------------------------------------- read ---

def check_read(lens, firsts, counts, heads, tokens, dim, codes, dtype, exps=(-7, -4), seed=0, strided=False,
               check=True):
    rng = np.random.default_rng(seed)
    npages = sum(kc.columns(n, tokens) for n in lens) + 2
    pool = random_pool(rng, npages, heads, tokens, dim, codes, exps)
    table = make_table(rng, lens, tokens, npages)
    total = sum(counts)
    want = [np.zeros((total, heads, dim)) for _ in range(2)]
    for b, (f, n, s0) in enumerate(zip(firsts, counts, starts(counts))):
        kv = kc.request_cache(pool, table[b], lens[b], heads, tokens, dim, codes)
        lo, hi = max(f, 0), min(f + n, lens[b])
        for w, x in zip(want, kv):
            if hi > lo:
                w[s0 + lo - f:s0 + hi - f] = x[lo:hi]
    want = [torch.from_numpy(w).to(TYPES[dtype]) for w in want]
    out = None
    if strided:
        both = torch.full((total + 2, 2 * heads + 1, dim + 8), 5.0, dtype=TYPES[dtype], device="cuda")
        out = dict(k=both[1:-1, :heads, :dim], v=both[1:-1, heads:2 * heads, :dim])
    f = None if not any(firsts) else i32(firsts)
    r = dd.kv_read(f, i32(starts(counts)), total, torch.from_numpy(pool).cuda(), i32(table), i32(lens), heads, tokens,
                   dim, codes=codes, dtype=TYPES[dtype], out=out, check=check)
    for x, w in zip((r["k"], r["v"]), want):
        assert x.dtype == w.dtype and torch.equal(torch.nan_to_num(x.cpu().double(), nan=1e9, posinf=1e300, neginf=-1e300),
                                                  torch.nan_to_num(w.double(), nan=1e9, posinf=1e300, neginf=-1e300))
    if strided:                                         # nothing else was touched
        both[1:-1, :2 * heads, :dim] = 5
        assert (both == 5).all()


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("dim,heads,tokens", [(64, 3, 16), (128, 2, 32), (256, 1, 64), (128, 5, 128), (64, 1, 1024)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_read(codes, dim, heads, tokens, dtype):
    lens = [1, 17, 33, 5, 16, 100, 47, 64]
    check_read(lens, [0] * 8, lens, heads, tokens, dim, codes, dtype)
    check_read(lens, [0, 3, 16, 5, 1, 37, 15, 63], [1, 14, 17, 0, 15, 40, 32, 1], heads, tokens, dim, codes, dtype,
               strided=True, seed=1)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_read_scales_at_their_ends(dtype):
    for codes in (kc.E4M3, kc.INT8):
        check_read([40, 20], [3, 0], [30, 20], 1, 16, 64, codes, dtype, exps=(-64, 118))


def test_read_every_code():
    pool = np.zeros((2, kc.page_bytes(1, 16, 64)), np.uint8)
    pool[1, :1024] = np.arange(1024) % 256
    pool[1, 1024:2048] = np.arange(1024) // 4
    pool[1, 2048:2056] = np.ones(2, np.float32).view(np.uint8)
    for codes in (kc.E4M3, kc.INT8):
        k, v = kc.request_cache(pool, np.array([1]), 16, 1, 16, 64, codes)
        for dt in TYPES.values():
            r = dd.kv_read(None, i32([0, 16]), 16, torch.from_numpy(pool).cuda(), i32([[1]]), i32([16]), 1, 16, 64,
                           codes=codes, dtype=dt)
            for x, w in zip((r["k"], r["v"]), (k, v)):
                assert torch.equal(torch.nan_to_num(x.double().cpu(), nan=1e9), torch.nan_to_num(torch.from_numpy(w).to(dt).double(), nan=1e9))


def test_read_outside_reads_zero():
    check_read([20, 33, 0], [-5, 30, 0], [40, 20, 3], 2, 16, 64, kc.INT8, "bf16", check=False)
    check_read([20, 33], [1 << 30, -(1 << 31)], [40, 20], 2, 16, 64, kc.E4M3, "fp32", check=False)
    heads, tokens, dim = 2, 16, 64
    rng = np.random.default_rng(1)
    pool = torch.from_numpy(random_pool(rng, 6, heads, tokens, dim, kc.INT8)).cuda()
    for bad in (6, -1, 1 << 30):
        args = (i32([0, 30]), 30, pool, i32([[0, bad, 2]]), i32([40]), heads, tokens, dim)
        with pytest.raises(dd.DmadescRefused) as e:
            dd.kv_read(None, *args, codes=dd.KV_INT8)
        assert e.value.out["status"].tolist() == [dd.KV_EPAGE]
        r = dd.kv_read(None, *args, codes=dd.KV_INT8, check=False)
        assert (r["k"][16:] == 0).all() and (r["v"][16:] == 0).all() and (r["k"][:16] != 0).any()
    for first, start, lens in (([-1], [0, 30], [40]), ([11], [0, 30], [40]), ([0], [0, 30], [49]), ([0], [1, 30], [40]),
                               ([0], [0, 29], [40]), ([0], [0, 30], [-1])):
        st = dd.kv_read_check(i32(first), i32(start), 30, pool, i32([[0, 1, 2]]), i32(lens), heads, tokens, dim)
        assert st.tolist() == [dd.KV_EINVAL]


def test_read_what_append_wrote():
    heads, tokens, dim, n = 3, 32, 128, 77
    pool = torch.zeros((4, dd.kv_page_bytes(heads, tokens, dim)), dtype=torch.uint8, device="cuda")
    k, v = (torch.randn((n, heads, dim), device="cuda") for _ in range(2))
    for codes, half in ((dd.KV_E4M3, 2.0 ** -4), (dd.KV_INT8, None)):
        dd.kv_append(k, v, i32([0, n]), pool, i32([[2, 0, 1]]), i32([n]), tokens, codes=codes)
        r = dd.kv_read(None, i32([0, n]), n, pool, i32([[2, 0, 1]]), i32([n]), heads, tokens, dim, codes=codes,
                       dtype=torch.float32)
        for x, y in ((k, r["k"]), (v, r["v"])):
            top = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -n % 16)).view(-1, 16, heads, dim).abs().amax((1, 3))
            top = top.repeat_interleave(16, 0)[:n, :, None]
            # A scale is under twice the least that holds its block: half a step of a
            # code is x 2^-4 (e4m3; its least codes 2^-10 of 448) or of 127 steps half a one.
            most = torch.maximum(x.abs() * 2.0 ** -4, top * 2 / 448 * 2.0 ** -10) if half else top * 2 / 127 / 2
            assert ((x - y).abs() <= most).all()
