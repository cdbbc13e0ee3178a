"""Attention of trees of drafted tokens over the paged 8-bit cache on the GPU against
its definition in 64 bits (tests/tree_cases.py), within bounds that count its
roundings."""
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


def check_tree(lens, parents, kv, group, tokens, dim, codes, dtype, seed=0, exps=(-7, -4), scale=None,
               spoil=None, extra_width=2, against_chain=False):
    rng = np.random.default_rng(seed)
    news = [len(p) for p in parents]
    npages = sum(kc.columns(n, tokens) for n in lens) + 1
    pool = random_pool(rng, npages, kv, tokens, dim, codes, exps)
    table = make_table(rng, lens, tokens, npages, extra_width)
    total, heads = int(sum(news)), kv * group
    wide = torch.from_numpy(rng.standard_normal((total, heads + 1, dim)).astype(np.float32))
    q = wide.to(TYPES[dtype]).cuda()[:, :heads]         # a strided view
    if spoil:
        spoil(pool, table, q)
    ref = tc.attend(pool, table, lens, parents, q.double().cpu().numpy(), kv, tokens, codes, scale)
    # What lies past the lengths is spoiled only now: it must not count.
    dirty = pool.copy()
    kcodes, vcodes, ks, vs = kc.split_page(dirty, kv, tokens, dim)
    for b, length in enumerate(lens):
        if length % tokens:
            p, at = table[b, length // tokens], length % tokens
            kcodes[p, :, at:] = 0x7f
            for t in range(at, tokens):
                vcodes[p, :, t // 16, :, t % 16] = 0xff
            first = -(-at // 16)
            ks[p, :, first:], vs[p, :, first:] = np.nan, np.inf
    flat = [x for p in parents for x in p]
    args = (i32(starts(news)),)
    cache = (torch.from_numpy(dirty).cuda(), i32(table), i32(lens), kv, tokens)
    full = max(l - n for l, n in zip(lens, news)) >= 0 and all(l >= n for l, n in zip(lens, news))
    r = dd.kv_attend_tree(q, *args, i32(flat), *cache, codes=codes, scale=scale, check=full)
    out, lse = r["out"].double().cpu().numpy(), r["lse"].double().cpu().numpy()
    bound, lse_bound = kc.attend_bounds(ref, dim, max(lens), q.dtype)
    empty = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(lse), empty)
    assert (out[empty] == 0).all()
    assert np.array_equal(np.isnan(out), np.isnan(ref["out"])), "NaN where the definition has it, and nowhere else"
    with np.errstate(invalid="ignore"):
        d = np.abs(out - ref["out"]) / bound
        dl = np.abs(lse - ref["lse"]) / lse_bound
    say(f"  worst out {np.nanmax(d, initial=0):.3f}, lse {np.nanmax(dl, initial=0):.3f} of the bound")
    assert np.nanmax(d, initial=0) <= 1
    assert np.nanmax(dl, initial=0) <= 1
    assert np.array_equal(np.isnan(lse), np.isnan(ref["lse"]))
    if against_chain:                                   # a chain is kv_attend's causal chunk: both within the bound
        c = dd.kv_attend(q, *args, *cache, codes=codes, scale=scale)
        assert (np.abs(c["out"].double().cpu().numpy() - out) <= 2 * bound).all()
        assert (np.abs(c["lse"].double().cpu().numpy() - lse) <= 2 * lse_bound).all()


def some_trees(seed, sizes, branch=4):
    rng = np.random.default_rng(seed)
    return [tc.random_tree(rng, n, branch) for n in sizes]


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "bf16"), (256, "bf16"), (64, "fp16"),
                                       (128, "fp16"), (256, "fp16")])
@pytest.mark.parametrize("nodes,group,tokens", [(1, 4, 64), (7, 1, 16), (5, 7, 32), (16, 4, 64), (33, 3, 16), (40, 2, 128)])
def test_attend_tree(codes, dim, dtype, nodes, group, tokens):
    say(f"tree {codes} {dim} {dtype} nodes {nodes} group {group} tokens {tokens}")
    lens = [nodes, 63 + nodes, 64, 200, 129]
    check_tree(lens, some_trees(nodes, [min(nodes, n) for n in lens]), 2, group, tokens, dim, codes, dtype)


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("nodes", [63, 64, 65, 130, 257, 511, 512])
def test_attend_large_trees(codes, nodes):
    # Trees over several tiles, and their starts at every part of a tile.
    check_tree([nodes + 1, nodes + 50, nodes], some_trees(nodes, [nodes, nodes, nodes], 3), 1, 1, 32, 64, codes, "bf16")


@pytest.mark.parametrize("shape", ["chain", "star", "forest"])
@pytest.mark.parametrize("nodes,group", [(6, 2), (90, 2)])
def test_attend_shapes(shape, nodes, group):
    one = {"chain": [j - 1 for j in range(nodes)], "star": [-1] + [0] * (nodes - 1), "forest": [-1] * nodes}[shape]
    for base in range(40, 72, 5):
        check_tree([base + nodes, nodes], [one, one], 1, group, 16, 64, kc.E4M3, "fp16", seed=base,
                   against_chain=shape == "chain")


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("kv,group,dim,length,nodes", [(1, 4, 64, 6000, 9), (1, 1, 128, 3000, 70),
                                                       (2, 8, 256, 2500, 20), (1, 2, 128, 5000, 12),
                                                       (2, 4, 256, 3100, 16)])
def test_attend_split_over_workgroups(codes, kv, group, dim, length, nodes):
    check_tree([length, 300, length - 77], some_trees(1, [nodes, nodes, 1]), kv, group, 64, dim, codes, "bf16")


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("nodes,group", [(8, 4), (30, 1)])
@pytest.mark.parametrize("requests,length,extra", [(1, 640, 0), (1, 900, 0), (1, 1290, 0), (1, 900, 30), (150, 530, 3)])
def test_attend_by_table_widths(codes, nodes, group, requests, length, extra):
    """About 32 rows a request: by 16 rows with no join over a narrow table that fits at
    once, in pieces of 32 rows past 8 tiles otherwise."""
    lens = [length] + [40 + i % 7 for i in range(requests - 1)]
    check_tree(lens, some_trees(9, [nodes] * requests), 2, group, 64, 64, codes, "bf16", extra_width=extra)


def test_attend_many_requests():
    # More requests than lanes, some without new tokens, some without a cache before them.
    rng = np.random.default_rng(8)
    news = rng.integers(0, 7, 150)
    lens = news + rng.integers(0, 2, 150) * rng.integers(0, 200, 150)
    check_tree([int(x) for x in lens], some_trees(8, news), 1, 3, 16, 64, kc.E4M3, "bf16")


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
def test_attend_a_large_tree_among_single_tokens(codes):
    check_tree([400] + [90] * 39, some_trees(2, [300] + [1] * 39), 1, 4, 32, 64, codes, "bf16")


@pytest.mark.parametrize("nodes", [6, 90])
@pytest.mark.parametrize("length", [100, 1700])
def test_attend_nan_codes(nodes, length):
    """A NaN code reaches the rows that see its token, and no other."""
    def spoil(pool, table, q):
        k, v, _, _ = kc.split_page(pool, 2, 16, 64)
        base = length - nodes
        for at, dim in ((3, 5), (base - 2, 7), (base + 1, 9), (base + nodes // 2, 11), (length - 1, 13)):
            v[table[0, at // 16], 0, 0, dim, at % 16] = 0xff if at % 2 else 0x7f
        k[table[0, (base + 2) // 16], 1, (base + 2) % 16, 3] = 0x7f
    check_tree([length, 40], some_trees(5, [nodes, 3]), 2, 2, 16, 64, kc.E4M3, "bf16", spoil=spoil)


@pytest.mark.parametrize("dim,nodes,group", [(64, 6, 2), (128, 20, 4), (256, 30, 2), (64, 90, 3), (128, 70, 2), (256, 140, 1)])
@pytest.mark.parametrize("share", [0.002, 0.3])
def test_attend_many_nan_codes(dim, nodes, group, share):
    """NaN codes all over a tree's tokens and the tile they begin in: siblings' in one word
    of four tokens, dimensions 16 apart, a row's own and others'."""
    def spoil(pool, table, q):
        v = kc.split_page(pool, 2, 32, dim)[1]
        rng = np.random.default_rng(nodes)
        for b, (length, n) in enumerate(((1500, nodes), (nodes + 9, nodes), (77, 5))):
            for at in range(max(0, length - n - 40), length):
                bad = rng.random((2, dim)) < share
                v[table[b, at // 32], :, at % 32 // 16, :, at % 16][bad] = 0xff if at % 2 else 0x7f
    check_tree([1500, nodes + 9, 77], some_trees(5, [nodes, nodes, 5]), 2, group, 32, dim, kc.E4M3, "bf16",
               spoil=spoil)


@pytest.mark.parametrize("nodes", [5, 100])
def test_attend_more_tokens_than_length(nodes):
    # What dd.kv_tree_check refuses: tokens before the cache's first are not there.
    check_tree([nodes - 3, 1, 0, 80], some_trees(4, [nodes, nodes, 2, 4]), 1, 2, 16, 64, kc.INT8, "bf16")


@pytest.mark.parametrize("scale", [-0.3, 1e-6, 2.0])
def test_attend_factors(scale):
    check_tree([300, 90], some_trees(6, [9, 60]), 1, 3, 32, 128, kc.E4M3, "bf16", scale=scale)


def test_attend_scales_far_apart():
    check_tree([200, 300], some_trees(7, [7, 5]), 1, 2, 16, 64, kc.E4M3, "bf16", exps=(-40, 10))
    check_tree([200, 300], some_trees(7, [70, 80]), 1, 2, 16, 64, kc.INT8, "fp16", exps=(-20, 0))


def test_tree_check_and_bad_arguments_on_the_device():
    kv, tokens, dim = 1, 16, 64
    pool = torch.zeros((8, dd.kv_page_bytes(kv, tokens, dim)), dtype=torch.uint8, device="cuda")
    table = i32([[0, 1, 2], [3, 4, 5], [6, 9, -1]])
    def status(lens, start, parent, table=table):
        return dd.kv_tree_check(i32(start), i32(parent), pool, table, i32(lens), kv, tokens, dim).tolist()
    good = [-1, 0, -1, 0, 1, -1]
    assert status([20, 30, 16], [0, 2, 5, 6], good) == [0, 0, 0]
    assert status([20, 30, 17], [0, 2, 5, 6], good) == [0, 0, dd.KV_EPAGE]
    for r, bad in ((0, [0, 0, -1, 0, 1, -1]), (0, [-1, 1, -1, 0, 1, -1]), (1, [-1, 0, -1, 3, 1, -1]),
                   (1, [-1, 0, -2, 0, 1, -1]), (2, [-1, 0, -1, 0, 1, 1 << 30])):
        assert [i for i, s in enumerate(status([20, 30, 16], [0, 2, 5, 6], bad)) if s] == [r]
        # Unchecked, a bad parent counts as none.
        q = torch.randn((6, 2, dim), device="cuda", dtype=torch.bfloat16)
        mended = list(bad)
        for j, first in enumerate([0, 0, 2, 2, 2, 5]):
            if not -1 <= bad[j] < j - first:
                mended[j] = -1
        args = (pool, table, i32([20, 30, 16]), kv, tokens)
        x = dd.kv_attend_tree(q, i32([0, 2, 5, 6]), i32(bad), *args, check=False)
        y = dd.kv_attend_tree(q, i32([0, 2, 5, 6]), i32(mended), *args)
        assert torch.equal(x["out"], y["out"]) and torch.equal(x["lse"], y["lse"])
        with pytest.raises(dd.DmadescRefused):
            dd.kv_attend_tree(q, i32([0, 2, 5, 6]), i32(bad), *args)
    assert status([1, 30, 16], [0, 2, 5, 6], good) == [dd.KV_EINVAL, 0, 0]         # more tokens than length
    assert status([20, 49, 16], [0, 2, 5, 6], good) == [0, dd.KV_EINVAL, 0]
    assert dd.KV_EINVAL in status([20, 30, 16], [0, 3, 2, 6], good)
    assert dd.KV_EINVAL in status([20, 30, 16], [0, 2, 5, 7], good)
    wide = i32(np.arange(40) % 8).view(1, 40)
    assert status([600], [0, 513], [-1] * 513, wide) == [dd.KV_EINVAL]
    assert status([600], [0, 512], [-1] * 512, wide) == [0]
    # More than TREE_MOST tokens, unchecked: memory-safe, the rows before it as ever.
    q = torch.randn((600, 2, dim), device="cuda", dtype=torch.bfloat16)
    chain = i32(np.arange(600) - 1)
    x = dd.kv_attend_tree(q, i32([0, 600]), chain, pool, wide, i32([600]), kv, tokens, check=False)
    y = dd.kv_attend(q, i32([0, 600]), pool, wide, i32([600]), kv, tokens)
    torch.cuda.synchronize()
    assert torch.equal(x["out"][:512], y["out"][:512])


def test_attend_tree_spares_bad_pages():
    kv, tokens, dim = 1, 16, 64
    rng = np.random.default_rng(1)
    pool = torch.from_numpy(random_pool(rng, 6, kv, tokens, dim, kc.E4M3)).cuda()
    for nodes in (3, 80):
        lens, width = 90, 6
        good = np.array([[0, 1, 2, 3, 4, 5]], np.int32)
        for bad in (6, -1, 1 << 30):
            table = good.copy()
            table[0, 1], table[0, 5] = bad, bad
            q = torch.randn((nodes, 2, dim), device="cuda", dtype=torch.bfloat16)
            tree = i32(tc.random_tree(rng, nodes))
            with pytest.raises(dd.DmadescRefused):
                dd.kv_attend_tree(q, i32([0, nodes]), tree, pool, i32(table), i32([lens]), kv, tokens)
            r = dd.kv_attend_tree(q, i32([0, nodes]), tree, pool, i32(table), i32([lens]), kv, tokens, check=False)
            torch.cuda.synchronize()
            assert r["out"].shape == q.shape and width == table.shape[1]


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("nodes", [3, 80])
def test_attend_tree_bad_pages_touch_no_other_request(nodes, codes):
    """Unchecked, a request with bad pages leaves its neighbours' results and the pool
    as they are, under both kernels."""
    kv, tokens, dim = 2, 16, 64
    rng = np.random.default_rng(nodes)
    pool = torch.from_numpy(random_pool(rng, 18, kv, tokens, dim, codes)).cuda()
    before = pool.clone()
    good = rng.permutation(18).astype(np.int32).reshape(3, 6)
    lens, start = i32([95, 90, 83]), i32([0, nodes, 2 * nodes, 3 * nodes])
    q = torch.randn((3 * nodes, 4, dim), device="cuda", dtype=torch.bfloat16)
    tree = i32(tc.random_tree(rng, nodes) * 3)
    want = dd.kv_attend_tree(q, start, tree, pool, i32(good), lens, kv, tokens, codes=codes)
    for bad in (18, -1, 1 << 30, -(1 << 31)):
        table = good.copy()
        table[1, 1] = table[1, 5] = bad
        r = dd.kv_attend_tree(q, start, tree, pool, i32(table), lens, kv, tokens, codes=codes, check=False)
        for x in ("out", "lse"):
            assert torch.equal(r[x][:nodes], want[x][:nodes]) and torch.equal(r[x][2 * nodes:], want[x][2 * nodes:])
        assert torch.equal(pool, before)


def test_attend_tree_without_the_log_sum_exp_and_into_a_given_output():
    kv, tokens, dim = 2, 16, 128
    rng = np.random.default_rng(2)
    pool = torch.from_numpy(random_pool(rng, 9, kv, tokens, dim, kc.INT8)).cuda()
    table, lens = i32([[0, 1, 2, 3, 4, 5, 6, 7]]), i32([121])
    q = torch.randn((5, 6, dim), device="cuda", dtype=torch.float16)
    tree = i32([-1, 0, 0, 1, 1])
    whole = dd.kv_attend_tree(q, i32([0, 5]), tree, pool, table, lens, kv, tokens, codes=dd.KV_INT8)
    out = torch.full((7, 6, dim), 3.0, device="cuda", dtype=torch.float16)
    r = dd.kv_attend_tree(q, i32([0, 5]), tree, pool, table, lens, kv, tokens, codes=dd.KV_INT8,
                          out=dict(out=out[1:6]))
    assert "lse" not in r and torch.equal(out[1:6], whole["out"])
    assert (out[0] == 3).all() and (out[6] == 3).all()


def test_two_trees_at_once():
    """Calls with workspaces of their own on two streams, and one on a stream that
    meanwhile gets other memory."""
    kv, tokens, dim = 2, 16, 64
    rng = np.random.default_rng(3)
    pool = torch.from_numpy(random_pool(rng, 400, kv, tokens, dim, kc.E4M3)).cuda()
    jobs = []
    for nodes in (12, 90):
        table = i32(rng.permutation(400)[:380].reshape(2, 190))
        q = torch.randn((2 * nodes, 4, dim), device="cuda", dtype=torch.bfloat16)
        parent = i32(tc.random_tree(rng, nodes) + tc.random_tree(rng, nodes))
        jobs.append((q, i32([0, nodes, 2 * nodes]), parent, pool, table, i32([3000, 2500]), kv, tokens))
    want = [dd.kv_attend_tree(*j) for j in jobs]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in jobs]
    for _ in range(20):
        got = [dd.kv_attend_tree(*j, stream=s, check=False) for j, s in zip(jobs, sides)]
        junk = [torch.full((1 << 16,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert junk
    for w, g in zip(want, got):
        assert torch.equal(w["out"], g["out"]) and torch.equal(w["lse"], g["lse"])
