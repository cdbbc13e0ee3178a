"""Verification of drafted tokens on the GPU against its rule in 64 bits
(tests/tree_cases.py): whole numbers, which have to be equal."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import memory_dma_descriptor_amd as dd
from tests import tree_cases as tc
from tests.gpu_cases import say
from tests.test_gpu_kv import TYPES, i32, starts

pytestmark = pytest.mark.gpu


def rows_of(rng, total, vocab, peak, dtype):
    x = rng.standard_normal((total, vocab)) * peak
    x = np.exp(x - x.max(1, keepdims=True))
    return torch.from_numpy(x / x.sum(1, keepdims=True)).to(TYPES[dtype])


def drafts(rng, parents, draft, vocab):
    """Tokens of every row, drawn from the draft's rows: siblings without replacement."""
    out, s0 = [], 0
    for parent in parents:
        tok = [0] * len(parent)
        for v in range(len(parent)):
            kids = [j for j in range(1, len(parent)) if parent[j] == v]
            if kids:
                d = tc.sound(draft[s0 + v])
                some = np.nonzero(d)[0]
                got = rng.choice(some, min(len(kids), len(some)), replace=False, p=d[some] / d[some].sum())
                for j, x in zip(kids, list(got) + [0] * len(kids)):
                    tok[j] = int(x)
        out += tok
        s0 += len(parent)
    return np.array(out, np.int32)


def check(parents, tokens, u, probs, draft, strided=False):
    total, vocab = probs.shape
    news = [len(p) for p in parents]
    p64, d64 = probs.double().numpy(), None if draft is None else draft.double().numpy()
    want_path, want_count, want_next, s0 = [], [], [], 0
    u32 = np.asarray(u, np.float32)
    for parent, n in zip(parents, news):
        at = slice(s0, s0 + n)
        path, nxt = tc.verify(parent, tokens[at].tolist(), u32[at].astype(np.float64), p64[at],
                              None if d64 is None else d64[at])
        want_path += path + [-1] * (n - len(path))
        want_count.append(len(path))
        want_next.append(nxt)
        s0 += n

    def dev(x):
        if x is None or not strided:
            return None if x is None else x.cuda()
        wide = torch.full((total, vocab + 3), 7.0, dtype=x.dtype, device="cuda")     # odd rows, no alignment
        wide[:, 1:vocab + 1] = x.cuda()
        return wide[:, 1:vocab + 1]
    r = dd.verify_drafts(dev(probs), i32(tokens), i32([x for p in parents for x in p]), i32(starts(news)),
                         torch.from_numpy(u32).cuda(), draft=dev(draft))
    say(f"  accepted {np.mean(want_count):.2f} rows on the average")
    assert r["count"].tolist() == want_count
    assert r["path"].tolist() == want_path
    assert r["next"].tolist() == want_next
    return r


def trees(seed, sizes, branch):
    rng = np.random.default_rng(seed)
    return [tc.random_tree(rng, n, branch) for n in sizes]


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("vocab", [1, 5, 300, 4095, 4096, 4097, 8193, 50257])
def test_verify(dtype, certain, vocab):
    rng = np.random.default_rng(vocab)
    sizes = [1, 6, 0, 13, 2, 30, 3, 9] if vocab < 10000 else [6, 1, 9]
    parents = trees(vocab, sizes, 3)
    total = sum(sizes)
    for peak, near in ((1.0, 0.5), (3.0, 0.3)):
        probs = rows_of(rng, total, vocab, peak, dtype)
        x = torch.log(probs.double().clamp(min=1e-30)) + torch.from_numpy(rng.standard_normal((total, vocab))) * near
        draft = torch.softmax(x, 1).to(TYPES[dtype])
        tokens = drafts(rng, parents, draft.double().numpy(), vocab)
        check(parents, tokens, rng.random(total), probs, None if certain else draft, strided=peak == 3.0)


@pytest.mark.parametrize("certain", [False, True])
def test_verify_many_requests(certain):
    rng = np.random.default_rng(1)
    sizes = rng.integers(0, 9, 700)
    parents = trees(1, sizes, 2)
    total, vocab = int(sizes.sum()), 50
    probs, draft = rows_of(rng, total, vocab, 2.0, "fp32"), rows_of(rng, total, vocab, 2.0, "fp32")
    tokens = drafts(rng, parents, draft.double().numpy(), vocab)
    check(parents, tokens, rng.random(total), probs, None if certain else draft)


@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("nodes", [64, 65, 129, 512])
@pytest.mark.parametrize("shape", ["chain", "star", "tree"])
def test_verify_large_trees(certain, nodes, shape):
    rng = np.random.default_rng(nodes)
    parent = {"chain": [j - 1 for j in range(nodes)], "star": [-1] + [0] * (nodes - 1),
              "tree": tc.random_tree(rng, nodes, 3, 20)}[shape]
    vocab = 1200
    probs = rows_of(rng, nodes, vocab, 0.3, "fp32")
    draft = probs if shape == "chain" else rows_of(rng, nodes, vocab, 0.3, "fp32")
    tokens = drafts(rng, [parent], draft.double().numpy(), vocab)
    u = rng.random(nodes)
    if shape == "chain":
        u[nodes - 3] = 1.0                             # accepted up to there: equal rows refuse nothing below 1
        if certain:
            u[:] = 0
    check([parent], tokens, u, probs, None if certain else draft)


def test_verify_borders():
    """Numbers with few bits, so that tests stand exactly on their borders."""
    p = torch.tensor([[.5, .25, .25, 0]] * 3)
    d = torch.tensor([[.25, .25, .5, 0]] * 3)
    root = [-1, 0, 0]
    for u, want in (([0, .5, .99], [0, 2]), ([0, .49, 0], [0, 1]), ([0, 0, 0], [0, 1])):
        r = check([root], np.array([0, 2, 0], np.int32), u, p, d)
        assert r["path"].tolist()[:2] == want
    for u0 in (0, .25, .5, .74999, .75, .9999, 1.0, 1.5, float("nan"), -1.0):     # the draw's borders, and past them
        for q in (p, torch.tensor([[0, .25, 0, .75]] * 3), torch.tensor([[0, 0, 1.0, 0]] * 3)):
            check([[-1]], np.zeros(1, np.int32), [u0], q[:1], None)
            check([[-1, 0]], np.array([0, 1], np.int32), [u0, 1.0], q[:2], None)
    for x in (-1, 4, 1 << 30, -(1 << 31)):                  # a token outside the vocabulary
        check([root], np.array([0, x, 0], np.int32), [.3, 0, .1], p, d)
        check([root], np.array([0, x, 0], np.int32), [.3, 0, .1], p, None)
    check([root], np.array([9, 2, 2], np.int32), [.3, .99, 0], p, d)         # the same token twice
    check([root], np.array([9, 1, 1], np.int32), [.3, .99, 0], p, None)


def test_verify_rows_out_of_the_ordinary():
    inf, nan = float("inf"), float("nan")
    rows = [[0] * 6, [nan] * 6, [inf, 0.25, 0, .25, -1, .25], [-.5, .5, .5, 0, 0, 0], [0, 0, 0, 0, 0, 1.0],
            [1e-45, 0, 0, 1e-40, 0, 0], [.1, .2, .3, .1, .2, .1], [3e38, 3e38, 1, 0, 0, 3e38]]
    for r in rows:
        for s in rows:
            p, d = (torch.tensor([x] * 3, dtype=torch.float32) for x in (r, s))
            for tokens in ([0, 1, 3], [0, 5, 0], [0, 2, 4]):
                for u in ([.5, .3, .7], [0, .999, .999], [.999, 0, 0]):
                    if r == rows[-1] or s == rows[-1]:       # sums of 10^38: one test of each kind only
                        tokens = [0, 2, 2]
                    check([[-1, 0, 0]], np.array(tokens, np.int32), u, p, None)
                    if not (r == rows[-1] and s == rows[-1]):
                        check([[-1, 0]], np.array(tokens[:2], np.int32), u[:2], p[:2], d[:2])
    # Equal rows, and a refusal all the same (u of 1): nothing remains, the row itself stands.
    p = torch.tensor([rows[6]] * 2, dtype=torch.float32)
    check([[-1, 0]], np.array([0, 2], np.int32), [.6, 1.0], p, p)
    # Certain, and nothing but the refused token has any mass.
    p = torch.tensor([rows[4]] * 2, dtype=torch.float32)
    check([[-1, 0]], np.array([0, 5], np.int32), [.6, 1.0], p, None)


@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("dtype,bits,inf", [("fp32", (0x7fc00000, 0x7f800001, 0x7fa00000, 0x7fffffff), 0x7f800000),
                                            ("bf16", (0x7fc0, 0x7f81, 0x7fbf, 0x7fff), 0x7f80),
                                            ("fp16", (0x7e00, 0x7c01, 0x7dff, 0x7fff), 0x7c00)])
def test_verify_every_nan_counts_as_zero(dtype, bits, inf, certain):
    """Quiet and signalling NaN of both signs, in the target's row and in the draft's, at
    a drafted token and elsewhere; vocabularies below a load's four numbers and above."""
    whole = {"fp32": torch.int32, "bf16": torch.int16, "fp16": torch.int16}[dtype]
    sign = 1 << (31 if dtype == "fp32" else 15)
    size = 2 * sign
    for nan in [x | s for x in bits for s in (0, sign)] + [inf | sign]:
        for vocab, token, at in ((3, 1, 1), (3, 0, 2), (6, 2, 2), (6, 2, 5), (300, 7, 7), (300, 7, 255)):
            for spoil in ("p",) if certain else ("p", "d", "pd"):
                p, d = (torch.full((2, vocab), 1 / vocab).to(TYPES[dtype]) for _ in range(2))
                for name, x in (("p", p), ("d", d)):
                    if name in spoil:
                        x.view(whole)[0, at] = nan - size if nan & sign else nan
                for u in ([.999, .5], [0, 1.0], [.6, 0]):
                    check([[-1, 0]], np.array([0, token], np.int32), u, p, None if certain else d)


@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("vocab", [262144, 262145, 300001, 1000003])
def test_verify_long_rows(vocab, dtype, certain):
    """Rows past 262,144 numbers: parts of more than 4,096, which the workgroup divides
    once more."""
    rng = np.random.default_rng(vocab)
    parents = [[-1, 0, 0, 1], [-1], [-1, 0]]
    probs = rows_of(rng, 7, vocab, 2.0, dtype)
    x = torch.log(probs.double().clamp(min=1e-30)) + torch.from_numpy(rng.standard_normal((7, vocab))) * 0.3
    draft = torch.softmax(x, 1).to(TYPES[dtype])
    tokens = drafts(rng, parents, draft.double().numpy(), vocab)
    for u in (rng.random(7), np.array([.9999, .9, .999, 0, 0, .5, .95])):
        check(parents, tokens, u, probs, None if certain else draft, strided=vocab % 2 == 1)


@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [4097, 16384, 50257])
def test_verify_long_rows_with_numbers_out_of_the_ordinary(vocab, dtype, certain):
    """Rows among whose probabilities are NaN of both kinds, negative numbers, numbers of 2
    and more and infinity, in the middle of a wave's share and at the row's end."""
    whole, snan = {"fp32": (torch.int32, 0x7f800001), "bf16": (torch.int16, 0x7f81), "fp16": (torch.int16, 0x7c01)}[dtype]
    rng = np.random.default_rng(vocab)
    parents = [[-1, 0, 0, 1], [-1, 0], [-1], [-1], [-1]]
    n = sum(len(p) for p in parents)
    for odd in (None, float("nan"), -0.25, 2.5, -0.0, float("inf"), -float("inf")):       # None: a signalling NaN
        probs = rows_of(rng, n, vocab, 2.0, dtype)
        x = torch.log(probs.double().clamp(min=1e-30)) + torch.from_numpy(rng.standard_normal((n, vocab))) * 0.3
        draft = torch.softmax(x, 1).to(TYPES[dtype])
        tokens = drafts(rng, parents, draft.double().numpy(), vocab)
        for rows in (probs,) if certain else (probs, draft):
            for row in range(n - 1):                                                       # the last row is ordinary
                at = rng.integers(0, vocab, 3)
                at[0] = vocab - 1 - row % 2
                if odd is None:
                    rows.view(whole)[row, at] = snan
                else:
                    rows[row, at] = odd
        check(parents, tokens, rng.random(n), probs, None if certain else draft, strided=vocab % 2 == 1)


def test_verify_every_part_of_a_long_row():
    """Equal weights of 2^-20, whose sums are exact: the place is floor(u vocab)."""
    for vocab in (262144, 262145, 524289, 1000003):
        n = 400
        rng = np.random.default_rng(vocab)
        u = rng.random(n).astype(np.float32)
        u[:6] = 0, .5, .25, .75, np.float32(1) - np.float32(2.0 ** -24), 2.0 ** -24
        p = torch.full((1, vocab), 2.0 ** -20, device="cuda").expand(n, vocab)      # one row for all
        r = dd.verify_drafts(p, i32([0] * n), i32([-1] * n), i32(np.arange(n + 1)), torch.from_numpy(u).cuda())
        assert r["next"].tolist() == [int(x) for x in np.floor(u.astype(np.float64) * vocab)]


def test_verify_refuses():
    p = torch.rand((6, 40), device="cuda")
    u = torch.rand(6, device="cuda")
    tok = i32([1] * 6)
    for start, parent, bad in (([0, 3, 6], [-1, 0, 2, -1, 0, 0], [0]), ([0, 3, 6], [-1, 0, 0, -1, 0, 2], [1]),
                               ([0, 3, 6], [-1, -2, 0, -1, 0, 0], [0]), ([0, 4, 3], [-1, 0, 0, 0, 0, 0], [1]),
                               ([1, 3, 6], [0, 0, 0, -1, 0, 0], [0]), ([0, 3, 5], [-1, 0, 0, -1, 0, 0], [1])):
        with pytest.raises(dd.DmadescRefused) as e:
            dd.verify_drafts(p, tok, i32(parent), i32(start), u)
        out = e.value.out
        assert [i for i, s in enumerate(out["status"].tolist()) if s] == bad
        for i in bad:
            assert out["count"].tolist()[i] == 0 and out["next"].tolist()[i] == -1
    big = torch.rand((513, 8), device="cuda")
    r = dd.verify_drafts(big, i32([0] * 513), i32([-1] * 513), i32([0, 513]), torch.rand(513, device="cuda"), check=False)
    assert r["status"].tolist() == [dd.KV_EINVAL] and r["path"].tolist() == [-1] * 513
    # Row 0's parent and token are not looked at.
    r = dd.verify_drafts(p, i32([99, 1, 1, -5, 1, 1]), i32([7, 0, 0, -9, 0, 0]), i32([0, 3, 6]), u)
    assert (r["count"] >= 1).all()
    # Requests without rows, and none at all.
    r = dd.verify_drafts(p[:0], tok[:0], tok[:0], i32([0, 0, 0]), u[:0])
    assert r["count"].tolist() == [0, 0] and r["next"].tolist() == [-1, -1]
    r = dd.verify_drafts(p[:0], tok[:0], tok[:0], i32([0]), u[:0])
    assert r["count"].numel() == 0
    with pytest.raises(TypeError):
        dd.verify_drafts(p, tok, tok, i32([0, 6]), u, draft=p.half())
    with pytest.raises(ValueError):
        dd.verify_drafts(p.T, tok, tok, i32([0, 6]), u)


@pytest.mark.parametrize("certain", [False, True])
def test_verify_samples_the_target(certain):
    """The first token after the root follows the target whatever the draft: 100,000
    seeded requests, every token within 5 deviations."""
    rng = np.random.default_rng(4)
    n, vocab = 100000, 7
    p, d = rng.dirichlet(np.ones(vocab)), rng.dirichlet(np.ones(vocab))
    p32 = torch.tensor(p, dtype=torch.float32, device="cuda").expand(4, vocab).repeat(n, 1)
    d32 = torch.tensor(d, dtype=torch.float32, device="cuda").expand(4, vocab).repeat(n, 1)
    g = torch.Generator(device="cuda").manual_seed(5)
    gum = torch.log(d32[::4]) - torch.log(-torch.log(torch.rand((n, vocab), generator=g, device="cuda")))
    kids = gum.topk(3, 1).indices if not certain else torch.tensor([5, 2, 3], device="cuda").expand(n, 3)
    tokens = torch.cat([torch.zeros((n, 1), dtype=torch.int64, device="cuda"), kids], 1).to(torch.int32)
    parent = torch.tensor([-1, 0, 0, 0], dtype=torch.int32, device="cuda").repeat(n)
    start = torch.arange(n + 1, dtype=torch.int32, device="cuda") * 4
    u = torch.rand(4 * n, generator=g, device="cuda")
    r = dd.verify_drafts(p32, tokens.flatten(), parent, start, u, draft=None if certain else d32)
    path = r["path"].view(n, 4)
    first = torch.where(r["count"] > 1, tokens.gather(1, path[:, 1:2].clamp(min=0).long())[:, 0], r["next"])
    seen = torch.bincount(first.long(), minlength=vocab).double().cpu().numpy() / n
    assert (np.abs(seen - p) <= 5 * np.sqrt(p * (1 - p) / n)).all(), (seen, p)
