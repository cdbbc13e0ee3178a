"""Decoding steps with drafted trees as they are used: reserve, append, attend along
the trees, verify, keep, cut, read; every part against its definition, captured in
a graph, and on another stream."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import memory_dma_descriptor_amd as dd
from tests import kv_cases as kc
from tests import tree_cases as tc
from tests.gpu_cases import say
from tests.test_gpu_kv import i32, make_table, random_pool, starts

pytestmark = pytest.mark.gpu

KV, HEADS, DIM, PAGE, VOCAB = 2, 4, 64, 16, 501


class Step:
    """The cache and one step's inputs; the trees are the same in every step."""

    def __init__(self, seed=0, codes=kc.E4M3):
        rng = np.random.default_rng(seed)
        self.codes = codes
        self.news = [7, 1, 20, 12]
        self.parents = [tc.random_tree(rng, n, 3) for n in self.news]
        self.lens0 = rng.integers(1, 60, 4).astype(np.int32)
        npages = 64
        pool = random_pool(rng, npages, KV, PAGE, DIM, codes)
        table = make_table(rng, self.lens0, PAGE, npages, 14)
        refs = np.zeros(npages, np.int32)
        refs[table[table >= 0]] = 1
        self.pool, self.refs, self.table, self.lens = (torch.from_numpy(x).cuda()
                                                       for x in (pool, refs, table, self.lens0))
        self.slots, self.n_new, self.start = i32(range(4)), i32(self.news), i32(starts(self.news))
        self.parent = i32([x for p in self.parents for x in p])
        g = torch.Generator(device="cuda").manual_seed(seed)
        total = sum(self.news)
        self.k, self.v = (torch.randn((total, KV, DIM), generator=g, device="cuda").bfloat16() for _ in range(2))
        self.q = torch.randn((total, HEADS, DIM), generator=g, device="cuda").bfloat16()
        self.head = torch.randn((HEADS * DIM, VOCAB), generator=g, device="cuda")
        self.draft = torch.softmax(torch.randn((total, VOCAB), generator=g, device="cuda") * 2, 1)
        self.tokens = self.draft.topk(3, 1).indices[torch.arange(total, device="cuda"),
                                                    torch.arange(total, device="cuda") % 3].to(torch.int32)
        self.u = torch.rand(total, generator=g, device="cuda")
        self.read_start = i32([0, 16, 16, 32, 40])

    def run(self, stream=None):
        kw = dict(stream=stream, check=False)
        state = (self.refs, self.table, self.lens)
        r = dd.kv_reserve(*state, self.slots, self.n_new, PAGE, **kw)
        dd.kv_copy_pages(self.pool, r["src"], r["dst"], stream=stream)
        dd.kv_append(self.k, self.v, self.start, self.pool, self.table, self.lens, PAGE, codes=self.codes, **kw)
        o = dd.kv_attend_tree(self.q, self.start, self.parent, self.pool, self.table, self.lens, KV, PAGE,
                              codes=self.codes, **kw)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            # The target's row: near the draft's, so that some drafts are accepted.
            probs = torch.softmax(o["out"].view(len(self.q), -1).float() @ self.head * 0.1
                                  + self.draft.log(), 1)
        ver = dd.verify_drafts(probs, self.tokens, self.parent, self.start, self.u, draft=self.draft, **kw)
        kept = dd.kv_keep(ver["path"], ver["count"], self.start, self.pool, self.table, self.lens, KV, PAGE, DIM,
                          codes=self.codes, **kw)
        dd.kv_free(*state, self.slots, PAGE, keep=kept["keep"], **kw)
        got = dd.kv_read(None, self.read_start, 40, self.pool, self.table, self.lens, KV, PAGE, DIM,
                         codes=self.codes, **kw)
        return dict(o, **ver, keep=kept["keep"], probs=probs, **got)

    def state(self):
        return self.pool, self.refs, self.table, self.lens


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
def test_steps_against_their_definitions(codes):
    s = Step(codes=codes)
    moved = 0
    for step in range(4):
        say(f"step {step}")
        before = [x.cpu().numpy().copy() for x in s.state()]
        s.u.uniform_(0, 1, generator=torch.Generator(device="cuda").manual_seed(step))
        out = s.run()
        pool, refs, table, lens = before
        kc.reserve(refs, table, lens, range(4), s.news, PAGE)
        pool = kc.append(pool, table, lens, starts(s.news), s.k.double().cpu().numpy(), s.v.double().cpu().numpy(),
                         PAGE, codes)
        ref = tc.attend(pool, table, lens, s.parents, s.q.double().cpu().numpy(), KV, PAGE, codes)
        bound, _ = kc.attend_bounds(ref, DIM, int(max(lens)), s.q.dtype)
        assert (np.abs(out["out"].double().cpu().numpy() - ref["out"]) <= bound).all()
        paths, nexts, p, d = [], [], out["probs"].double().cpu().numpy(), s.draft.double().cpu().numpy()
        for b, (s0, n) in enumerate(zip(starts(s.news), s.news)):
            at = slice(s0, s0 + n)
            path, nxt = tc.verify(s.parents[b], s.tokens[at].tolist(), s.u[at].double().tolist(), p[at], d[at])
            paths.append(path)
            nexts.append(nxt)
        assert out["next"].tolist() == nexts and out["count"].tolist() == [len(x) for x in paths]
        moved += sum(x != list(range(len(x))) for x in paths)
        pool = tc.keep(pool, table, lens, paths, s.news, KV, DIM, PAGE, codes)
        keep = [int(l) - n + len(x) for l, n, x in zip(lens, s.news, paths)]
        assert out["keep"].tolist() == keep
        kc.free(refs, table, lens, range(4), PAGE, keep)
        assert tc.same_codes(s.pool.cpu().numpy(), pool, KV, PAGE, DIM, codes)
        for a, b in zip(s.state()[1:], (refs, table, lens)):
            assert np.array_equal(a.cpu().numpy(), b)
    assert moved > 0


def test_step_in_a_graph():
    s, e = Step(), Step()
    w = Step()
    w.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = s.run()
    for replay in range(4):
        say(f"replay {replay}")
        for x in (s, e):
            x.u.uniform_(0, 1, generator=torch.Generator(device="cuda").manual_seed(replay))
            x.k.add_(0.25)
        want = e.run()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(e.state(), s.state()):
            assert torch.equal(a, b)
        for name in want:
            assert torch.equal(want[name], got[name]), name
        assert float(torch.ones(1000, device="cuda").sum()) == 1000


def test_step_on_another_stream():
    e, s = Step(1), Step(1)
    want = e.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = s.run(side)
    junk = [torch.full((1 << 16,), 7, dtype=torch.uint8, device="cuda") for _ in range(50)]
    side.synchronize()
    assert junk
    for name in want:
        assert torch.equal(want[name], got[name]), name
    for a, b in zip(e.state(), s.state()):
        assert torch.equal(a, b)


def test_two_verifications_at_once():
    rng = np.random.default_rng(0)
    def one(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        p = torch.softmax(torch.randn((40, 30001), generator=g, device="cuda") * 3, 1)
        d = torch.softmax(p.log() + torch.randn(p.shape, generator=g, device="cuda") * 0.5, 1)
        tok = torch.multinomial(d, 1, generator=g)[:, 0].roll(1).to(torch.int32)
        return (p, tok, i32([-1 if j % 8 == 0 else j % 8 - 1 for j in range(40)]), i32(range(0, 41, 8)),
                torch.rand(40, generator=g, device="cuda")), dict(draft=d)
    jobs = [one(int(x)) for x in rng.integers(0, 1 << 30, 2)]
    want = [dd.verify_drafts(*a, **k) for a, k in jobs]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in jobs]
    for _ in range(20):
        got = [dd.verify_drafts(*a, **k, stream=s, check=False) for (a, k), s in zip(jobs, sides)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for name in w:
            assert torch.equal(w[name], g[name]), name


def test_pages_past_4_gib():
    """The same pages low in one pool and past 4 GiB of another: the same results."""
    kv, tokens, dim, nodes = 2, 128, 128, 90
    rng = np.random.default_rng(4)
    low = torch.from_numpy(random_pool(rng, 12, kv, tokens, dim, kc.E4M3)).cuda()
    size = low.shape[1]
    at = (1 << 32) // size - 5                          # some pages before the border, most behind it
    high = torch.empty((at + 12, size), dtype=torch.uint8, device="cuda")
    high[at:] = low
    table = rng.permutation(12)[:10].reshape(2, 5).astype(np.int32)
    lens, start = i32([600, 580]), i32([0, nodes, nodes + 7])
    parent = i32(tc.random_tree(rng, nodes) + tc.random_tree(rng, 7))
    q = torch.randn((nodes + 7, 4, dim), device="cuda").bfloat16()
    path = torch.full((nodes + 7,), -1, dtype=torch.int32, device="cuda")
    path[:30] = i32(np.sort(rng.permutation(nodes)[:30]))
    path[nodes:nodes + 2] = i32([0, 6])
    def step(pool, table):
        o = dd.kv_attend_tree(q, start, parent, pool, i32(table), lens, kv, tokens)
        few = dd.kv_attend_tree(q[nodes:], i32([0, 0, 7]), parent[nodes:], pool, i32(table), lens, kv, tokens)
        dd.kv_keep(path, i32([30, 2]), start, pool, i32(table), lens, kv, tokens, dim)
        got = dd.kv_read(None, i32([0, 600, 1180]), 1180, pool, i32(table), lens, kv, tokens, dim)
        return o["out"], few["out"], got["k"], got["v"]
    for a, b in zip(step(low, table), step(high, table + at)):
        assert torch.equal(a, b)
    assert torch.equal(low, high[at:])


def test_rows_past_32_bits():
    """Rows of probs and draft more than 2^32 numbers from the first."""
    vocab, rows = 1000, 5
    wide = torch.empty((rows, 1 << 30), dtype=torch.bfloat16, device="cuda")[:, 7:7 + vocab]
    g = torch.Generator(device="cuda").manual_seed(0)
    p = torch.softmax(torch.randn((rows, vocab), generator=g, device="cuda") * 3, 1).bfloat16()
    d = torch.softmax(p.float().log() + torch.randn(p.shape, generator=g, device="cuda"), 1).bfloat16()
    args = (i32([0] + d.float().argmax(1).tolist()[:4]), i32([-1, 0, 1, 2, 3]), i32([0, rows]))
    for seed in range(6):
        u = torch.rand(rows, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")
        want = dd.verify_drafts(p, *args, u, draft=d)
        far = dd.verify_drafts(wide.copy_(p), *args, u, draft=d)
        both = dd.verify_drafts(p, *args, u, draft=wide.copy_(d))
        for name in want:
            assert torch.equal(want[name], far[name]) and torch.equal(want[name], both[name]), name
