"""Decoding with drafted trees over the paged 8-bit cache as it is measured:
inputs, plain forms and the library's calls.

Four operators: `tree` (attention of a tree of drafted tokens over the cache),
`verify` (which of them the target accepts, and the token after them), `keep`
(bringing the accepted ones together in the cache) and `read` (the cache back
in 16 or 32 bits). Where `own` is false, run() computes them with elementary
torch operations; where it is true, through this package.

A page holds T tokens of H heads of D values: K codes [H][T][D], V codes
[H][T/16][D][16], K scales float32 [H][T/16], V scales [H][T/16], padded to
512 bytes. A scale is a power of two for 16 tokens of one head.

A request's new tokens are a tree in rows of its own: parent[j] is the row,
within the request, of the token before row j, less than j; -1 for the first.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BLOCK = 16                       # tokens under one scale
E_MIN = -64                      # least exponent of a scale
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # One request answering alone with a small tree: the call's latency counts.
        dict(name="tree one request", kind="tree", batch=1, nodes=8, branch=3, depth=4, lo=900, hi=900,
             heads=32, kv=8, dim=128, page=64, codes="e4m3", dtype="bf16"),
        # A serving batch, 16 nodes each, lengths as they come.
        dict(name="tree batch", kind="tree", batch=32, nodes=16, branch=4, depth=5, lo=200, hi=9000,
             heads=32, kv=8, dim=128, page=64, codes="e4m3", dtype="bf16"),
        # Ragged trees, seven heads on one key head, small pages.
        dict(name="tree ragged int8", kind="tree", batch=33, nodes=27, branch=5, depth=7, lo=30, hi=4001,
             heads=28, kv=4, dim=128, page=16, codes="int8", dtype="fp16"),
        # Wide trees over long conversations: the matrix products count.
        dict(name="tree wide", kind="tree", batch=12, nodes=64, branch=8, depth=8, lo=1000, hi=16000,
             heads=32, kv=8, dim=128, page=64, codes="e4m3", dtype="bf16"),
        # One request's tree, its sure drafts from a lookup of earlier text.
        dict(name="verify one request", kind="verify", batch=1, nodes=25, branch=4, depth=6, vocab=32000,
             draft=False, dtype="fp32"),
        # A batch of chains of five drafts, drawn from a draft model.
        dict(name="verify chains", kind="verify", batch=64, nodes=6, branch=1, depth=6, vocab=131072,
             draft=True, dtype="fp32"),
        # Trees drawn from a draft model, rows of an odd length in 16 bits.
        dict(name="verify trees", kind="verify", batch=24, nodes=32, branch=4, depth=6, vocab=50257,
             draft=True, dtype="bf16"),
        # The accepted tokens of a serving batch's trees.
        dict(name="keep step", kind="keep", batch=64, nodes=16, branch=4, depth=6, lo=20, hi=3000, kv=8,
             dim=128, page=64, codes="e4m3"),
        # Long accepted paths of many requests: whole blocks move.
        dict(name="keep long paths", kind="keep", batch=200, nodes=90, branch=2, depth=60, lo=90, hi=1000,
             kv=4, dim=256, page=16, codes="int8"),
        # The last tokens of one request.
        dict(name="read one request", kind="read", batch=1, lo=600, hi=600, most=40, kv=8, dim=128,
             page=64, codes="e4m3", dtype="bf16"),
        # Whole prompts, for a layer that needs them in 16 bits.
        dict(name="read prompts", kind="read", batch=9, lo=800, hi=9000, most=9000, kv=8, dim=128,
             page=64, codes="e4m3", dtype="bf16"),
        # Pieces of many requests that start and end inside blocks, in 32 bits.
        dict(name="read pieces int8", kind="read", batch=70, lo=5, hi=2000, most=700, kv=3, dim=64,
             page=32, codes="int8", dtype="fp32"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    kind = rng.choice(["tree", "tree", "tree", "verify", "verify", "keep", "read"])
    shape = dict(branch=rng.choice([1, 2, 3, 4, 8]), depth=_spread(rng, 2, 20))
    cache = dict(dim=rng.choice([64, 128, 128, 256]), page=rng.choice([16, 32, 64, 128]),
                 codes=rng.choice(["e4m3", "int8"]))
    if kind == "tree":
        kv, group = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 4, 7, 8])
        batch, nodes = _spread(rng, 1, 60), _spread(rng, 1, 130)
        # No more cache, and no more products, than the largest listed case.
        hi = min(30000, 12 * 16000 * 8 * 128 // (batch * kv * cache["dim"]),
                 12 * 64 * 16000 * 32 * 128 // (batch * nodes * kv * group * cache["dim"]))
        hi = max(nodes, _spread(rng, 16, max(16, hi)))
        return dict(kind=kind, batch=batch, nodes=nodes, lo=max(nodes, hi // rng.choice([1, 2, 20])),
                    hi=hi, heads=kv * group, kv=kv, dtype=rng.choice(["bf16", "fp16"]), **shape, **cache)
    if kind == "verify":
        nodes, vocab = _spread(rng, 1, 60), _spread(rng, 300, 150000)
        batch = _spread(rng, 1, max(1, min(128, 50000000 // (nodes * vocab))))
        return dict(kind=kind, batch=batch, nodes=nodes, vocab=vocab, draft=rng.random() < 0.6,
                    dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]), **shape)
    if kind == "keep":
        nodes = _spread(rng, 1, 120)
        return dict(kind=kind, batch=_spread(rng, 1, 200), nodes=nodes, lo=nodes,
                    hi=nodes + _spread(rng, 1, 900), kv=rng.choice([1, 2, 4]), **shape, **cache)
    batch, kv, hi = _spread(rng, 1, 100), rng.choice([1, 2, 3, 8]), _spread(rng, 20, 6000)
    most = max(1, min(hi, 12000 * 8 * 128 // (batch * kv * cache["dim"])))
    return dict(kind=kind, batch=batch, lo=_spread(rng, 1, hi), hi=hi, most=_spread(rng, 1, most), kv=kv,
                dtype=rng.choice(["bf16", "fp16", "fp32"]), **cache)


# --------------------------------------------------------------------------
# sizes that follow from a case
# --------------------------------------------------------------------------

def page_layout(case):
    """(code bytes of K or V, scales of K or V, page bytes)."""
    codes = case["kv"] * case["page"] * case["dim"]
    scales = case["kv"] * (case["page"] // BLOCK)
    return codes, scales, -(-(2 * codes + 8 * scales) // 512) * 512


def lengths(case):
    """Tokens of every request: spread over lo..hi, both reached."""
    n = case["batch"]
    rng = random.Random(n * 1000003 + case["hi"])
    out = [rng.randint(case["lo"], case["hi"]) for _ in range(n)]
    out[0] = case["hi"]
    if n > 1:
        out[-1] = case["lo"]
    return out


def trees(case):
    """Every request's parents: `nodes` rows, fewer for some where there are many,
    at most `branch` children of a row and `depth` rows on a path."""
    rng = random.Random(case["batch"] * 7919 + case["nodes"])
    out = []
    for b in range(case["batch"]):
        n = case["nodes"] if case["nodes"] < 9 or b % 3 == 0 else rng.randint(1, case["nodes"])
        parent, depth, kids = [-1], [1], [0]
        while len(parent) < n:
            can = [j for j in range(len(parent)) if kids[j] < case["branch"] and depth[j] < case["depth"]]
            if not can:
                break                                # the tree is full: fewer rows
            p = can[0] if rng.random() < 0.3 else rng.choice(can[-8:])
            kids[p] += 1
            parent.append(p)
            depth.append(depth[p] + 1)
            kids.append(0)
        out.append(parent)
    return out


def paths(case):
    """Every request's accepted rows, in order: from the first row towards a leaf,
    all of the way or a part."""
    rng = random.Random(case["batch"] * 31 + case["nodes"])
    out = []
    for parent in trees(case):
        at, path = rng.randrange(len(parent) // 2, len(parent)), []
        while at >= 0:
            path.append(at)
            at = parent[at]
        path.reverse()
        out.append(path if rng.random() < 0.7 else path[:rng.randint(1, len(path))])
    return out


def pieces(case):
    """(first token, tokens) that are read of every request."""
    rng = random.Random(case["batch"] * 17 + case["hi"])
    out = []
    for n in lengths(case):
        count = min(n, case["most"])
        if n > case["most"]:
            first = rng.randint(0, n - count)
        else:
            first = 0
        out.append((first, count))
    return out


def _ceil(a, b):
    return -(-a // b)


def _power(e):
    """2^e in float32 (no smaller than 2^-126), from the format."""
    return ((e.clamp(min=-126).to(torch.int32) + 127) << 23).view(torch.float32)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(counts):
    return _i32([0] + counts).cumsum(0).to(torch.int32)


def _cache(case, g):
    """Pages as earlier appends left them: values around zero, a scale that
    follows each block's largest value; every request's pages anywhere."""
    dev = torch.device("cuda")
    codes, scales, page_bytes = page_layout(case)
    lens = lengths(case)
    need = [_ceil(x, case["page"]) for x in lens]
    npages = sum(need) + 8
    pool = torch.zeros((npages, page_bytes), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 27) // (2 * codes))
    for p in range(0, npages, step):
        n = min(step, npages - p)
        x = torch.randn((n, 2 * codes), generator=g, device=dev)
        if case["codes"] == "e4m3":
            x = (x * 110).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            x = (x * 32).round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
        pool[p:p + n, :2 * codes] = x
    e = torch.randint(-7, -4, (npages, 2 * scales), generator=g, device=dev)
    if case["codes"] == "int8":
        e += 2
    pool[:, 2 * codes:2 * codes + 8 * scales] = _power(e).view(torch.uint8)
    order = torch.randperm(npages, generator=g, device=dev).to(torch.int32)
    wide = max(need) + 1
    start = torch.tensor([0] + need, dtype=torch.int64, device=dev).cumsum(0)
    col = torch.arange(wide, device=dev)
    used = col < torch.tensor(need, device=dev)[:, None]
    table = torch.where(used, order[(start[:-1, None] + col).clamp(max=npages - 1)], -1).to(torch.int32)
    return dict(pool=pool, table=table, lens=_i32(lens), rows=len(lens), longest=max(lens))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    s = dict(case=case, rows=case["batch"])
    if kind != "verify":
        s.update(_cache(case, g))
    if kind == "read":
        todo = pieces(case)
        s.update(first=_i32([a for a, _ in todo]), start=_starts([n for _, n in todo]),
                 total=sum(n for _, n in todo), most=max(n for _, n in todo))
        return s

    shape = trees(case)
    s.update(q_start=_starts([len(p) for p in shape]), parent=_i32([x for p in shape for x in p]),
             total=sum(len(p) for p in shape), most=max(len(p) for p in shape))
    if kind == "tree":
        s["q"] = torch.randn((s["total"], case["heads"], case["dim"]), generator=g,
                             device="cuda").to(DTYPES[case["dtype"]])
    elif kind == "keep":
        todo = paths(case)
        flat = [-1] * s["total"]
        at = 0
        for p, tree in zip(todo, shape):
            flat[at:at + len(p)] = p
            at += len(tree)
        s.update(path=_i32(flat), count=_i32([len(p) for p in todo]))
    else:
        _drafts(s, shape, g)
    return s


def _drafts(s, shape, g):
    """The target's and the draft's probabilities after every row, peaked as a
    language model's are and not far from each other, and tokens drawn from the
    draft's row of the parent: siblings one after another, none twice."""
    case = s["case"]
    total, vocab, dt = s["total"], case["vocab"], DTYPES[case["dtype"]]
    kids = max(1, case["branch"])
    probs = torch.empty((total, vocab), dtype=dt, device="cuda")
    draft = torch.empty((total, vocab), dtype=dt, device="cuda")
    best = torch.empty((total, min(kids, vocab)), dtype=torch.int64, device="cuda")
    step = max(1, (1 << 25) // vocab)
    for a in range(0, total, step):
        x = torch.randn((min(step, total - a), vocab), generator=g, device="cuda") * 2.5
        x += 12 * (torch.rand(x.shape, generator=g, device="cuda") < 8 / vocab)
        y = x + torch.randn(x.shape, generator=g, device="cuda") * 0.6
        probs[a:a + step] = torch.softmax(x, 1).to(dt)
        y = torch.softmax(y, 1).to(dt)
        draft[a:a + step] = y
        y = y.float().log()
        if case["draft"]:                            # largest of these: drawn without replacement
            u = torch.rand(y.shape, generator=g, device="cuda").clamp_(min=1e-20)
            y -= torch.log(-torch.log(u).clamp_(min=1e-20))
        best[a:a + step] = y.topk(best.shape[1], 1).indices
    rank, at = [], 0
    row = []
    for p in shape:
        seen = [0] * len(p)
        for x in p:
            row.append(at + max(x, 0))
            rank.append(seen[x] if x >= 0 else 0)
            if x >= 0:
                seen[x] += 1
        at += len(p)
    s["tokens"] = best[torch.tensor(row, device="cuda"), torch.tensor(rank, device="cuda")].to(torch.int32)
    s.update(probs=probs, draft=draft if case["draft"] else None,
             u=torch.rand(total, generator=g, device="cuda"))


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _values(case, codes):
    """Codes (uint8) as the numbers they stand for, in float32."""
    return codes.view(torch.float8_e4m3fn if case["codes"] == "e4m3" else torch.int8).float()


def _views(case, pool):
    """K codes [pages][H][T/16][16][D], V codes [pages][H][T/16][D][16] and the
    scales [pages][H][T/16] as views of the pool."""
    kv, dim, nb = case["kv"], case["dim"], case["page"] // BLOCK
    codes, scales, _ = page_layout(case)
    k = pool[:, :codes].unflatten(1, (kv, nb, BLOCK, dim))
    v = pool[:, codes:2 * codes].unflatten(1, (kv, nb, dim, BLOCK))
    f = pool.view(torch.float32)[:, codes // 2:codes // 2 + 2 * scales].unflatten(1, (2, kv, nb))
    return k, v, f[:, 0], f[:, 1]


def _ancestors(s):
    """[rows][most][most]: whether row i of a request is row j or on its path."""
    q_start = s["q_start"].long()
    j = torch.arange(s["most"], device=q_start.device)
    at = (q_start[:-1, None] + j).clamp(max=s["total"] - 1)
    there = j < (q_start[1:] - q_start[:-1])[:, None]
    parent = torch.where(there, s["parent"][at].long(), -1)
    a = ((parent[:, :, None] == j) | (j[:, None] == j)).float()
    reach = 1
    while reach < s["most"]:                         # paths of twice the length each time
        a = (torch.matmul(a, a) > 0).float()
        reach *= 2
    return a > 0


def _plain_tree(s):
    case = s["case"]
    kv, dim, T, heads = case["kv"], case["dim"], case["page"], case["heads"]
    group, batch, most = heads // kv, s["rows"], s["most"]
    dev = s["q"].device
    lens, q_start = s["lens"].long(), s["q_start"].long()
    pages = s["table"][:, :_ceil(s["longest"], T)].long().clamp(min=0)
    kc, vc, ks, vs = _views(case, s["pool"])
    n = pages.shape[1] * T
    k = _values(case, kc[pages]) * ks[pages][..., None, None]        # B P H nb 16 D
    k = k.permute(0, 2, 1, 3, 4, 5).reshape(batch, kv, n, dim)
    v = _values(case, vc[pages]) * vs[pages][..., None, None]        # B P H nb D 16
    v = v.permute(0, 2, 1, 3, 5, 4).reshape(batch, kv, n, dim)

    base = lens - (q_start[1:] - q_start[:-1])
    j = torch.arange(most, device=dev)
    at = (q_start[:-1, None] + j).clamp(max=s["total"] - 1)
    q = s["q"][at].float().reshape(batch, most, kv, group, dim).permute(0, 2, 3, 1, 4)
    sc = torch.matmul(q.reshape(batch, kv, group * most, dim), k.transpose(2, 3).contiguous())
    sc = sc.reshape(batch, kv, group, most, n) * (1.0 / math.sqrt(dim))
    t = torch.arange(n, device=dev)
    node = t - base[:, None]                                         # of every cached token
    seen = _ancestors(s).gather(2, node.clamp(0, most - 1)[:, None].expand(batch, most, n))
    seen = (seen | (node < 0)[:, None]) & (t < lens[:, None])[:, None]
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(sc - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(batch, kv, group * most, n), v).reshape(batch, kv, group, most, dim)
    o = torch.where(total == 0, torch.zeros_like(o), o / total)
    lse = (top + torch.log(total))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, most, heads, dim)
    lse = lse.permute(0, 3, 1, 2).reshape(batch, most, heads)
    tok = torch.arange(s["total"], device=dev)
    b = torch.searchsorted(q_start, tok, right=True) - 1
    at = (b, tok - q_start[b])
    return dict(out=o[at].to(s["q"].dtype), lse=lse[at])


def _sound(x):
    """Probabilities in float64, what is not positive and finite as 0."""
    x = x.double()
    return torch.where((x > 0) & (x < math.inf), x, 0.0)


def _plain_verify(s):
    case, dev = s["case"], s["probs"].device
    batch, most, vocab = s["rows"], s["most"], case["vocab"]
    q_start, parent, tokens = s["q_start"].long(), s["parent"].long(), s["tokens"].long()
    j = torch.arange(most, device=dev)
    at = (q_start[:-1, None] + j).clamp(max=s["total"] - 1)
    there = j < (q_start[1:] - q_start[:-1])[:, None]
    up = torch.where(there & (j > 0), parent[at], -1)                # B most
    # child[b][i][k]: the k-th child of row i, -1 where there are fewer.
    same = (up[:, :, None] == up[:, None, :]) & (j[None, :] < j[:, None])
    rank = same.sum(2)
    kids = case["branch"]
    child = torch.full((batch, most, kids + 1), -1, dtype=torch.int64, device=dev)
    b = torch.arange(batch, device=dev)
    slot = torch.where(up >= 0, rank, kids)
    child[b[:, None], up.clamp(min=0), slot] = torch.where(up >= 0, j.expand_as(up), -1)
    child = child[..., :kids]

    f64 = dict(dtype=torch.float64, device=dev)
    node = torch.zeros(batch, dtype=torch.int64, device=dev)
    going = q_start[1:] > q_start[:-1]
    path = torch.full((batch, most), -1, dtype=torch.int64, device=dev)
    path[:, 0] = torch.where(going, 0, -1)
    count = going.long()
    weights = torch.zeros((batch, vocab), **f64)     # what the next token is drawn from
    for step in range(min(case["depth"], most)):
        row = q_start[:-1] + node
        row = row.clamp(max=s["total"] - 1)
        p = _sound(s["probs"][row])
        d = _sound(s["draft"][row]) if case["draft"] else None
        c, W, Q = (torch.full((batch,), x, **f64) for x in (0.0, 1.0, 1.0))
        left = p                                     # the remainder, whose mass is W
        fresh = d if case["draft"] else p            # without the tokens refused here
        taken = torch.full((batch,), -1, dtype=torch.int64, device=dev)
        for k in range(kids):
            kid = child[b, node, k]
            open_ = going & (kid >= 0) & (taken < 0)
            row = (q_start[:-1] + kid.clamp(min=0)).clamp(max=s["total"] - 1)
            x, u = tokens[row], s["u"][row].double()
            ok = (x >= 0) & (x < vocab)
            x = x.clamp(0, vocab - 1)
            if case["draft"]:
                dx = fresh[b, x]
                ok = ok & (dx > 0) & (Q > 0)
                yes = open_ & ok & (u * dx * W < left[b, x] * Q)
                no = open_ & ok & ~yes
                c_new = c + W / Q
                after = (p - c_new[:, None] * d).clamp(min=0)
                mass = after.sum(1)
                change = no & (mass > 0)
                left = torch.where(change[:, None], after, left)
                c = torch.where(change, c_new, c)
                W = torch.where(change, mass, W)
                Q = torch.where(no, Q - dx, Q)
            else:
                px = fresh[b, x]
                ok = ok & (px > 0)
                yes = open_ & ok & (u * W < px)
                no = open_ & ok & ~yes
                after = left.scatter(1, x[:, None], 0.0)
                left = torch.where((no & (after.sum(1) > 0))[:, None], after, left)
                W = torch.where(no, W - px, W)
            fresh = torch.where(no[:, None], fresh.scatter(1, x[:, None], 0.0), fresh)
            taken = torch.where(yes, kid, taken)
        weights = torch.where((going & (taken < 0))[:, None], left, weights)
        going = going & (taken >= 0)
        node = torch.where(going, taken, node)
        if step + 1 < most:
            path[:, step + 1] = torch.where(going, taken, path[:, step + 1])
        count = count + going
    row = q_start[:-1].clamp(max=s["total"] - 1)
    sums = weights.cumsum(1)
    hit = (weights > 0) & (sums > (s["u"][row].double() * sums[:, -1])[:, None])
    last = vocab - 1 - (weights > 0).flip(1).to(torch.uint8).argmax(1)
    nxt = torch.where(hit.any(1), hit.to(torch.uint8).argmax(1), last)
    nxt = torch.where(sums[:, -1] > 0, nxt, -1)
    tok = torch.arange(s["total"], device=dev)
    of = torch.searchsorted(q_start, tok, right=True) - 1
    return dict(path=path[of, tok - q_start[of]].to(torch.int32), count=count.to(torch.int32),
                next=nxt.to(torch.int32))


def _exponent(case, amax):
    """Least e >= E_MIN with amax <= largest code * 2^e."""
    m, e = torch.frexp(amax)                         # amax = m * 2^e, 0.5 <= m < 1
    big, shift = (0.875, 9) if case["codes"] == "e4m3" else (127 / 128, 7)
    e = e - shift + (m > big)
    return torch.where(amax > 0, e.clamp(min=E_MIN), torch.full_like(e, E_MIN))


def _quantise(case, x):
    if case["codes"] == "e4m3":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)


def _plain_keep(s):
    case, dev = s["case"], s["pool"].device
    T, per = case["page"], case["page"] // BLOCK
    lens, q_start, count = s["lens"].long(), s["q_start"].long(), s["count"].long()
    base = lens - (q_start[1:] - q_start[:-1])
    end = base + count
    j = torch.arange(s["most"], device=dev)
    at = (q_start[:-1, None] + j).clamp(max=s["total"] - 1)
    path = torch.where(j < count[:, None], s["path"][at].long(), j)
    moved = path != j                                # ascending: all from the first on
    first = base + torch.where(moved.any(1), moved.to(torch.uint8).argmax(1), count)
    # Blocks from the first moved token's on, at most most / 16 + 2 of a request.
    nth = torch.arange(s["most"] // BLOCK + 2, device=dev)
    block = (first // BLOCK)[:, None] + nth
    real = ((block * BLOCK < end[:, None]) & (first < end)[:, None]).flatten()
    b = torch.arange(s["rows"], device=dev).repeat_interleave(len(nth))
    block = block.flatten()
    pos = block[:, None] * BLOCK + torch.arange(BLOCK, device=dev)           # n 16
    new = (pos >= first[b][:, None]) & (pos < end[b][:, None]) & real[:, None]
    old = (pos < first[b][:, None]) & real[:, None]
    src = base[b][:, None] + path[b[:, None], (pos - base[b][:, None]).clamp(0, s["most"] - 1)]
    src = torch.where(new, src, pos).clamp(max=s["table"].shape[1] * T - 1)
    kc, vc, ks, vs = _views(case, s["pool"])
    heads = torch.arange(case["kv"], device=dev)
    page = s["table"][b, (block // per).clamp(max=s["table"].shape[1] - 1)].long().clamp(min=0)
    where = (page[:, None], heads[None], (block % per)[:, None])             # n H
    from_ = s["table"][b[:, None], src // T].long().clamp(min=0)             # n 16
    from_ = (from_[..., None], heads[None, None], (src // BLOCK % per)[..., None])
    place = (src % BLOCK)[..., None]
    out = []
    for codes, scale, is_v in ((kc, ks, False), (vc, vs, True)):
        if is_v:
            x = _values(case, codes.transpose(3, 4)[(*from_, place)])        # n 16 H D
        else:
            x = _values(case, codes[(*from_, place)])
        was = scale[where]                                                   # n H
        held = codes[where].permute(0, 3, 1, 2) if is_v else codes[where].permute(0, 2, 1, 3)
        value = x * scale[from_][..., None]
        amax = torch.where(new[..., None, None], value, 0.0).abs().amax((1, 3))
        e_was = torch.frexp(was)[1] - 1
        e = torch.maximum(_exponent(case, amax), torch.where(old.any(1)[:, None], e_was, E_MIN))
        y = torch.where(new[..., None, None], value * _power(-e)[:, None, :, None],
                        x * _power(e_was - e)[:, None, :, None])
        y = torch.where((new | old)[..., None, None], _quantise(case, y), held)
        out.append((codes, scale, is_v, y, torch.where(real[:, None], _power(e), was)))
    # Entries without a block repeat the first one (or write back what is there).
    one = torch.where(real, torch.arange(len(real), device=dev), real.to(torch.uint8).argmax())
    where = tuple(w[one] if w.shape[0] == len(one) else w for w in where)
    for codes, scale, is_v, y, sc in out:
        y = y[one]
        codes[where] = y.permute(0, 2, 3, 1) if is_v else y.permute(0, 2, 1, 3)
        scale[where] = sc[one]
    return end.to(torch.int32)


def _plain_read(s):
    case, dev = s["case"], s["pool"].device
    T, start = case["page"], s["start"].long()
    tok = torch.arange(s["total"], device=dev)
    b = torch.searchsorted(start, tok, right=True) - 1
    pos = s["first"].long()[b] + tok - start[b]
    page = s["table"][b, pos // T].long()
    kc, vc, ks, vs = _views(case, s["pool"])
    heads = torch.arange(case["kv"], device=dev)
    where = (page[:, None], heads[None], (pos % T // BLOCK)[:, None])
    place = (pos % BLOCK)[:, None]
    dt = DTYPES[case["dtype"]]
    k = _values(case, kc[(*where, place)]) * ks[where][..., None]
    v = _values(case, vc.transpose(3, 4)[(*where, place)]) * vs[where][..., None]
    return dict(k=k.to(dt), v=v.to(dt))


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _code_type(case):
    return torch.float8_e4m3fn if case["codes"] == "e4m3" else torch.int8


def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        import memory_dma_descriptor_amd as dd
        codes = dd.KV_INT8 if case.get("codes") == "int8" else dd.KV_E4M3
    if kind == "tree":
        if own:
            r = dd.kv_attend_tree(s["q"], s["q_start"], s["parent"], s["pool"], s["table"], s["lens"],
                                  case["kv"], case["page"], codes=codes, check=False)
            return dict(out=r["out"], lse=r["lse"])
        return _plain_tree(s)
    if kind == "verify":
        if own:
            r = dd.verify_drafts(s["probs"], s["tokens"], s["parent"], s["q_start"], s["u"],
                                 draft=s["draft"], check=False)
            return dict(path=r["path"], count=r["count"], next=r["next"])
        return _plain_verify(s)
    if kind == "read":
        if own:
            return dd.kv_read(s["first"], s["start"], s["total"], s["pool"], s["table"], s["lens"],
                              case["kv"], case["page"], case["dim"], codes=codes,
                              dtype=DTYPES[case["dtype"]], check=False)
        return _plain_read(s)
    if own:
        r = dd.kv_keep(s["path"], s["count"], s["q_start"], s["pool"], s["table"], s["lens"], case["kv"],
                       case["page"], case["dim"], codes=codes, check=False)
        keep = r["keep"]
    else:
        keep = _plain_keep(s)
    code_bytes, scales, _ = page_layout(case)
    pool = s["pool"]
    return dict(codes=pool[:, :2 * code_bytes].view(_code_type(case)), keep=keep,
                scales=pool.view(torch.float32)[:, code_bytes // 2:code_bytes // 2 + 2 * scales])


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    kind = case["kind"]
    if kind == "verify":
        size = 4 if case["dtype"] == "fp32" else 2
        total = sum(len(p) for p in trees(case))
        rows = 2 if case["draft"] else 1             # of the node where each request's path ends
        return {"bytes": case["batch"] * (rows * case["vocab"] * size + 12) + 16 * total,
                "flops": 3 * case["batch"] * case["vocab"]}
    kv, dim, T = case["kv"], case["dim"], case["page"]
    lens = lengths(case)
    if kind == "tree":
        shape, heads = trees(case), case["heads"]
        rows = sum(len(p) for p in shape)
        nbytes = (sum(lens) * kv * 2 * dim + sum(lens) // BLOCK * kv * 8 + rows * (heads * (4 * dim + 4) + 4)
                  + 4 * sum(_ceil(x, T) for x in lens))
        pairs = sum(len(p) * (x - len(p)) for p, x in zip(shape, lens))
        for p in shape:
            depth = []
            for x in p:
                depth.append(1 if x < 0 else depth[x] + 1)
            pairs += sum(depth)
        return {"bytes": nbytes, "flops": 4 * dim * heads * pairs}
    if kind == "keep":
        moved = sum(sum(x != k for k, x in enumerate(p)) for p in paths(case))
        return {"bytes": 2 * moved * kv * 2 * dim + 8 * kv * _ceil(moved, BLOCK)
                + 4 * sum(len(p) for p in trees(case)) + 16 * case["batch"], "flops": 4 * moved * kv * dim}
    n = sum(x for _, x in pieces(case))
    size = 4 if case["dtype"] == "fp32" else 2
    return {"bytes": 2 * n * kv * dim * (size + 1) + 8 * kv * _ceil(n, BLOCK) + 4 * _ceil(n, T),
            "flops": 2 * n * kv * dim}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def _e4m3(byte):
    """e4m3 codes as float64, from the format: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    b = byte.long()
    sign = 1.0 - 2.0 * (b >> 7).double()
    e, m = (b >> 3) & 15, (b & 7).double()
    size = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2((e - 7).double()))
    return sign * torch.where((b & 127) == 127, torch.full_like(size, math.nan), size)


def _int8(byte):
    b = byte.long()
    return (b - 256 * (b >> 7)).double()


def _row_cache(s, b, upto):
    """Keys and values [tokens][H][D] of one request's first `upto` tokens, float64."""
    case = s["case"]
    kv, dim, T = case["kv"], case["dim"], case["page"]
    codes, scales, _ = page_layout(case)
    pages = s["pool"][s["table"][b, :_ceil(upto, T)].long()]
    read = _e4m3 if case["codes"] == "e4m3" else _int8
    sc = pages[:, 2 * codes:2 * codes + 8 * scales].contiguous().view(torch.float32).double()
    sc = sc.reshape(-1, 2, kv, T // BLOCK).repeat_interleave(BLOCK, 3)      # page, K/V, head, token
    k = read(pages[:, :codes]).reshape(-1, kv, T, dim) * sc[:, 0, :, :, None]
    v = read(pages[:, codes:2 * codes]).reshape(-1, kv, T // BLOCK, dim, BLOCK)
    v = v.transpose(3, 4).reshape(-1, kv, T, dim) * sc[:, 1, :, :, None]
    return [x.transpose(1, 2).reshape(-1, kv, dim)[:upto] for x in (k, v)]


def _exact_tree(s):
    case = s["case"]
    dim, group = case["dim"], case["heads"] // case["kv"]
    outs, sums, at = [], [], 0
    for b, (length, parent) in enumerate(zip(lengths(case), trees(case))):
        k, v = _row_cache(s, b, length)
        n = len(parent)
        seen = torch.zeros((n, length), dtype=torch.bool)
        seen[:, :length - n] = True
        for j in range(n):
            i = j
            while i >= 0:
                seen[j, length - n + i] = True
                i = parent[i]
        seen = seen.to(k.device)
        o = torch.zeros((n, case["heads"], dim), dtype=torch.float64, device=k.device)
        lse = torch.zeros((n, case["heads"]), dtype=torch.float64, device=k.device)
        for h in range(case["heads"]):
            sc = s["q"][at:at + n, h].double() @ k[:, h // group].T.contiguous() / math.sqrt(dim)
            sc = torch.where(seen, sc, -math.inf)
            lse[:, h] = torch.logsumexp(sc, 1)
            o[:, h] = torch.exp(sc - lse[:, h, None]) @ v[:, h // group].contiguous()
        outs.append(o)
        sums.append(lse)
        at += n
    return dict(out=torch.cat(outs), lse=torch.cat(sums))


def _exact_verify(s):
    """The rule as it is usually told: the remainder and the draft's row, each
    brought to mass 1, are subtracted after every refusal."""
    case = s["case"]
    path, counts, nexts, at = [], [], [], 0
    for parent in trees(case):
        n, node, taken = len(parent), 0, [0]
        tok, u = s["tokens"][at:at + n].tolist(), s["u"][at:at + n].double().tolist()
        while True:
            w = s["probs"][at + node].double()
            d = s["draft"][at + node].double().clone() if case["draft"] else None
            mass, rest, step = 1.0, 1.0, -1
            for kid in (j for j in range(1, n) if parent[j] == node):
                x = tok[kid]
                px, dx = float(w[x]), float(d[x]) if case["draft"] else 1.0
                if not case["draft"]:
                    if u[kid] * mass < px:
                        step = kid
                        break
                    mass -= px
                    was = px
                    w = w.clone()
                    w[x] = 0
                    if float(w.sum()) <= 0:
                        w[x] = was
                elif dx > 0 and rest > 0:
                    if u[kid] * (dx / rest) < px / mass:
                        step = kid
                        break
                    after = (w / mass - d / rest).clamp(min=0)
                    if float(after.sum()) > 0:
                        w, mass = after, float(after.sum())
                    d[x] = 0
                    rest -= dx
            if step < 0:
                break
            taken.append(step)
            node = step
        sums = w.cumsum(0)
        hit = ((sums > u[0] * float(sums[-1])) & (w > 0)).nonzero()
        nexts.append(int(hit[0]) if len(hit) else int((w > 0).nonzero()[-1]))
        counts.append(len(taken))
        path += taken + [-1] * (n - len(taken))
        at += n
    return dict(path=_i32(path), count=_i32(counts), next=_i32(nexts))


def _exact_keep(s):
    case = s["case"]
    codes, scales, _ = page_layout(case)
    kv, per, T, dim = case["kv"], case["page"] // BLOCK, case["page"], case["dim"]
    pool = s["pool"]
    read = _e4m3 if case["codes"] == "e4m3" else _int8
    most = 448.0 if case["codes"] == "e4m3" else 127.0

    def nearest(x):                                  # the code value next to x, ties to even
        if case["codes"] == "e4m3":
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
        else:
            step = torch.ones_like(x)
        return (torch.round(x / step) * step).clamp(-most, most)

    value = read(pool[:, :2 * codes])
    scale = pool[:, 2 * codes:2 * codes + 8 * scales].contiguous().view(torch.float32).double()
    # [page][K, V][H][block]; K as [page][H][block][16][D], V turned the same way.
    k = value[:, :codes].reshape(-1, kv, per, BLOCK, dim).clone()
    v = value[:, codes:].reshape(-1, kv, per, dim, BLOCK).transpose(3, 4).clone()
    scale = scale.reshape(-1, 2, kv, per).clone()
    keep = []
    for b, (length, tree, path) in enumerate(zip(lengths(case), trees(case), paths(case))):
        base = length - len(tree)
        end = base + len(path)
        keep.append(end)
        go = [i for i, x in enumerate(path) if x != i]
        if not go:
            continue
        first = base + go[0]
        pages = s["table"][b].tolist()
        src = torch.tensor([base + x for x in path[go[0]:]])
        pg = torch.tensor([pages[t // T] for t in src.tolist()], device=pool.device)
        src = src.to(pool.device)
        for z, held in ((0, k), (1, v)):
            sub = src % T // BLOCK
            real = held[pg, :, sub, src % BLOCK] * scale[pg, z, :, sub][..., None]      # tokens H D
            for blk in range(first // BLOCK, (end - 1) // BLOCK + 1):
                a, o = max(first, blk * BLOCK), min(end, blk * BLOCK + BLOCK)
                part = real[a - first:o - first]
                e = torch.full((kv,), float(E_MIN), dtype=torch.float64, device=pool.device)
                top = part.abs().amax((0, 2))
                guess = torch.ceil(torch.log2((top / most).clamp(min=2.0 ** E_MIN)))
                for near in (guess + 1, guess, guess - 1):           # the least that holds them all
                    guess = torch.where(top <= most * torch.exp2(near), near, guess)
                e = torch.maximum(e, guess)
                page, sub_ = pages[blk // per], blk % per
                was = scale[page, z, :, sub_]
                here = held[page, :, sub_]                           # H 16 D, a view
                if a > blk * BLOCK:
                    e = torch.maximum(e, torch.log2(was))
                    early = here[:, :a - blk * BLOCK]
                    early.copy_(nearest(early * (was / torch.exp2(e))[:, None, None]))
                here[:, a - blk * BLOCK:o - blk * BLOCK] = nearest(
                    part / torch.exp2(e)[:, None]).transpose(0, 1)
                scale[page, z, :, sub_] = torch.exp2(e)
    flat = torch.cat([k.flatten(1), v.transpose(3, 4).flatten(1)], 1)
    return dict(codes=flat, keep=_i32(keep), scales=scale.flatten(1))


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "tree":
        return _exact_tree(s)
    if case["kind"] == "verify":
        return _exact_verify(s)
    if case["kind"] == "keep":
        return _exact_keep(s)
    ks, vs = [], []
    for b, (first, n) in enumerate(pieces(case)):
        k, v = _row_cache(s, b, first + n)
        ks.append(k[first:])
        vs.append(v[first:])
    return dict(k=torch.cat(ks), v=torch.cat(vs))
