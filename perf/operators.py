"""The paged 8-bit key/value cache as it is measured: inputs, plain forms and
the library's calls.

Three operators: `attend` (attention of new tokens over the cache), `append`
(quantising new keys and values into its pages) and the page operations
(`step`: free, fork, reserve, copy; `compact`: gather the live pages at the
front). Where `own` is false, run() computes them with elementary torch
operations; where it is true, through this package.

A page holds T tokens of H heads of D values: K codes [H][T][D], V codes
[H][T/16][D][16], K scales float32 [H][T/16], V scales [H][T/16], padded to
512 bytes. A scale is a power of two for 16 tokens of one head.
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
        # One request answering alone: every call's latency counts.
        dict(name="attend one token", kind="attend", batch=1, news=1, lo=900, hi=900, heads=32,
             kv=8, dim=128, page=64, codes="e4m3", dtype="bf16", causal=True),
        # A serving batch, a token each, lengths as they come.
        dict(name="attend batch", kind="attend", batch=64, news=1, lo=200, hi=9000, heads=32,
             kv=8, dim=128, page=64, codes="e4m3", dtype="bf16", causal=True),
        # A few long documents, a token each: the cache is the whole cost.
        dict(name="attend long", kind="attend", batch=4, news=1, lo=100000, hi=131072, heads=32,
             kv=8, dim=128, page=128, codes="e4m3", dtype="bf16", causal=True),
        # Checking five drafted tokens of each request, seven heads on one key head, small pages.
        dict(name="attend drafts int8", kind="attend", batch=33, news=5, lo=17, hi=4001, heads=28,
             kv=4, dim=128, page=16, codes="int8", dtype="fp16", causal=True),
        # A piece of a long prompt against what is already cached.
        dict(name="attend chunk", kind="attend", batch=1, news=2048, lo=16384, hi=16384, heads=32,
             kv=8, dim=128, page=64, codes="e4m3", dtype="bf16", causal=True),
        # Ragged prompts of a model whose every head has its own keys, none shared.
        dict(name="attend prompts", kind="attend", batch=7, news=777, lo=777, hi=2100, heads=16,
             kv=16, dim=64, page=32, codes="int8", dtype="fp16", causal=True),
        # The same serving batch's write: one token of each request.
        dict(name="append step", kind="append", batch=128, news=1, lo=1, hi=4000, kv=8, dim=128,
             page=64, codes="e4m3", dtype="bf16"),
        # Prompts written whole; ends inside blocks and pages.
        dict(name="append prompts", kind="append", batch=9, news=4097, lo=4097, hi=9000, kv=8,
             dim=128, page=64, codes="e4m3", dtype="bf16"),
        dict(name="append prompts int8", kind="append", batch=5, news=1555, lo=1555, hi=1600, kv=4,
             dim=256, page=32, codes="int8", dtype="fp32"),
        # A sampling step of a few requests: two end, four branch, all take a token.
        dict(name="step small", kind="step", rows=24, free=2, fork=4, lo=40, hi=900, kv=2, dim=64,
             page=16, slack=200, codes="int8"),
        # The same for thousands of requests in a large heap.
        dict(name="step large", kind="step", rows=4096, free=256, fork=512, lo=100, hi=6000, kv=1,
             dim=128, page=32, slack=30000, codes="int8"),
        # Bringing the live pages together before the rest of the heap is given back.
        dict(name="compact", kind="compact", rows=200, lo=64, hi=4000, kv=8, dim=128, page=64,
             slack=5000, codes="e4m3"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "append", "append", "step", "compact"])
    codes = rng.choice(["e4m3", "int8"])
    page = rng.choice([16, 32, 64, 128])
    if kind == "attend":
        kv = rng.choice([1, 2, 4, 5, 8])
        dim = rng.choice([64, 128, 128, 256])
        group = rng.choice([1, 2, 3, 4, 7, 8])
        if rng.random() < 0.6:                       # few tokens of each request
            batch = _spread(rng, 1, 100)
            news = rng.choice([1, 1, 1, 2, 4, 7])
            hi = _spread(rng, 16, min(100000, 1000000 // batch))
        else:                                        # chunks of prompts
            batch = _spread(rng, 1, 6)
            news = _spread(rng, 20, 1500)
            hi = _spread(rng, news, 8000)
        # No more cache, and no more products, than the largest listed cases.
        hi = min(hi, 10 ** 9 // (batch * kv * 2 * dim),
                 2048 * 16384 * 32 * 128 // (batch * news * kv * group * dim))
        lo = max(news, hi // rng.choice([1, 2, 20]))
        return dict(kind=kind, batch=batch, news=news, lo=lo, hi=max(lo, hi), heads=kv * group,
                    kv=kv, dim=dim, page=page, codes=codes, dtype=rng.choice(["bf16", "fp16"]),
                    causal=rng.random() < 0.8)
    if kind == "append":
        news = rng.choice([1, 1, 3, _spread(rng, 5, 4000)])
        batch = _spread(rng, 1, 200) if news < 5 else _spread(rng, 1, max(1, 20000 // news))
        return dict(kind=kind, batch=batch, news=news, lo=news, hi=news + _spread(rng, 1, 3000),
                    kv=rng.choice([1, 2, 4, 8]), dim=rng.choice([64, 128, 256]), page=page,
                    codes=codes, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if kind == "step":
        rows = _spread(rng, 20, 3000)
        return dict(kind=kind, rows=rows, free=max(1, rows // 16), fork=max(1, rows // 9),
                    lo=_spread(rng, 1, 60), hi=_spread(rng, 100, 4000), kv=1, dim=64, page=page,
                    slack=_spread(rng, 3 * rows, 20000), codes=codes)
    return dict(kind=kind, rows=_spread(rng, 5, 300), lo=_spread(rng, 16, 100),
                hi=_spread(rng, 200, 3000), kv=rng.choice([1, 2, 4]), dim=128, page=page,
                slack=_spread(rng, 20, 8000), codes=codes)


# --------------------------------------------------------------------------
# sizes that follow from a case
# --------------------------------------------------------------------------

def page_layout(case):
    """(code bytes of K or V, scales of K or V, page bytes)."""
    codes = case["kv"] * case["page"] * case["dim"]
    scales = case["kv"] * (case["page"] // BLOCK)
    return codes, scales, -(-(2 * codes + 8 * scales) // 512) * 512


def lengths(case):
    """Tokens of every request (or row): spread over lo..hi, both reached."""
    n = case.get("batch") or case["rows"]
    rng = random.Random(n * 1000003 + case["hi"])
    out = [rng.randint(case["lo"], case["hi"]) for _ in range(n)]
    out[0] = case["hi"]
    if n > 1:
        out[-1] = case["lo"]
    return out


def new_tokens(case):
    """New tokens of every request: `news`, fewer for some where there are many."""
    n, k = case["batch"], case["news"]
    if k < 8:
        return [k] * n
    return [k if b % 3 == 0 else max(1, k // (1 + b % 5)) for b in range(n)]


def _ceil(a, b):
    return -(-a // b)


def _power(e):
    """2^e in float32 (no smaller than 2^-126), from the format."""
    return ((e.clamp(min=-126).to(torch.int32) + 127) << 23).view(torch.float32)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")
    kv, dim, T = case["kv"], case["dim"], case["page"]
    codes, scales, page_bytes = page_layout(case)
    lens = lengths(case)
    need = [_ceil(x, T) for x in lens]
    spare = case.get("slack", 8)
    npages = sum(need) + spare
    wide = max(need) + 2
    i32 = dict(dtype=torch.int32, device=dev)

    # Pages as earlier appends left them: values around zero with a few larger
    # channels, a scale that follows each block's largest value.
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
    sc = _power(e).view(torch.uint8)
    pool[:, 2 * codes:2 * codes + 8 * scales] = sc

    order = torch.randperm(npages, generator=g, device=dev).to(torch.int32)
    rows = len(lens)
    table = torch.full((rows, wide), -1, **i32)
    start = torch.tensor([0] + need, dtype=torch.int64, device=dev).cumsum(0)
    col = torch.arange(wide, device=dev)
    at = start[:-1, None] + col
    used = col < torch.tensor(need, device=dev)[:, None]
    table = torch.where(used, order[at.clamp(max=npages - 1)], table)
    lens_t = torch.tensor(lens, **i32)
    s = dict(case=case, pool=pool, table=table, lens=lens_t, rows=rows, npages=npages, wide=wide)

    if case["kind"] in ("attend", "append"):
        news = new_tokens(case)
        q_start = torch.tensor([0] + news, dtype=torch.int64).cumsum(0).to(torch.int32)
        s.update(q_start=q_start.to(dev), total=sum(news), most=max(news), longest=max(lens))
        dt = DTYPES[case["dtype"]]
        if case["kind"] == "attend":
            s["q"] = torch.randn((s["total"], case["heads"], dim), generator=g, device=dev).to(dt)
        else:
            both = torch.randn((s["total"], 2 * kv, dim), generator=g, device=dev)
            both[:, :kv, ::37] *= 5                  # keys have a few large channels
            both = both.to(dt)                       # one projection's output: k and v are strided
            s["k"], s["v"] = both[:, :kv], both[:, kv:]
        return s

    # Which pages are in use, by how many rows.
    refs = torch.zeros(npages, **i32)
    refs[table[used].long()] = 1
    s["refs"] = refs
    # Buffers that a pass works on, so that every pass starts alike.
    s.update(refs_w=refs.clone(), table_w=table.clone(), lens_w=lens_t.clone())
    if case["kind"] == "step":
        f, k = case["free"], case["fork"]
        some = torch.randperm(rows, generator=g, device=dev)[:f + k].to(torch.int32)
        gone, parent = some[:f].contiguous(), some[f:].contiguous()
        # Children take the ended rows first, then rows kept free for them.
        extra = torch.arange(rows, rows + k, **i32)
        child = torch.cat([gone, extra])[:k].contiguous()
        s["table"] = torch.cat([table, torch.full((k, wide), -1, **i32)])
        s["lens"] = torch.cat([lens_t, torch.zeros(k, **i32)])
        s.update(table_w=s["table"].clone(), lens_w=s["lens"].clone(), gone=gone, parent=parent,
                 child=child)
        live = torch.ones(rows + k, dtype=torch.bool, device=dev)
        live[gone.long()] = False
        live[rows:] = False
        live[child.long()] = True
        s["slot"] = live.nonzero().flatten().to(torch.int32)
        s["n_new"] = torch.ones(s["slot"].numel(), **i32)
    return s


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
    n = pool.shape[0]
    k = pool[:, :codes].unflatten(1, (kv, nb, BLOCK, dim))
    v = pool[:, codes:2 * codes].unflatten(1, (kv, nb, dim, BLOCK))
    f = pool.view(torch.float32)[:, codes // 2:codes // 2 + 2 * scales].unflatten(1, (2, kv, nb))
    assert k.shape[0] == n
    return k, v, f[:, 0], f[:, 1]


def _plain_attend(s):
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

    count = q_start[1:] - q_start[:-1]
    j = torch.arange(most, device=dev)
    at = (q_start[:-1, None] + j).clamp(max=s["total"] - 1)
    q = s["q"][at].float().reshape(batch, most, kv, group, dim).permute(0, 2, 3, 1, 4)
    sc = torch.matmul(q.reshape(batch, kv, group * most, dim), k.transpose(2, 3).contiguous())
    sc = sc.reshape(batch, kv, group, most, n) * (1.0 / math.sqrt(dim))
    t = torch.arange(n, device=dev)
    seen = (t < lens[:, None])[:, None, :].expand(batch, most, n)
    if case["causal"]:
        seen = seen & (t <= (lens - count)[:, None, None] + j[:, None])
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


def _merge(case, x, old_codes, old_scale, is_new, is_old):
    """Codes and scales of blocks [n][16][H][D] that hold old and new tokens."""
    has_old = is_old.any(1)[:, None]                                       # n 1
    new = is_new[:, :, None, None]
    old = is_old[:, :, None, None]
    amax = torch.where(new, x, torch.zeros_like(x)).abs().amax((1, 3))     # n H
    e_old = torch.where(has_old, torch.frexp(old_scale)[1] - 1, torch.full_like(amax, E_MIN).int())
    e = torch.maximum(_exponent(case, amax), e_old)
    up = _power(-e)[:, None, :, None]
    again = _power(e_old - e)[:, None, :, None]
    y = torch.where(new, x * up, torch.where(old, old_codes * again, torch.zeros_like(x)))
    return _quantise(case, y), _power(e)


def _plain_append(s):
    case, dev = s["case"], s["pool"].device
    T, per = case["page"], case["page"] // BLOCK
    lens, q_start = s["lens"].long(), s["q_start"].long()
    count = q_start[1:] - q_start[:-1]
    first = lens - count
    # Touched blocks of every request, at most ceil((n + 15) / 16) of n tokens.
    blocks = torch.where(count > 0, (lens - 1) // BLOCK - first // BLOCK + 1, torch.zeros_like(lens))
    base = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), blocks.cumsum(0)])
    i = torch.arange(s["total"] // BLOCK + 2 * s["rows"], device=dev)
    i = torch.minimum(i, base[-1] - 1)               # the last block again, with the same values
    b = torch.searchsorted(base, i, right=True) - 1
    block = first[b] // BLOCK + i - base[b]
    page = s["table"][b, block // per].long()
    sub = block % per
    pos = block[:, None] * BLOCK + torch.arange(BLOCK, device=dev)          # n 16
    is_new = (pos >= first[b][:, None]) & (pos < lens[b][:, None])
    is_old = pos < first[b][:, None]
    at = (q_start[b][:, None] + pos - first[b][:, None]).clamp(0, s["total"] - 1)
    kc, vc, ks, vs = _views(case, s["pool"])
    heads = torch.arange(case["kv"], device=dev)
    where = (page[:, None], heads[None], sub[:, None])                      # n H
    k, k_scale = _merge(case, s["k"][at].float(), _values(case, kc[where]).permute(0, 2, 1, 3),
                        ks[where], is_new, is_old)
    v, v_scale = _merge(case, s["v"][at].float(), _values(case, vc[where]).permute(0, 3, 1, 2),
                        vs[where], is_new, is_old)
    kc[where] = k.permute(0, 2, 1, 3)
    vc[where] = v.permute(0, 2, 3, 1)
    ks[where] = k_scale
    vs[where] = v_scale


def _plain_step(s):
    case, T, dev = s["case"], s["case"]["page"], s["pool"].device
    refs, table, lens = s["refs_w"], s["table_w"], s["lens_w"]
    col = torch.arange(s["wide"], device=dev)

    def change(rows, by):                            # references of the pages of some rows
        at = table[rows]
        used = (col < ((lens[rows] + T - 1) // T)[:, None])
        refs.index_add_(0, at.clamp(min=0).flatten().long(), (used * by).flatten().to(torch.int32))

    gone, parent, child, slot = (s[k].long() for k in ("gone", "parent", "child", "slot"))
    change(gone, -1)
    table[gone] = -1
    lens[gone] = 0
    table[child] = table[parent]
    lens[child] = lens[parent]
    change(child, 1)

    length, new = lens[slot], s["n_new"]
    have, want = (length + T - 1) // T, (length + new + T - 1) // T
    last = table[slot, (have - 1).clamp(min=0).long()].clamp(min=0)
    shared = (length % T != 0) & (refs[last.long()] > 1) & (new > 0)
    take = want - have + shared.int()
    before = take.cumsum(0) - take
    free = torch.argsort((refs != 0).to(torch.uint8), stable=True).to(torch.int32)
    none = torch.full_like(last, -1)
    fresh_from = have - shared.int()
    at = col[None] - fresh_from[:, None]                                    # which of its new pages
    given = (at >= 0) & (at < take[:, None])
    page = free[(before[:, None] + at).clamp(0, s["npages"] - 1)]
    src = torch.where(shared, last, none)
    dst = torch.where(shared, free[before.clamp(max=s["npages"] - 1).long()], none)
    table[slot] = torch.where(given, page, table[slot])
    refs.index_add_(0, page.flatten().long(), given.flatten().to(torch.int32))
    refs.index_add_(0, last.long(), -shared.to(torch.int32))
    lens[slot] = length + new
    _plain_copy(s["pool"], src, dst)
    return src, dst


def _plain_copy(pool, src, dst):
    """Copies the listed pages; entries of -1 repeat the first listed copy (or
    copy page 0 to itself where none is listed)."""
    one = (src >= 0).to(torch.uint8).argmax()
    fill_src, fill_dst = src[one].clamp(min=0), dst[one].clamp(min=0)
    a = torch.where(src >= 0, src, fill_src).long()
    b = torch.where(src >= 0, dst, fill_dst).long()
    pool[b] = pool[a]


def _plain_compact(s):
    dev, n = s["pool"].device, s["npages"]
    refs, table = s["refs_w"], s["table_w"]
    ids = torch.arange(n, dtype=torch.int32, device=dev)
    live = refs > 0
    total = live.sum().to(torch.int32)
    hole = ~live & (ids < total)
    mover = live & (ids >= total)
    half = n // 2
    moves = mover.sum().to(torch.int32)
    listed_ = torch.arange(half, device=dev) < moves
    none = torch.full((half,), -1, dtype=torch.int32, device=dev)
    src = torch.where(listed_, torch.argsort((~mover).to(torch.uint8), stable=True)[:half].int(), none)
    dst = torch.where(listed_, torch.argsort((~hole).to(torch.uint8), stable=True)[:half].int(), none)
    rank = (mover.cumsum(0) - 1).clamp(0, half - 1)
    name = torch.where(mover, dst[rank], ids)
    used = table >= 0
    table.copy_(torch.where(used, name[table.clamp(min=0).long()], table))
    moved = torch.zeros_like(refs)
    moved.index_add_(0, name.long(), refs)           # free pages keep their name and add nothing
    refs.copy_(moved)
    _plain_copy(s["pool"], src, dst)
    return src, dst, moves


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _code_type(case):
    return torch.float8_e4m3fn if case["codes"] == "e4m3" else torch.int8


def run(s):
    case = s["case"]
    kind, T = case["kind"], case["page"]
    if own:
        import memory_dma_descriptor_amd as dd
        codes = dd.KV_E4M3 if case["codes"] == "e4m3" else dd.KV_INT8
    if kind == "attend":
        if own:
            r = dd.kv_attend(s["q"], s["q_start"], s["pool"], s["table"], s["lens"], case["kv"], T,
                             codes=codes, causal=case["causal"], check=False)
            return dict(out=r["out"], lse=r["lse"])
        return _plain_attend(s)
    if kind == "append":
        if own:
            dd.kv_append(s["k"], s["v"], s["q_start"], s["pool"], s["table"], s["lens"], T,
                         codes=codes, check=False)
        else:
            _plain_append(s)
        code_bytes, scales, _ = page_layout(case)
        pool = s["pool"]
        return dict(codes=pool[:, :2 * code_bytes].view(_code_type(case)),
                    scales=pool.view(torch.float32)[:, code_bytes // 2:code_bytes // 2 + 2 * scales])
    s["refs_w"].copy_(s["refs"])
    s["table_w"].copy_(s["table"])
    s["lens_w"].copy_(s["lens"])
    state = dict(refs=s["refs_w"], table=s["table_w"], lens=s["lens_w"], pool=s["pool"])
    if kind == "step":
        if own:
            kv = (s["refs_w"], s["table_w"], s["lens_w"])
            dd.kv_free(*kv, s["gone"], T, check=False)
            dd.kv_fork(*kv, s["parent"], s["child"], T, check=False)
            r = dd.kv_reserve(*kv, s["slot"], s["n_new"], T, check=False)
            dd.kv_copy_pages(s["pool"], r["src"], r["dst"])
            src, dst = r["src"], r["dst"]
        else:
            src, dst = _plain_step(s)
        return dict(state, src=src, dst=dst)
    if own:
        r = dd.kv_compact(s["refs_w"], s["table_w"], s["lens_w"], T)
        dd.kv_copy_pages(s["pool"], r["src"], r["dst"], count=r["moves"])
        src, dst, moves = r["src"], r["dst"], r["moves"][0]
    else:
        src, dst, moves = _plain_compact(s)
    return dict(state, src=src, dst=dst, moves=moves)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    kv, dim, T = case["kv"], case["dim"], case["page"]
    _, _, page_bytes = page_layout(case)
    lens = lengths(case)
    if case["kind"] == "attend":
        news, heads = new_tokens(case), case["heads"]
        cached = sum(lens)
        rows = sum(news) * heads
        pairs = sum(n * x - (n * (n - 1) // 2 if case["causal"] else 0) for n, x in zip(news, lens))
        nbytes = (cached * kv * 2 * dim + cached // BLOCK * kv * 8 + rows * (4 * dim + 4)
                  + 4 * sum(_ceil(x, T) for x in lens))
        return {"bytes": nbytes, "flops": 4 * dim * heads * pairs}
    if case["kind"] == "append":
        n = sum(new_tokens(case))
        size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
        return {"bytes": 2 * n * kv * dim * (size + 1) + 8 * kv * _ceil(n, BLOCK), "flops": 6 * n * kv * dim}
    pages = sum(_ceil(x, T) for x in lens)
    npages = pages + case["slack"]
    wide = max(_ceil(x, T) for x in lens) + 2
    rows = case["rows"] + case.get("fork", 0)
    start = 4 * 2 * (npages + rows * wide + rows)    # the state that a pass starts from
    if case["kind"] == "step":
        mean = pages / case["rows"]
        copies = 2 * case["fork"] * (T - 1) / T      # parent and child both leave the shared page
        entries = 4 * mean * (2 * case["free"] + 3 * case["fork"])
        return {"bytes": int(start + 4 * npages + entries + 2 * page_bytes * copies), "flops": 0}
    moves = pages * case["slack"] / npages           # live pages past the last place they may keep
    return {"bytes": int(start + 8 * npages + 8 * pages + 2 * page_bytes * moves), "flops": 0}


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


def exact(case, seed):
    if case["kind"] in ("step", "compact"):
        return None                                  # whole numbers and copied bytes
    s = prepare(case, seed)
    lens, news = lengths(case), new_tokens(case)
    kv, dim = case["kv"], case["dim"]
    if case["kind"] == "attend":
        group = case["heads"] // kv
        outs, sums, at = [], [], 0
        for b, (length, n) in enumerate(zip(lens, news)):
            k, v = _row_cache(s, b, length)
            pos = torch.arange(length - n, length, device=k.device)
            seen = torch.arange(length, device=k.device) <= (pos[:, None] if case["causal"] else length)
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

    # append: every touched block written anew from the definition.
    codes, scales, _ = page_layout(case)
    per = case["page"] // BLOCK
    pool = s["pool"]
    read = _e4m3 if case["codes"] == "e4m3" else _int8
    most, least = (448.0, 2.0 ** -9) if case["codes"] == "e4m3" else (127.0, 1.0)

    def nearest(x):                                  # the code value next to x, ties to even
        if case["codes"] == "e4m3":
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
        else:
            step = torch.full_like(x, least)
        return (torch.round(x / step) * step).clamp(-most, most)

    value = read(pool[:, :2 * codes])
    scale = pool[:, 2 * codes:2 * codes + 8 * scales].contiguous().view(torch.float32).double()
    k = value[:, :codes].unflatten(1, (kv, per, BLOCK, dim))
    v = value[:, codes:].unflatten(1, (kv, per, dim, BLOCK))
    ks, vs = (scale.unflatten(1, (2, kv, per))[:, x] for x in (0, 1))
    # Every request's first touched block may hold earlier tokens; handled one by one.
    at = 0
    for b, (length, n) in enumerate(zip(lens, news)):
        first = length - n
        b0, b1 = first // BLOCK, (length - 1) // BLOCK
        pages = s["table"][b].long()
        block = torch.arange(b0, b1 + 1, device=pool.device)
        where = (pages[block // per], block % per)
        for x, held, sc, perm in ((s["k"], k, ks, (0, 2, 1, 3)), (s["v"], v, vs, (0, 3, 1, 2))):
            y = torch.zeros(((b1 - b0 + 1) * BLOCK, kv, dim), dtype=torch.float64, device=pool.device)
            y[first - b0 * BLOCK:length - b0 * BLOCK] = x[at:at + n].double()
            y = y.reshape(-1, BLOCK, kv, dim)
            top = y.abs().amax((1, 3))
            e = torch.ceil(torch.log2((top / most).clamp(min=2.0 ** E_MIN)))
            e += (top > most * torch.exp2(e)).double() - (top <= most * torch.exp2(e - 1)).double()
            e = e.clamp(min=E_MIN)
            if first % BLOCK:
                was = sc[where[0][0], :, where[1][0]]
                e[0] = torch.maximum(e[0], torch.log2(was))
            y = nearest(y / torch.exp2(e)[:, None, :, None])
            if first % BLOCK:
                old = held[where[0][0], :, where[1][0]]                     # H 16 D or H D 16
                old = old.permute(1, 0, 2) if perm[1] == 2 else old.permute(2, 0, 1)
                old = nearest(old * (was / torch.exp2(e[0]))[None, :, None])
                y[0, :first % BLOCK] = old[:first % BLOCK]
            back = (0, 2, 1, 3) if perm[1] == 2 else (0, 2, 3, 1)
            held[where[0], :, where[1]] = y.permute(*back)
            sc[where[0], :, where[1]] = torch.exp2(e)
        at += n
    return dict(codes=value, scales=scale)
