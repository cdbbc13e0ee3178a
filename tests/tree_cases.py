"""Decoding with drafted trees by its definition, in 64 bits and plain Python, for
the tests: attention along a tree's paths, verification, keeping and reading."""
from __future__ import annotations

import math

import numpy as np

from tests import kv_cases as kc


def random_tree(rng, n, branch=4, back=8):
    """Parents of n tokens: earlier ones, at most `branch` children each."""
    parent, kids = [-1] * min(n, 1), [0] * n
    for j in range(1, n):
        can = [i for i in range(j) if kids[i] < branch][-back:]
        p = int(rng.choice(can))
        parent.append(p)
        kids[p] += 1
    return parent


def sees(parent):
    """[n][n]: row j sees row i, itself or one on its way up."""
    n = len(parent)
    out = np.zeros((n, n), bool)
    for j in range(n):
        i = j
        while i >= 0:
            out[j, i] = True
            i = parent[i]
    return out


def attend(pool, table, lens, parents, q, heads_kv, tokens, codes, scale=None):
    """As kv_cases.attend, along the paths of every request's tree."""
    total, heads, dim = q.shape
    group = heads // heads_kv
    scale = 1 / math.sqrt(dim) if scale is None else scale
    out, mass = np.zeros((total, heads, dim)), np.zeros((total, heads, dim))
    lse, size = np.full((total, heads), -math.inf), np.zeros((total, heads))
    s0 = 0
    for b, parent in enumerate(parents):
        n, length = len(parent), int(lens[b])
        if n and length:
            k, v = kc.request_cache(pool, table[b], length, heads_kv, tokens, dim, codes)
            seen = np.zeros((n, length), bool)
            seen[:, :max(length - n, 0)] = True
            own = sees(parent)
            first = max(n - length, 0)                # tokens before the cache's first are not there
            seen[:, length - n + first:] = own[:, first:]
            for j in range(n):
                t = np.nonzero(seen[j])[0]
                if not len(t):
                    continue
                for h in range(heads):
                    kk, vv = k[t, h // group], v[t, h // group]
                    with np.errstate(invalid="ignore", over="ignore"):
                        s = kk @ q[s0 + j, h] * scale
                        top = s.max()
                        p = np.exp(s - top)
                        lse[s0 + j, h] = top + np.log(p.sum())
                        p /= p.sum()
                        out[s0 + j, h] = p @ vv
                        mass[s0 + j, h] = p @ np.abs(vv)
                        size[s0 + j, h] = (np.abs(kk) @ np.abs(q[s0 + j, h])).max() * abs(scale)
        s0 += n
    return dict(out=out, lse=lse, mass=mass, size=size)


def sound(x):
    """Negative and NaN as 0, infinity as the largest float32."""
    x = np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=float(np.finfo(np.float32).max), neginf=0.0)
    return np.maximum(x, 0.0)


def verify(parent, tokens, u, probs, draft=None):
    """(path, next) of one request: after every refusal the remainder and the draft's
    row, both brought to mass 1, are subtracted."""
    n, vocab = len(parent), probs.shape[1]
    if n == 0:
        return [], -1
    node, path = 0, [0]
    while True:
        w = sound(probs[node])
        d = sound(draft[node]) if draft is not None else None
        fresh = (w if d is None else d).copy()        # 0 for the tokens refused here
        mass, rest, taken = 1.0, 1.0, -1
        for j in range(1, n):
            x = tokens[j]
            if parent[j] != node or not 0 <= x < vocab or not fresh[x] > 0:
                continue
            if d is None:
                if u[j] * mass < fresh[x]:
                    taken = j
                    break
                mass -= fresh[x]
                after = w.copy()
                after[x] = 0
                if math.fsum(after) > 0:
                    w = after
            else:
                if not rest > 0:
                    continue
                if u[j] * d[x] * mass < w[x] * rest:
                    taken = j
                    break
                # w / mass - d / rest, times mass
                after = np.maximum(w - d * (mass / rest), 0)
                left = math.fsum(after)
                rest -= d[x]
                if left > 0:
                    w, mass = after, left
            fresh[x] = 0
        if taken < 0:
            break
        path.append(taken)
        node = taken
    total = math.fsum(w)
    if not total > 0:
        return path, -1
    run = np.cumsum(w.astype(np.longdouble))
    hit = np.nonzero((run > np.longdouble(u[0]) * run[-1]) & (w > 0))[0]
    return path, int(hit[0]) if len(hit) else int(np.nonzero(w > 0)[0][-1])


def keep(pool, table, lens, paths, news, heads, dim, tokens, codes):
    """The pool (a copy of the numpy one) with every request's kept tokens together."""
    was, out = pool, pool.copy()
    views = kc.split_page(out, heads, tokens, dim)
    per = tokens // kc.BLOCK
    for b, (path, n) in enumerate(zip(paths, news)):
        base = int(lens[b]) - n
        go = [k for k, p in enumerate(path) if p != k]
        if not go:
            continue
        first, end = base + go[0], base + len(path)
        k, v = kc.request_cache(was, table[b], int(lens[b]), heads, tokens, dim, codes)
        at = [base + p for p in path[go[0]:]]
        for x, codes_of, scale_of, is_v in ((k, views[0], views[2], False), (v, views[1], views[3], True)):
            for blk in range(first // kc.BLOCK, (end - 1) // kc.BLOCK + 1):
                page, sub = table[b, blk // per], blk % per
                lo, hi = max(first, blk * kc.BLOCK), min(end, (blk + 1) * kc.BLOCK)
                old = lo - blk * kc.BLOCK
                for h in range(heads):
                    c = codes_of[page, h, sub].T if is_v else \
                        codes_of[page, h, sub * kc.BLOCK:(sub + 1) * kc.BLOCK]
                    new = x[at[lo - first:hi - first], h]
                    fin = np.abs(new[np.isfinite(new)])
                    e = kc.exponent(fin.max() if fin.size else 0.0, codes)
                    if old:
                        e_was = int(math.log2(scale_of[page, h, sub]))
                        if e > e_was:
                            c[:old] = kc.nearest(kc.TABLE[codes][c[:old]] * 2.0 ** (e_was - e), codes)
                        e = max(e, e_was)
                    c[old:hi - blk * kc.BLOCK] = kc.nearest(new / 2.0 ** e, codes)
                    scale_of[page, h, sub] = 2.0 ** e
    return out


def same_codes(got, want, heads, tokens, dim, codes):
    """Pools alike, either sign of zero and of NaN being the same value."""
    n = 2 * heads * tokens * dim
    a, b = got[:, :n].copy(), want[:, :n].copy()
    if codes == kc.E4M3:
        for x in (a, b):
            x[x == 0x80] = 0
            x[x == 0xff] = 0x7f
    return np.array_equal(a, b) and np.array_equal(got[:, n:], want[:, n:])
