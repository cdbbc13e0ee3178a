"""The key/value cache by its definition, in 64 bits and plain Python, for the
tests: page layout, quantisation, attention and the page operations."""
from __future__ import annotations

import math

import numpy as np
import torch

BLOCK = 16
E_MIN = -64
E4M3, INT8 = 0, 1
TOP = {E4M3: 448.0, INT8: 127.0}


def page_bytes(heads, tokens, dim):
    return -(-(2 * heads * tokens * dim + 8 * heads * (tokens // BLOCK)) // 512) * 512


def e4m3_table():
    """Value of each of the 256 e4m3 bytes: sign, 4 exponent bits (bias 7), 3
    mantissa bits; 0x7f and 0xff are NaN and there is no infinity."""
    out = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[b] = math.nan if b & 127 == 127 else x
        if b & 128:
            out[b] = -out[b]
    return out


def int8_table():
    return np.array([b - 256 * (b >> 7) for b in range(256)], np.float64)


TABLE = {E4M3: e4m3_table(), INT8: int8_table()}


def split_page(pool, heads, tokens, dim):
    """K codes [p][H][T][D], V codes [p][H][T/16][D][16], scales [p][H][T/16]
    (K, V) as views of a numpy pool u8[pages][page bytes]."""
    n, nb = heads * tokens * dim, tokens // BLOCK
    k = pool[:, :n].reshape(-1, heads, tokens, dim)
    v = pool[:, n:2 * n].reshape(-1, heads, nb, dim, BLOCK)
    s = pool[:, 2 * n:2 * n + 8 * heads * nb].view(np.float32).reshape(-1, 2, heads, nb)
    return k, v, s[:, 0], s[:, 1]


def exponent(amax, codes):
    """Least e >= E_MIN with amax <= TOP * 2^e."""
    e = E_MIN
    while amax > TOP[codes] * 2.0 ** e:
        e += 1
    return e


_MIDS = {}


def nearest(y, codes):
    """The codes (bytes) nearest to y, ties to even, from the table of values;
    infinities and what lies past the largest code saturate; NaN is the NaN code
    (e4m3, sign kept aside) or 0 (int8)."""
    y = np.asarray(y, np.float64)
    if codes == INT8:
        z = np.clip(np.nan_to_num(y, nan=0.0, posinf=1e30, neginf=-1e30), -127, 127)
        return np.rint(z).astype(np.int8).view(np.uint8)
    mag = np.clip(np.abs(np.nan_to_num(y, nan=0.0, posinf=1e30, neginf=-1e30)), 0, 448.0)
    vals = TABLE[E4M3][:127]                             # ascending, codes 0..126
    hi = np.clip(np.searchsorted(vals, mag), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    dl, dh = mag - vals[lo], vals[hi] - mag
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    out = pick.astype(np.uint8) | (np.signbit(y).astype(np.uint8) << 7)
    return np.where(np.isnan(y), np.uint8(127), out).astype(np.uint8)


def append(pool, table, lens, q_start, k, v, tokens, codes):
    """Writes k, v (numpy float64 [total][H][D]) into a copy of the numpy pool."""
    pool = pool.copy()
    _, heads, dim = k.shape
    kc, vc, ks, vs = split_page(pool, heads, tokens, dim)
    per = tokens // BLOCK
    for b in range(len(lens)):
        s0, s1 = int(q_start[b]), int(q_start[b + 1])
        first, length = int(lens[b]) - (s1 - s0), int(lens[b])
        if s1 == s0:
            continue
        for blk in range(first // BLOCK, (length - 1) // BLOCK + 1):
            page, sub = table[b, blk // per], blk % per
            for h in range(heads):
                for x, c, s in ((k, kc[page, h, sub * BLOCK:(sub + 1) * BLOCK], ks),
                                (v, vc[page, h, sub].T, vs)):
                    old = max(0, first - blk * BLOCK)
                    end = min(BLOCK, length - blk * BLOCK)
                    new = x[s0 + blk * BLOCK + old - first:s0 + blk * BLOCK + end - first, h]
                    fin = np.abs(new[np.isfinite(new)])
                    e = exponent(fin.max() if fin.size else 0.0, codes)
                    if old:
                        was = float(s[page, h, sub])
                        e = max(e, int(math.log2(was)))
                    if old and 2.0 ** e > was:           # earlier codes stand unless the scale grew
                        held = TABLE[codes][c[:old]] * (was / 2.0 ** e)
                        c[:old] = nearest(held, codes)
                    c[old:end] = nearest(new / 2.0 ** e, codes)
                    c[end:] = 0
                    s[page, h, sub] = 2.0 ** e
    return pool


def request_cache(pool, table_row, length, heads, tokens, dim, codes):
    """K, V [length][H][D] in float64 of one request."""
    n = -(-length // tokens)
    kc, vc, ks, vs = split_page(np.ascontiguousarray(pool[table_row[:n]]), heads, tokens, dim)
    rep = lambda s: np.repeat(s.astype(np.float64), BLOCK, axis=2)[..., None]   # noqa: E731
    with np.errstate(invalid="ignore"):
        k = TABLE[codes][kc] * rep(ks)
        v = TABLE[codes][vc].transpose(0, 1, 2, 4, 3).reshape(n, heads, tokens, dim) * rep(vs)
    flat = lambda x: x.transpose(0, 2, 1, 3).reshape(n * tokens, heads, dim)[:length]   # noqa: E731
    return flat(k), flat(v)


def attend(pool, table, lens, q_start, q, heads_kv, tokens, codes, causal, scale=None):
    """dict(out, lse, mass, size): float64 outputs, sum p |V| per output value and
    the largest scale * sum |q||k| of a row (both for error bounds)."""
    total, heads, dim = q.shape
    group = heads // heads_kv
    scale = 1 / math.sqrt(dim) if scale is None else scale
    out = np.zeros((total, heads, dim))
    mass = np.zeros((total, heads, dim))
    lse = np.full((total, heads), -math.inf)
    size = np.zeros((total, heads))
    for b in range(len(lens)):
        s0, s1, length = int(q_start[b]), int(q_start[b + 1]), int(lens[b])
        if length == 0 or s1 == s0:
            continue
        k, v = request_cache(pool, table[b], length, heads_kv, tokens, dim, codes)
        for j in range(s1 - s0):
            upto = length - (s1 - s0) + j + 1 if causal else length
            if upto <= 0:
                continue
            for h in range(heads):
                kk, vv = k[:upto, h // group], v[:upto, h // group]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = kk @ q[s0 + j, h] * scale
                    top = s.max()
                    p = np.exp(s - top)
                    p_sum = p.sum()
                    out[s0 + j, h] = p / p_sum @ vv
                    mass[s0 + j, h] = p / p_sum @ np.abs(vv)
                    lse[s0 + j, h] = top + np.log(p_sum)
                    size[s0 + j, h] = (np.abs(kk) @ np.abs(q[s0 + j, h])).max() * abs(scale)
    return dict(out=out, lse=lse, mass=mass, size=size)


def attend_bounds(ref, dim, longest, dtype):
    """(bound of out, bound of lse) from the roundings made, counted in half
    steps: the probabilities to f16 (eps/2 of f16 each, relative to sum p|V|), the
    output to its type, and f32 below: a dot product of dim terms (dim half
    steps of sum |q||k|, and four for its scaling), one exponential (two half steps
    and its argument's error), a running sum (a half step for each of a lane's
    longest / 4 terms at most, 64 for the joins)."""
    h32 = 2.0 ** -24
    score = (dim + 4) * h32 * ref["size"]
    add = (longest / 4 + 64 + 8) * h32
    lse = score + add + 4 * h32 * np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0))
    rel = 2.0 ** -11 + (2 * score + 2 * add)[..., None] + 4 * 2.0 ** -11 * 2.0 ** -11
    out_half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    err = rel * ref["mass"]
    return err + out_half * (np.abs(ref["out"]) + err) + tiny, lse


# ------------------------------------------------------------ page operations ---

def columns(length, tokens):
    return -(-length // tokens)


def free(refs, table, lens, rows, tokens, keep=None):
    for i, r in enumerate(rows):
        left = 0 if keep is None else int(keep[i])
        new = min(left, int(lens[r]))
        for c in range(columns(new, tokens), columns(int(lens[r]), tokens)):
            refs[table[r, c]] -= 1
        table[r, columns(new, tokens):] = -1
        lens[r] = new


def fork(refs, table, lens, parents, children, tokens):
    for p, c in zip(parents, children):
        table[c] = table[p]
        lens[c] = lens[p]
        for k in range(columns(int(lens[p]), tokens)):
            refs[table[p, k]] += 1


def reserve(refs, table, lens, slots, news, tokens):
    """(src, dst, status), state updated in place; statuses 0, 1 (bad), 3 (full)."""
    before = refs.copy()
    spare = [int(p) for p in np.nonzero(before == 0)[0]]
    src, dst, status, used = [], [], [], 0
    for r, n in zip(slots, news):
        r, n = int(r), int(n)
        src.append(-1)
        dst.append(-1)
        status.append(0)
        if not 0 <= r < len(lens) or n < 0 or lens[r] + n > table.shape[1] * tokens or lens[r] < 0:
            status[-1] = 1
            continue
        have, want = columns(int(lens[r]), tokens), columns(int(lens[r]) + n, tokens)
        shared = n > 0 and lens[r] % tokens != 0 and before[table[r, have - 1]] > 1
        take = want - have + shared
        got = spare[used:used + take]
        used += take
        if len(got) < take:
            status[-1] = 3
            continue
        if shared:
            src[-1], dst[-1] = int(table[r, have - 1]), got[0]
            refs[src[-1]] -= 1
        for i, p in enumerate(got):
            table[r, have - shared + i] = p
            refs[p] = 1
        lens[r] += n
    return np.array(src), np.array(dst), np.array(status)


def compact(refs, table):
    live = int((refs > 0).sum())
    holes = [p for p in range(live) if refs[p] <= 0]
    movers = [p for p in range(live, len(refs)) if refs[p] > 0]
    name = {m: h for m, h in zip(movers, holes)}
    for m, h in name.items():
        refs[h], refs[m] = refs[m], 0
    for i, p in enumerate(table.flat):
        if int(p) in name:
            table.flat[i] = name[int(p)]
    return movers, holes
