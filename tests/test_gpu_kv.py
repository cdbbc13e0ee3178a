"""The paged 8-bit key/value cache on the GPU against its definition in 64 bits
(tests/kv_cases.py): codes, scales and page states exactly, attention within
bounds that count its roundings."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import memory_dma_descriptor_amd as dd
from tests import kv_cases as kc
from tests.gpu_cases import say

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def starts(news):
    return np.concatenate([[0], np.cumsum(news)]).astype(np.int32)


def make_table(rng, lens, tokens, npages, spare=2):
    """Every request's pages in shuffled order, -1 past its last."""
    need = [kc.columns(n, tokens) for n in lens]
    width = max(max(need, default=0) + spare, 1)
    order = rng.permutation(npages).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    assert at <= npages
    return table


def random_pool(rng, npages, heads, tokens, dim, codes, exps=(-7, -4), garbage=0x55):
    """Pages of random finite codes and scales 2^exps."""
    pool = np.full((npages, kc.page_bytes(heads, tokens, dim)), garbage, np.uint8)
    n, nb = heads * tokens * dim, tokens // 16
    x = rng.integers(0, 256, (npages, 2 * n), dtype=np.uint8)
    if codes == kc.E4M3:
        x = kc.nearest(rng.standard_normal((npages, 2 * n)).astype(np.float32) * 60, codes)
    pool[:, :2 * n] = x
    e = rng.integers(exps[0], exps[1] + 1, (npages, 2 * heads * nb)).astype(np.float32)
    pool[:, 2 * n:2 * n + 8 * heads * nb] = np.exp2(e).astype(np.float32).view(np.uint8)
    return pool


# ------------------------------------------------------------------ append ---

def check_append(lens, news, heads, tokens, dim, codes, dtype, seed=0, edit=None, strided=True):
    rng = np.random.default_rng(seed)
    npages = sum(kc.columns(n, tokens) for n in lens) + 3
    pool = random_pool(rng, npages, heads, tokens, dim, codes)
    table = make_table(rng, lens, tokens, npages)
    total = int(sum(news))
    both = torch.from_numpy(rng.standard_normal((total, 2 * heads, dim)).astype(np.float32))
    both[:, :, ::13] *= 6
    if edit:
        edit(both)
    both = both.to(TYPES[dtype]).cuda()
    k, v = both[:, :heads], both[:, heads:]
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    want = kc.append(pool, table, lens, starts(news), k.double().cpu().numpy(),
                     v.double().cpu().numpy(), tokens, codes)
    dev_pool = torch.from_numpy(pool).cuda()
    dd.kv_append(k, v, i32(starts(news)), dev_pool, i32(table), i32(lens), tokens, codes=codes)
    got = dev_pool.cpu().numpy()
    n = 2 * heads * tokens * dim
    a, b = got[:, :n].copy(), want[:, :n].copy()
    if codes == kc.E4M3:                              # either sign of zero and of NaN is the same value
        for x in (a, b):
            x[x == 0x80] = 0
            x[x == 0xff] = 0x7f
    assert np.array_equal(got[:, n:], want[:, n:]), "scales or padding"
    assert np.array_equal(a, b), "codes"


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("dim,dtype,heads,tokens", [(64, "bf16", 3, 16), (128, "fp16", 2, 32),
                                                    (256, "fp32", 1, 64), (128, "bf16", 5, 128),
                                                    (64, "fp32", 2, 1024), (256, "fp16", 2, 16)])
def test_append(codes, dim, dtype, heads, tokens):
    say(f"append {codes} {dim} {dtype} {heads} {tokens}")
    check_append([1, 17, 33, 5, 16, 100, 47, 64], [1, 1, 33, 0, 16, 71, 3, 1], heads, tokens, dim,
                 codes, dtype)


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
def test_append_many_requests(codes):
    # More requests than one probe of the search sees, with empty ones among them.
    rng = np.random.default_rng(5)
    news = rng.integers(0, 4, 150)
    check_append(list(news + rng.integers(0, 40, 150)), list(news), 1, 16, 64, codes, "bf16")


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
def test_append_values_out_of_the_ordinary(codes):
    def edit(x):
        x[0] = 0                                      # a block of zeros: the least scale
        x[1, 0, 3], x[1, 1, 5], x[2, 2, 0] = float("inf"), float("-inf"), float("nan")
        x[3] *= 1e30                                  # the scale grows over earlier tokens
        x[4] *= 1e-30                                 # below the least scale
        x[5, :, :] = 448.0 * 2.0 ** -3                # exactly a border of the scale
        x[5, :, 1] = 127.0 * 2.0 ** -2
        x[6, 0, :] = float("nan")
    check_append([1, 20, 30, 19, 18, 33, 16, 7], [1] * 8, 2, 16, 64, codes, "fp32", edit=edit,
                 strided=False)


def test_append_refuses_and_spares_bad_pages():
    heads, tokens, dim = 2, 16, 64
    rng = np.random.default_rng(1)
    pool = torch.from_numpy(random_pool(rng, 6, heads, tokens, dim, kc.E4M3)).cuda()
    before = pool.clone()
    k = torch.randn((4, heads, dim), device="cuda", dtype=torch.bfloat16)
    lens = i32([5, 20, 40, 3])
    table = i32([[6, -1, -1], [0, -7, -1], [1, 2, 1 << 30], [3, -1, -1]])
    start = i32([0, 1, 2, 3, 4])
    with pytest.raises(dd.DmadescRefused) as e:
        dd.kv_append(k, k, start, pool, table, lens, tokens)
    assert e.value.out["status"].tolist() == [dd.KV_EPAGE] * 3 + [dd.KV_OK]
    dd.kv_append(k, k, start, pool, table, lens, tokens, check=False)
    torch.cuda.synchronize()
    same = (pool == before).all(1).tolist()
    assert same == [True, True, True, False, True, True]       # only the good request's page
    for lens_, start_ in (([2, 1, 1, 0], [0, 3, 3, 3, 4]), ([-1, 1, 1, 1], [0, 0, 1, 2, 4]),
                          ([1, 1, 1, 49], [0, 1, 2, 3, 4]), ([1, 1, 1, 1], [0, 2, 1, 3, 4])):
        table = i32([[0, 1, 2], [3, -1, -1], [4, -1, -1], [5, 1, 0]])
        st = dd.kv_check(i32(start_), 4, pool, table, i32(lens_), heads, tokens, dim, appending=True)
        assert dd.KV_EINVAL in st.tolist()
        dd.kv_append(k, k, i32(start_), pool, table, i32(lens_), tokens, check=False)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ attend ---

def check_attend(lens, news, kv, group, tokens, dim, codes, dtype, causal=True, seed=0, exps=(-7, -4),
                 q_scale=1.0, scale=None, spoil=None, extra_width=2):
    rng = np.random.default_rng(seed)
    npages = sum(kc.columns(n, tokens) for n in lens) + 1
    pool = random_pool(rng, npages, kv, tokens, dim, codes, exps)
    table = make_table(rng, lens, tokens, npages, extra_width)
    total, heads = int(sum(news)), kv * group
    wide = torch.from_numpy(rng.standard_normal((total, heads + 1, dim)).astype(np.float32) * q_scale)
    q = wide.to(TYPES[dtype]).cuda()[:, :heads]         # a strided view
    if spoil:
        spoil(pool, table, q)
    ref = kc.attend(pool, table, lens, starts(news), q.double().cpu().numpy(), kv, tokens, codes,
                    causal, scale)
    # What lies past the lengths is spoiled only now: it must not count.
    n = kv * tokens * dim
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
    assert n
    r = dd.kv_attend(q, i32(starts(news)), torch.from_numpy(dirty).cuda(), i32(table), i32(lens), kv,
                     tokens, codes=codes, causal=causal, scale=scale)
    out, lse = r["out"].double().cpu().numpy(), r["lse"].double().cpu().numpy()
    bound, lse_bound = kc.attend_bounds(ref, dim, max(lens), q.dtype)
    empty = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(lse), empty)
    assert (out[empty] == 0).all()
    nan = np.isnan(ref["out"])
    assert np.array_equal(np.isnan(out), nan), "NaN where the definition has it, and nowhere else"
    with np.errstate(invalid="ignore"):
        d = np.abs(out - ref["out"]) / bound
        dl = np.abs(lse - ref["lse"]) / lse_bound
    say(f"  worst out {np.nanmax(d, initial=0):.3f}, lse {np.nanmax(dl, initial=0):.3f} of the bound")
    assert np.nanmax(d, initial=0) <= 1
    assert np.nanmax(dl, initial=0) <= 1
    assert np.array_equal(np.isnan(lse), np.isnan(ref["lse"]))
    return r


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "bf16"), (256, "bf16"), (64, "fp16"),
                                       (128, "fp16"), (256, "fp16")])
@pytest.mark.parametrize("news,group,tokens", [(1, 4, 64), (1, 1, 16), (5, 7, 32), (40, 3, 16),
                                               (1, 20, 128)])
def test_attend(codes, dim, dtype, news, group, tokens):
    say(f"attend {codes} {dim} {dtype} news {news} group {group} tokens {tokens}")
    lens = [news, 63 + news, 64, 200, 129]
    check_attend(lens, [min(news, n) for n in lens], 2, group, tokens, dim, codes, dtype)


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_empty_requests_and_rows(codes, causal):
    # Lengths of zero, requests without new tokens, more new tokens than cached
    # ones (causal: the first rows see nothing).
    say(f"attend empty {codes} {causal}")
    check_attend([0, 5, 1, 0, 70, 16], [3, 0, 4, 0, 1, 40], 3, 2, 16, 64, codes, "bf16", causal=causal)
    check_attend([0], [2], 1, 1, 16, 128, codes, "fp16", causal=causal)


@pytest.mark.parametrize("kv,group,dim,length,news", [(1, 1, 128, 30000, 1), (2, 8, 64, 9001, 3),
                                                      (1, 4, 256, 5000, 1), (1, 2, 128, 3333, 100)])
@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
def test_attend_split_over_workgroups(kv, group, dim, length, news, codes):
    say(f"attend long {codes} {kv} {group} {dim} {length} {news}")
    check_attend([length, 40], [news, 1], kv, group, 16, dim, codes, "bf16", exps=(-8, -6))


def test_attend_many_requests():
    # More requests than threads of a workgroup, lengths 0..120.
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 120, 600)
    news = np.minimum(rng.integers(0, 3, 600), 2)
    check_attend(list(lens), list(news), 1, 2, 16, 64, kc.INT8, "fp16")


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
def test_attend_a_chunk_among_single_tokens(codes):
    # Few rows on the average and one request of many: both kernels and the join
    # share the requests. Requests of 32 and 33 tokens lie on either side.
    lens = [5 + 7 * i for i in range(60)] + [900, 3000, 64, 65, 400]
    news = [1] * 60 + [600, 1, 32, 33, 0]
    check_attend(lens, news, 1, 2, 32, 64, codes, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
def test_attend_scales_far_apart(dtype, codes):
    # Scales over 2^-64..2^3, peaked and flat scores.
    check_attend([300, 77], [1, 4], 2, 2, 32, 64, codes, dtype, exps=(-64, 3), q_scale=0.05)
    check_attend([300, 77], [1, 4], 2, 2, 32, 64, codes, dtype, exps=(-40, -30))
    check_attend([300, 77], [20, 4], 2, 2, 32, 128, codes, dtype, scale=-0.3)
    check_attend([3000], [1], 1, 2, 16, 128, codes, dtype, scale=1e-6)


@pytest.mark.parametrize("news", [6, 90])
def test_attend_nan_codes(news):
    # A NaN among the seen values reaches its dimension of the rows that see its
    # token and no other; NaN keys and queries reach whole rows.
    def spoil(pool, table, q):
        kcodes, vcodes, _, _ = kc.split_page(pool, 2, 16, 64)
        at = lambda b, t: (table[b, t // 16], t % 16)                       # noqa: E731
        p, t = at(0, 200 - news + news // 2)
        vcodes[p, 1, 0, 7, t] = 0x7f
        vcodes[p, 0, 0, 63, t] = 0xff
        p, t = at(0, 199)
        vcodes[p, 0, 0, 0, t] = 0xff
        p, t = at(1, 100 - news + 3)
        kcodes[p, 0, t, 9] = 0x7f
        p, t = at(2, 5)
        vcodes[p, 0, 0, 20, t] = 0x7f
        q[2 * news + 1, 1, 3] = float("nan")
    check_attend([200, 100, 120], [news] * 3, 2, 3, 16, 64, kc.E4M3, "bf16", spoil=spoil)


def test_attend_refuses_and_spares_bad_pages():
    heads, tokens, dim = 1, 16, 64
    rng = np.random.default_rng(1)
    pool = torch.from_numpy(random_pool(rng, 6, heads, tokens, dim, kc.E4M3)).cuda()
    q = torch.randn((4, 2, dim), device="cuda", dtype=torch.bfloat16)
    lens, start = i32([5, 20, 40, 3]), i32([0, 1, 2, 3, 4])
    table = i32([[6, -1, -1], [0, -7, -1], [1, 2, 1 << 30], [3, -1, -1]])
    with pytest.raises(dd.DmadescRefused) as e:
        dd.kv_attend(q, start, pool, table, lens, heads, tokens)
    assert e.value.out["status"].tolist() == [dd.KV_EPAGE] * 3 + [dd.KV_OK]
    r = dd.kv_attend(q, start, pool, table, lens, heads, tokens, check=False)
    good = dd.kv_attend(q[3:], i32([0, 1]), pool, table[3:].contiguous(), lens[3:].contiguous(), heads,
                        tokens)
    assert torch.equal(r["out"][3:], good["out"])
    # Orders and lengths that the host cannot see: refused by the check, harmless without it.
    for lens_, start_ in (([-5, 1, 1, 1], [0, 1, 2, 3, 4]), ([49, 1, 1, 1], [0, 1, 2, 3, 4]),
                          ([9, 9, 9, 9], [0, 4, 0, 4, 4]), ([9, 9, 9, 9], [0, -3, 900, 5, 4]),
                          ([9, 9, 9, 9], [1, 2, 3, 4, 4])):
        st = dd.kv_check(i32(start_), 4, pool, table, i32(lens_), heads, tokens, dim)
        assert dd.KV_EINVAL in st.tolist()
        dd.kv_attend(q, i32(start_), pool, table, i32(lens_), heads, tokens, check=False)
    torch.cuda.synchronize()


@pytest.mark.parametrize("codes", [kc.E4M3, kc.INT8])
def test_attend_many_rows_spares_bad_pages(codes):
    # Prompts whose table names pages outside the pool, beside a good one.
    tokens, dim = 16, 128
    rng = np.random.default_rng(4)
    pool = torch.from_numpy(random_pool(rng, 12, 1, tokens, dim, codes)).cuda()
    q = torch.randn((150, 2, dim), device="cuda", dtype=torch.bfloat16)
    lens, start = i32([60, 100, 50]), i32([0, 60, 100, 150])
    table = i32([[-1, 12, 1 << 30, -(1 << 31)] + [-1] * 4, [0, 1, -5, 3, 99, 5, 6] + [-1],
                 [7, 8, 9, 10] + [-1] * 4])
    st = dd.kv_check(start, 150, pool, table, lens, 1, tokens, dim)
    assert st.tolist() == [dd.KV_EPAGE, dd.KV_EPAGE, dd.KV_OK]
    r = dd.kv_attend(q, start, pool, table, lens, 1, tokens, codes=codes, check=False)
    good = dd.kv_attend(q[100:], i32([0, 50]), pool, table[2:].contiguous(), lens[2:].contiguous(), 1,
                        tokens, codes=codes)
    assert torch.equal(r["out"][100:], good["out"]) and torch.equal(r["lse"][100:], good["lse"])


def test_attend_past_four_gigabytes():
    # Pages on both sides of 2^32 bytes of the pool.
    heads, tokens, dim = 8, 128, 128
    size = kc.page_bytes(heads, tokens, dim)
    npages = (1 << 32) // size + 40
    rng = np.random.default_rng(2)
    small = random_pool(rng, 40, heads, tokens, dim, kc.INT8)
    pool = torch.empty((npages, size), dtype=torch.uint8, device="cuda")
    where = np.concatenate([np.arange(3), npages - 37 + np.arange(37)]).astype(np.int32)
    pool[torch.from_numpy(where.astype(np.int64)).cuda()] = torch.from_numpy(small).cuda()
    lens, news = [1000, 2049], [2, 1]
    table = make_table(rng, lens, tokens, 40)
    far = np.where(table >= 0, where[np.maximum(table, 0)], -1).astype(np.int32)
    q = torch.randn((3, heads, dim), device="cuda", dtype=torch.float16)
    r = dd.kv_attend(q, i32(starts(news)), pool, i32(far), i32(lens), heads, tokens, codes=dd.KV_INT8)
    s = dd.kv_attend(q, i32(starts(news)), torch.from_numpy(small).cuda(), i32(table), i32(lens), heads,
                     tokens, codes=dd.KV_INT8)
    assert torch.equal(r["out"], s["out"]) and torch.equal(r["lse"], s["lse"])
    k = torch.randn((3, heads, dim), device="cuda", dtype=torch.float16)
    near = torch.from_numpy(small).cuda()
    dd.kv_append(k, k, i32(starts(news)), pool, i32(far), i32(lens), tokens, codes=dd.KV_INT8)
    dd.kv_append(k, k, i32(starts(news)), near, i32(table), i32(lens), tokens, codes=dd.KV_INT8)
    assert torch.equal(pool[torch.from_numpy(where.astype(np.int64)).cuda()], near)


# --------------------------------------------------------- page operations ---

def random_state(rng, rows, tokens, npages, longest, shared=0.3):
    """refs, table, lens with some rows sharing another row's pages."""
    width = kc.columns(longest, tokens) + 3
    table = np.full((rows, width), -1, np.int32)
    lens = np.zeros(rows, np.int32)
    refs = np.zeros(npages, np.int32)
    order = list(rng.permutation(npages))
    for r in range(rows):
        if r and rng.random() < shared:
            o = int(rng.integers(0, r))
            table[r], lens[r] = table[o], lens[o]
        else:
            n = int(rng.integers(0, longest + 1))
            need = kc.columns(n, tokens)
            if need > len(order):
                continue
            table[r, :need] = [order.pop() for _ in range(need)]
            lens[r] = n
        for c in range(kc.columns(int(lens[r]), tokens)):
            refs[table[r, c]] += 1
    return refs, table, lens


def on_gpu(*arrays):
    return [torch.from_numpy(a.copy()).cuda() for a in arrays]


def same_state(gpu, host):
    for name, g, h in zip(("refs", "table", "lens"), gpu, host):
        assert np.array_equal(g.cpu().numpy(), h), name


@pytest.mark.parametrize("rows,tokens,npages,longest", [(1, 16, 4, 40), (12, 16, 100, 90),
                                                        (300, 32, 9000, 700), (900, 64, 5000, 400)])
def test_page_steps(rows, tokens, npages, longest):
    rng = np.random.default_rng(rows)
    state = random_state(rng, rows, tokens, npages, longest)
    gpu = on_gpu(*state)
    for step in range(3):
        say(f"page step {rows} {tokens} {npages} {step}")
        gone = rng.permutation(rows)[:max(1, rows // 5)].astype(np.int32)
        keep = rng.integers(0, longest, len(gone)).astype(np.int32) if step == 1 else None
        kc.free(*state, gone, tokens, keep)
        r = dd.kv_free(*gpu, i32(gone), tokens, keep=None if keep is None else i32(keep))
        assert (r["status"] == dd.KV_OK).all()
        same_state(gpu, state)
        empty = np.nonzero(state[2] == 0)[0][:max(1, rows // 8)]
        full = np.setdiff1d(np.arange(rows), empty)
        parents = rng.choice(full, len(empty)) if len(full) else full
        child = empty[:len(parents)].astype(np.int32)
        kc.fork(*state, parents, child, tokens)
        dd.kv_fork(*gpu, i32(parents), i32(child), tokens)
        same_state(gpu, state)
        slots = rng.permutation(rows).astype(np.int32)
        news = rng.integers(0, 3 * tokens, rows).astype(np.int32)
        src, dst, status = kc.reserve(*state, slots, news, tokens)
        r = dd.kv_reserve(*gpu, i32(slots), i32(news), tokens, check=False)
        assert np.array_equal(r["status"].cpu().numpy(), status)
        assert np.array_equal(r["src"].cpu().numpy(), src)
        assert np.array_equal(r["dst"].cpu().numpy(), dst)
        same_state(gpu, state)
    movers, holes = kc.compact(state[0], state[1])
    r = dd.kv_compact(*gpu, tokens)
    same_state(gpu, state)
    n = len(movers)
    assert int(r["moves"].item()) == n
    src, dst = r["src"].cpu().numpy(), r["dst"].cpu().numpy()
    assert list(src[:n]) == movers and list(dst[:n]) == holes
    assert (src[n:] == -1).all() and (dst[n:] == -1).all()


def test_reserve_many_slots():
    # More slots than running sums fit LDS (1,024 chunks of 256), pages for all
    # but the last, each taking a page or replacing a shared one.
    rows, tokens = 300000, 16
    rng = np.random.default_rng(8)
    table = np.full((rows, 2), -1, np.int32)
    lens = rng.choice([0, 0, 16, 3], rows).astype(np.int32)
    held = np.nonzero(lens)[0]
    npages = len(held) + 100000
    refs = np.zeros(npages, np.int32)
    pages = rng.permutation(npages)[:len(held)].astype(np.int32)
    pages[1::2] = pages[:len(pages) // 2 * 2:2]              # pairs of rows share a page
    table[held, 0] = pages
    np.add.at(refs, pages, 1)
    state = (refs, table, lens)
    gpu = on_gpu(*state)
    slots = rng.permutation(rows).astype(np.int32)
    news = rng.integers(0, 20, rows).astype(np.int32)
    src, dst, status = kc.reserve(*state, slots, news, tokens)
    assert (status == 3).any() and (status == 0).any() and (src >= 0).any()
    r = dd.kv_reserve(*gpu, i32(slots), i32(news), tokens, check=False)
    assert np.array_equal(r["status"].cpu().numpy(), status)
    assert np.array_equal(r["src"].cpu().numpy(), src)
    assert np.array_equal(r["dst"].cpu().numpy(), dst)
    same_state(gpu, state)


def test_reserve_runs_out_and_refuses():
    refs, table, lens = on_gpu(np.array([1, 0, 0, 0, 1], np.int32),
                               np.array([[0, -1, -1, -1], [4, -1, -1, -1], [-1] * 4], np.int32),
                               np.array([10, 16, 0], np.int32))
    with pytest.raises(dd.DmadescRefused) as e:
        dd.kv_reserve(refs, table, lens, i32([0, 1, 2]), i32([16, 40, 1]), 16)
    # one page for row 0; row 1 wants three of the two left; row 2 comes after it
    assert e.value.out["status"].tolist() == [dd.KV_OK, dd.KV_ENOSPC, dd.KV_ENOSPC]
    assert table.tolist() == [[0, 1, -1, -1], [4, -1, -1, -1], [-1] * 4]
    assert lens.tolist() == [26, 16, 0] and refs.tolist() == [1, 1, 0, 0, 1]
    r = dd.kv_reserve(refs, table, lens, i32([-1, 3, 1, 0, 2]), i32([1, 1, 100, -1, 0]), 16, check=False)
    assert r["status"].tolist() == [dd.KV_EINVAL] * 4 + [dd.KV_OK]
    assert lens.tolist() == [26, 16, 0] and refs.tolist() == [1, 1, 0, 0, 1]


def test_page_calls_refuse_rows():
    state = on_gpu(np.array([1, 1, 0], np.int32), np.array([[0, -1], [1, -1], [-1, -1]], np.int32),
                   np.array([3, 16, 0], np.int32))
    r = dd.kv_free(*state, i32([-1, 3, 1 << 30]), 16, check=False)
    assert r["status"].tolist() == [dd.KV_EINVAL] * 3
    r = dd.kv_free(*state, i32([0]), 16, keep=i32([-1]), check=False)
    assert r["status"].tolist() == [dd.KV_EINVAL]
    r = dd.kv_fork(*state, i32([0, 0, 5, -1, 2]), i32([0, 1, 2, 2, 9]), 16, check=False)
    assert r["status"].tolist() == [dd.KV_EINVAL] * 5         # itself, not empty, out of range
    with pytest.raises(dd.DmadescRefused):
        dd.kv_fork(*state, i32([0]), i32([1]), 16)
    assert state[0].tolist() == [1, 1, 0] and state[2].tolist() == [3, 16, 0]
    # A damaged table: pages outside the pool are left alone.
    state[1][0, 0] = 77
    dd.kv_free(*state, i32([0]), 16)
    assert state[0].tolist() == [1, 1, 0]


@pytest.mark.parametrize("npages", [0, 1, 2, 5, 2048, 2049, 7000])
def test_compact_pools(npages):
    rng = np.random.default_rng(npages)
    refs = (rng.random(npages) < 0.4).astype(np.int32) * rng.integers(1, 4, npages).astype(np.int32)
    live = np.nonzero(refs)[0]
    table = np.full((3, max(1, len(live))), -1, np.int32)
    table[1, :len(live)] = rng.permutation(live)
    lens = np.zeros(3, np.int32)
    g = on_gpu(refs, table, lens)
    movers, holes = kc.compact(refs, table)
    r = dd.kv_compact(*g, 16)
    same_state(g, (refs, table, lens))
    n = len(movers)
    assert int(r["moves"].item()) == n and r["src"].tolist() == movers + [-1] * (npages // 2 - n)
    assert r["dst"].tolist() == holes + [-1] * (npages // 2 - n)


@pytest.mark.parametrize("size", [16, 512, 4096 + 512, 16384, 16384 * 3 + 512])
def test_copy_pages(size):
    g = torch.Generator().manual_seed(size)
    pool = torch.randint(0, 256, (40, size), dtype=torch.uint8, generator=g)
    src = [3, -1, 7, 9, 40, 5, 6, 8]
    dst = [20, 21, -1, 22, 23, 5, 1 << 30, 24]
    for count in (None, 0, 4, 8, 99, -3):
        dev = pool.cuda()
        want = pool.clone()
        n = 8 if count is None else max(0, min(8, count))
        for s, d in list(zip(src, dst))[:n]:
            if 0 <= s < 40 and 0 <= d < 40:
                want[d] = pool[s]
        dd.kv_copy_pages(dev, i32(src), i32(dst), count=None if count is None else i32([count]))
        assert torch.equal(dev.cpu(), want), count


# ------------------------------------------------------------ graphs, streams ---

def serving_state(seed=0, rows=6, tokens=16, kv=2, dim=64):
    rng = np.random.default_rng(seed)
    lens = rng.integers(1, 50, rows).astype(np.int32)
    npages = 64
    pool = random_pool(rng, npages, kv, tokens, dim, kc.E4M3)
    table = make_table(rng, lens, tokens, npages, 4)
    refs = np.zeros(npages, np.int32)
    refs[table[table >= 0]] = 1
    return [torch.from_numpy(x).cuda() for x in (pool, refs, table, lens)]


def one_step(pool, refs, table, lens, k, v, q, stream=None):
    """Row 1 ends, row 0 branches into it, all rows take a token and attend."""
    kw = dict(stream=stream, check=False)
    dd.kv_free(refs, table, lens, one_step.gone, 16, **kw)
    dd.kv_fork(refs, table, lens, one_step.parent, one_step.gone, 16, **kw)
    r = dd.kv_reserve(refs, table, lens, one_step.slots, one_step.ones, 16, **kw)
    dd.kv_copy_pages(pool, r["src"], r["dst"], stream=stream)
    dd.kv_append(k, v, one_step.start, pool, table, lens, 16, **kw)
    o = dd.kv_attend(q, one_step.start, pool, table, lens, 2, 16, **kw)
    c = dd.kv_compact(refs, table, lens, 16, stream=stream)
    dd.kv_copy_pages(pool, c["src"], c["dst"], count=c["moves"], stream=stream)
    return o


def step_inputs():
    one_step.gone, one_step.parent = i32([1]), i32([0])
    one_step.slots, one_step.ones, one_step.start = i32(range(6)), i32([1] * 6), i32(range(7))
    g = torch.Generator(device="cuda").manual_seed(4)
    mk = lambda h: torch.randn((6, h, 64), device="cuda", generator=g, dtype=torch.bfloat16)   # noqa: E731
    return mk(2), mk(2), mk(4)


def test_step_in_a_graph():
    k, v, q = step_inputs()
    warm = serving_state()
    one_step(*warm, k, v, q)
    torch.cuda.synchronize()
    eager, captured = serving_state(), serving_state()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = one_step(*captured, k, v, q)
    for replay in range(4):
        say(f"replay {replay}")
        want = one_step(*eager, k, v, q)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert torch.equal(a, b)
        assert torch.equal(want["out"], out["out"]) and torch.equal(want["lse"], out["lse"])
        k.add_(0.5)                                   # eager work between the replays
        assert float(torch.ones(1000, device="cuda").sum()) == 1000


def test_step_on_another_stream():
    k, v, q = step_inputs()
    want_state, state = serving_state(), serving_state()
    want = one_step(*want_state, k, v, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = one_step(*state, k, v, q, stream=side)
    junk = [torch.full((1 << 16,), 7, dtype=torch.uint8, device="cuda") for _ in range(50)]
    side.synchronize()
    assert junk and torch.equal(want["out"], got["out"]) and torch.equal(want["lse"], got["lse"])
    for a, b in zip(want_state, state):
        assert torch.equal(a, b)
