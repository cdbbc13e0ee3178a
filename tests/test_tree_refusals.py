"""The calls for drafted trees refuse bad arguments on the host, and their oracles
against hand-made cases: nothing here reaches a GPU."""
import ctypes
import errno

import numpy as np
import pytest
import torch

import memory_dma_descriptor_amd as dd
from tests import kv_cases as kc
from tests import tree_cases as tc

EINVAL = -errno.EINVAL
NULL = None
P = 0x1000       # never dereferenced: every call below is refused before a launch

no_gpu_only = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                 reason="dummy-pointer probes run only without a GPU")


def cache(**kw):
    f = dict(pool=P, table=P, lens=P, npages=8, rows=2, width=4, kv_heads=2, page_tokens=32,
             dim=64, codes=0)
    f.update(kw)
    return ctypes.byref(dd._KvCache(*[f[n] for n, _ in dd._KvCache._fields_]))


BAD_CACHES = [dict(pool=NULL), dict(pool=P + 8), dict(table=NULL), dict(lens=NULL), dict(npages=1 << 31),
              dict(rows=1 << 24), dict(width=1 << 27), dict(kv_heads=0), dict(page_tokens=48), dict(dim=96),
              dict(codes=2)]


def refuses(f, ok, bad):
    for k, x in bad:
        args = list(ok)
        args[k] = x
        assert f(*args) == EINVAL, (f, k, x)


@no_gpu_only
@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches(bad):
    lib = dd.lib()
    c = cache(**bad)
    assert lib.dmadesc_kv_attend_tree(c, P, 256, 64, P, P, 4, 4, 0, 0.0, P, P, P, 1 << 40, NULL) == EINVAL
    assert lib.dmadesc_kv_tree_check(c, P, P, 4, P, NULL) == EINVAL
    assert lib.dmadesc_kv_keep(c, P, P, P, 4, P + 4, P, NULL) == EINVAL
    assert lib.dmadesc_kv_read(c, P, P, 4, 0, P, 128, 64, P, 128, 64, NULL) == EINVAL
    assert lib.dmadesc_kv_read_check(c, P, P, 4, P, NULL) == EINVAL


@no_gpu_only
def test_attend_tree_arguments():
    lib = dd.lib()
    size = lib.dmadesc_kv_attend_tree_workspace_bytes
    need = size(4, 2, 4, 2, 64, 128, 32)
    assert need > 0 and need % 256 == 0 and size(4, 2, 4, 2, 64, 4, 32) == 0
    for bad in ((0, 2, 4, 2, 64, 4, 32), (4, 0, 4, 2, 64, 4, 32), (4, 2, 3, 2, 64, 4, 32), (4, 2, 4, 2, 80, 4, 32)):
        assert size(*bad) == 0, bad
    ok = [cache(width=128), P, 256, 64, P, P, 4, 4, 0, 0.0, P, P, P, need, NULL]
    refuses(lib.dmadesc_kv_attend_tree, ok,
            [(0, NULL), (1, NULL), (1, P + 8), (2, 4), (2, -8), (3, 12), (4, NULL), (5, NULL), (5, P + 2),
             (6, 1 << 31), (7, 0), (7, 3), (8, 2), (9, float("nan")), (9, 3e38), (10, NULL), (10, P + 8),
             (11, P + 1), (12, NULL), (12, P + 16), (13, need - 1)])
    assert lib.dmadesc_kv_attend_tree(*[0 if i == 6 else x for i, x in enumerate(ok)]) == 0
    ok = [cache(), P, P, 4, P, NULL]
    refuses(lib.dmadesc_kv_tree_check, ok, [(1, NULL), (1, P + 1), (2, NULL), (2, P + 2), (3, 1 << 31), (4, NULL)])
    assert lib.dmadesc_kv_tree_check(cache(rows=0, lens=NULL, table=NULL), *ok[1:]) == 0


@no_gpu_only
def test_keep_and_read_arguments():
    lib = dd.lib()
    ok = [cache(), P, P, P, 4, P + 4, P, NULL]
    refuses(lib.dmadesc_kv_keep, ok, [(1, NULL), (1, P + 1), (2, NULL), (2, P + 2), (3, NULL), (3, P + 2),
                                      (4, 1 << 31), (5, NULL), (5, P + 2), (5, P), (6, NULL)])
    assert lib.dmadesc_kv_keep(cache(rows=0, lens=NULL, table=NULL), *ok[1:]) == 0
    assert lib.dmadesc_kv_keep(cache(rows=1 << 22, kv_heads=2), *ok[1:]) == EINVAL            # past a launch
    assert lib.dmadesc_kv_keep(cache(rows=(1 << 22) - 1, kv_heads=2), *ok[1:]) not in (0, EINVAL)
    ok = [cache(), P, P, 4, 0, P, 128, 64, P, 128, 64, NULL]
    refuses(lib.dmadesc_kv_read, ok,
            [(1, P + 1), (2, NULL), (2, P + 2), (3, 1 << 31), (4, 3), (5, NULL), (5, P + 8), (6, 4), (6, -8),
             (7, 12), (8, NULL), (8, P + 2), (9, 1), (10, 7)])
    for zero in ((3, 0),):
        args = list(ok)
        args[zero[0]] = zero[1]
        assert lib.dmadesc_kv_read(*args) == 0
    assert lib.dmadesc_kv_read(cache(rows=0, lens=NULL, table=NULL), *ok[1:]) == 0
    assert lib.dmadesc_kv_read(cache(rows=1 << 22, kv_heads=8), *ok[1:]) == EINVAL
    ok = [cache(), P, P, 4, P, NULL]
    refuses(lib.dmadesc_kv_read_check, ok, [(1, P + 1), (2, NULL), (2, P + 1), (3, 1 << 31), (4, NULL)])


@no_gpu_only
def test_keep_writes_over_none_of_its_inputs():
    lib = dd.lib()
    at = dict(path=0x10000, count=0x20000, q_start=0x30000)
    for same in (P, *at.values()):
        assert lib.dmadesc_kv_keep(cache(), *at.values(), 4, same, P, NULL) == EINVAL
    assert lib.dmadesc_kv_keep(cache(), *at.values(), 4, 0x40000, P, NULL) not in (0, EINVAL)


@no_gpu_only
def test_verify_arguments():
    lib = dd.lib()
    ok = [P, 1000, P, 1000, 1000, 2, P, P, P, 2, 6, P, P, P, P, P, NULL]
    refuses(lib.dmadesc_verify_drafts, ok,
            [(0, NULL), (0, P + 2), (1, -1), (2, P + 1), (3, -8), (4, 0), (4, 1 << 31), (5, 3), (6, NULL),
             (6, P + 2), (7, NULL), (7, P + 1), (8, NULL), (8, P + 2), (9, 1 << 22), (10, 1 << 31), (11, NULL),
             (11, P + 2), (12, NULL), (12, P + 1), (13, NULL), (13, P + 1), (14, NULL), (14, P + 3), (15, NULL)])
    assert lib.dmadesc_verify_drafts(*[0 if i == 9 else x for i, x in enumerate(ok)]) == 0


def test_binding_refuses_wrong_tensors():
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)             # noqa: E731
    pool = torch.zeros((4, dd.kv_page_bytes(2, 16, 64)), dtype=torch.uint8)
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    p = torch.rand((3, 7))
    for f in (lambda: dd.kv_attend_tree(q, i32(2), i32(1), pool, i32(1, 4), i32(1), 2, 16),
              lambda: dd.kv_tree_check(i32(2), i32(1), pool, i32(4), i32(1), 2, 16, 64),
              lambda: dd.verify_drafts(p, i32(3), i32(3), i32(2), torch.rand(3)),          # host tensors
              lambda: dd.verify_drafts(p[0], i32(3), i32(3), i32(2), torch.rand(3)),
              lambda: dd.kv_keep(i32(1), i32(1), i32(2), pool, i32(1, 4), i32(1), 2, 32, 64),
              lambda: dd.kv_read(None, i32(2), 1, pool, i32(1, 4), i32(1), 2, 16, 64)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError, match="scale"):
        dd.kv_attend_tree(q, None, None, None, None, None, 2, 16, scale=1e-50)


# ------------------------------------------------- the oracles against themselves ---

def test_tree_by_hand():
    seen = tc.sees([-1, 0, 0, 1, 2, -1])
    assert [list(np.nonzero(r)[0]) for r in seen] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4], [5]]


def test_verify_by_hand():
    p = np.array([[.5, .25, .25, 0]] * 3)
    d = np.array([[.25, .25, .5, 0]] * 3)
    # u d < p, strictly: .5 * .5 is not less than .25
    assert tc.verify([-1, 0], [0, 2], [0, .49], p[:2], d[:2])[0] == [0, 1]
    assert tc.verify([-1, 0], [0, 2], [0, .5], p[:2], d[:2])[0] == [0]
    # refused: what is left is max(p - d, 0), all of it at token 0
    assert tc.verify([-1, 0], [0, 2], [.99, .5], p[:2], d[:2]) == ([0], 0)
    # its sibling, token 0: w / W = 1 against d / Q = 1/2
    assert tc.verify([-1, 0, 0], [0, 2, 0], [0, .5, .99], p, d)[0] == [0, 2]
    # certain drafts: token 1 refused (u >= 1/4), then token 0 against 1/2 of 3/4
    assert tc.verify([-1, 0, 0], [0, 1, 0], [.99, .25, .66], p) == ([0, 2], 2)
    assert tc.verify([-1, 0, 0], [0, 1, 0], [.99, .25, .67], p) == ([0], 2)
    assert tc.verify([-1, 0], [0, 3], [0.5, 0], p[:2]) == ([0], 1)     # p = 0: passed over


@pytest.mark.parametrize("certain", [False, True])
def test_verify_samples_the_target(certain):
    """Accepted or drawn, the first token after the root follows the target, whatever
    the draft: integrated exactly over u on a fine grid of the tests' numbers would be
    slow, so 20,000 seeded samples, each token within 5 deviations."""
    rng = np.random.default_rng(3)
    p, d = rng.dirichlet(np.ones(5)), rng.dirichlet(np.ones(5))
    n, seen = 20000, np.zeros(5)
    for _ in range(n):
        kids = [1, 3, 4] if certain else list(rng.choice(5, 3, replace=False, p=d))
        probs, draft = np.stack([p] * 4), None if certain else np.stack([d] * 4)
        tokens = [0] + [int(k) for k in kids]
        path, nxt = tc.verify([-1, 0, 0, 0], tokens, rng.random(4), probs, draft)
        seen[tokens[path[1]] if len(path) > 1 else nxt] += 1
    assert (np.abs(seen / n - p) <= 5 * np.sqrt(p * (1 - p) / n)).all()


def test_keep_of_the_oracle_is_append_of_the_values():
    rng = np.random.default_rng(0)
    heads, tokens, dim = 2, 16, 64
    pool = np.zeros((4, kc.page_bytes(heads, tokens, dim)), np.uint8)
    table = np.array([[2, 0, 3]], np.int32)
    x = rng.standard_normal((40, heads, dim))
    pool = kc.append(pool, table, [40], [0, 40], x, x[::-1], tokens, kc.INT8)
    path = [0, 2, 3, 9, 20, 21]                       # of 25 new tokens, places 15 ..
    got = tc.keep(pool, table, [40], [path], [25], heads, dim, tokens, kc.INT8)
    k, v = kc.request_cache(pool, table[0], 40, heads, tokens, dim, kc.INT8)
    at = [15 + p for p in path[1:]]
    want = kc.append(pool, table, [21], [0, 5], k[at], v[at], tokens, kc.INT8)
    kg, vg = kc.request_cache(got, table[0], 21, heads, tokens, dim, kc.INT8)
    kw, vw = kc.request_cache(want, table[0], 21, heads, tokens, dim, kc.INT8)
    assert np.array_equal(kg, kw) and np.array_equal(vg, vw)
    assert np.array_equal(got[3], pool[3]) and np.array_equal(got[2], pool[2])
