"""Key/value cache calls refuse bad arguments on the host: nothing here reaches
a GPU."""
import ctypes
import errno

import numpy as np
import pytest
import torch

import memory_dma_descriptor_amd as dd
from tests import kv_cases as kc

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


BAD_CACHES = [dict(pool=NULL), dict(pool=P + 8), dict(table=NULL), dict(lens=NULL),
              dict(lens=P + 2), dict(npages=1 << 31), dict(rows=1 << 24), dict(width=1 << 27),
              dict(kv_heads=0), dict(kv_heads=1025), dict(page_tokens=8), dict(page_tokens=48),
              dict(page_tokens=2048), dict(dim=0), dict(dim=96), dict(dim=512), dict(codes=2)]


def test_page_bytes():
    for h in (1, 3, 8):
        for t in (16, 64, 1024):
            for d in (64, 128, 256):
                assert dd.kv_page_bytes(h, t, d) == kc.page_bytes(h, t, d)
    for bad in ((0, 16, 64), (1, 15, 64), (1, 24, 64), (1, 16, 80), (1024, 1024, 256 * 4)):
        assert dd.kv_page_bytes(*bad) == 0


@no_gpu_only
@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_bad_caches(bad):
    lib = dd.lib()
    need = 1 << 40
    assert lib.dmadesc_kv_check(cache(**bad), P, 4, 0, P, NULL) == EINVAL
    assert lib.dmadesc_kv_append(cache(**bad), P, 128, 64, P, 128, 64, P, 4, 0, NULL) == EINVAL
    assert lib.dmadesc_kv_attend(cache(**bad), P, 256, 64, P, 4, 4, 0, 1, 0.0, P, P, P, need,
                                 NULL) == EINVAL


@no_gpu_only
def test_append_arguments():
    f = dd.lib().dmadesc_kv_append
    ok = [cache(), P, 128, 64, P, 128, 64, P, 4, 0, NULL]
    for k, bad in [(0, NULL), (1, NULL), (1, P + 8), (2, 4), (2, -8), (3, 12), (4, NULL),
                   (4, P + 2), (5, 1), (6, 7), (7, NULL), (8, 1 << 31), (9, 3)]:
        args = list(ok)
        args[k] = bad
        assert f(*args) == EINVAL, (k, bad)
    assert f(*[0 if i == 8 else x for i, x in enumerate(ok)]) == 0          # nothing to do
    assert f(cache(rows=0, lens=NULL, table=NULL), *ok[1:]) == 0
    assert f(cache(npages=0, pool=NULL), *ok[1:]) == 0


@no_gpu_only
def test_attend_arguments():
    lib = dd.lib()
    size = lib.dmadesc_kv_attend_workspace_bytes
    need = size(4, 2, 4, 2, 64, 128, 32)
    assert need > 0 and need % 256 == 0
    assert size(4, 2, 4, 2, 64, 4, 32) == 0                   # 128 tokens are never split
    ok = [cache(width=128), P, 256, 64, P, 4, 4, 0, 1, 0.0, P, P, P, need, NULL]
    for k, bad in [(0, NULL), (1, NULL), (1, P + 8), (2, 4), (2, -8), (3, 12), (4, NULL),
                   (5, 1 << 31), (6, 0), (6, 3), (7, 2), (8, 2), (9, float("nan")), (10, NULL),
                   (10, P + 8), (11, P + 1), (12, NULL), (12, P + 16), (13, need - 1)]:
        args = list(ok)
        args[k] = bad
        assert lib.dmadesc_kv_attend(*args) == EINVAL, (k, bad)
    assert lib.dmadesc_kv_attend(*[0 if i == 5 else x for i, x in enumerate(ok)]) == 0
    for bad in ((0, 2, 4, 2, 64, 4, 32), (4, 0, 4, 2, 64, 4, 32), (4, 2, 3, 2, 64, 4, 32),
                (4, 2, 4, 2, 80, 4, 32), (4, 2, 4, 2, 64, 4, 33), (1 << 31, 2, 4, 2, 64, 4, 32)):
        assert lib.dmadesc_kv_attend_workspace_bytes(*bad) == 0, bad


@no_gpu_only
def test_page_call_arguments():
    lib = dd.lib()
    state = [P, 8, P, P, 2, 4, 32]
    bad_state = [(0, NULL), (1, 1 << 31), (2, NULL), (3, NULL), (4, 1 << 24), (5, 1 << 27), (6, 8),
                 (6, 48)]
    need = dd.workspace_bytes(dd.OP_KV_RESERVE, 8, 2)
    calls = [(lib.dmadesc_kv_free, [P, NULL, 2, P, NULL], [(7, NULL), (9, 1 << 24), (10, NULL)]),
             (lib.dmadesc_kv_fork, [P, P, 2, P, NULL],
              [(7, NULL), (8, NULL), (9, 1 << 24), (10, NULL)]),
             (lib.dmadesc_kv_reserve, [P, P, 2, P, P, P, P, need, NULL],
              [(7, NULL), (8, NULL), (9, 1 << 24), (10, NULL), (11, NULL), (12, NULL), (13, NULL),
               (13, P + 8), (14, need - 1)])]
    for f, rest, bad_rest in calls:
        for k, bad in bad_state + bad_rest:
            args = state + rest
            args[k] = bad
            assert f(*args) == EINVAL, (f, k, bad)
        args = state + rest
        args[9] = 0
        assert f(*args) == 0
    need = dd.workspace_bytes(dd.OP_KV_COMPACT, 8)
    ok = [P, 8, P, 2, 4, P, P, P, P, need, NULL]
    for k, bad in [(0, NULL), (1, 1 << 31), (2, NULL), (3, 1 << 24), (5, NULL), (6, NULL),
                   (7, NULL), (8, NULL), (8, P + 64), (9, need - 1)]:
        args = list(ok)
        args[k] = bad
        assert lib.dmadesc_kv_compact(*args) == EINVAL, (k, bad)
    ok = [P, 8, 4096, P, P, 4, NULL, NULL]
    for k, bad in [(0, NULL), (0, P + 4), (1, 1 << 31), (2, 0), (2, 4100), (2, 1 << 31), (3, NULL),
                   (4, NULL), (5, 1 << 31)]:
        args = list(ok)
        args[k] = bad
        assert lib.dmadesc_kv_copy_pages(*args) == EINVAL, (k, bad)
    assert lib.dmadesc_kv_copy_pages(P, 8, 4096, P, P, 0, NULL, NULL) == 0


def test_workspaces_grow_with_their_sizes():
    ws = dd.workspace_bytes
    assert ws(dd.OP_KV_RESERVE, 1 << 31, 1) == 0 and ws(dd.OP_KV_COMPACT, 1 << 31) == 0
    assert 0 < ws(dd.OP_KV_RESERVE, 0, 1) < ws(dd.OP_KV_RESERVE, 10000, 1) \
        < ws(dd.OP_KV_RESERVE, 10000, 5000)
    assert 0 < ws(dd.OP_KV_COMPACT, 0) < ws(dd.OP_KV_COMPACT, 10000)
    # a bit of every page, three words of every slot; every page's mover number
    assert ws(dd.OP_KV_RESERVE, 10000, 5000) > 1250 + 60000 and ws(dd.OP_KV_COMPACT, 10000) > 40000


def test_binding_refuses_wrong_tensors():
    pool = torch.zeros((4, dd.kv_page_bytes(2, 16, 64)), dtype=torch.uint8)
    table = torch.zeros((1, 4), dtype=torch.int32)
    lens = torch.zeros(1, dtype=torch.int32)
    start = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):                       # host tensors
        dd.kv_attend(q, start, pool, table, lens, 2, 16)
    with pytest.raises(ValueError):
        dd.kv_append(q, q, start, pool, table, lens, 16)
    with pytest.raises(ValueError):                       # a pool of other pages
        dd.kv_attend(q, start, pool, table, lens, 2, 32)
    with pytest.raises(ValueError):
        dd.kv_check(None, 0, pool, table.flatten(), lens, 2, 16, 64)
    with pytest.raises(ValueError):
        dd.kv_copy_pages(pool.flatten(), lens, lens)
    for f in (dd.kv_free, ):
        with pytest.raises(ValueError):
            f(lens, table, lens, lens, 16)


# ------------------------------------------------- the oracle against itself ---

def test_codes_of_the_oracle():
    t = kc.TABLE[kc.E4M3]
    assert t[0x7e] == 448 and t[1] == 2.0 ** -9 and np.isnan(t[0x7f]) and t[0xfe] == -448
    for codes in (kc.E4M3, kc.INT8):
        vals = kc.TABLE[codes]
        keep = np.isfinite(vals) & (np.abs(vals) <= kc.TOP[codes])
        b = np.arange(256, dtype=np.uint8)[keep]
        assert np.array_equal(kc.nearest(vals[keep], codes), b)       # codes are fixed points
    assert kc.nearest([17.0], kc.E4M3)[0] == kc.nearest([16.0], kc.E4M3)[0]       # tie to even
    assert kc.nearest([19.0], kc.E4M3)[0] == kc.nearest([20.0], kc.E4M3)[0]
    assert kc.nearest([2.5], kc.INT8)[0] == 2 and kc.nearest([np.inf], kc.INT8)[0] == 127
    # e4m3 against torch's own conversion
    x = torch.randn(4096) * 100
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kc.nearest(x.double().numpy(), kc.E4M3), want)


def test_exponent_borders():
    for codes in (kc.E4M3, kc.INT8):
        top = kc.TOP[codes]
        assert kc.exponent(top, codes) == 0 and kc.exponent(np.nextafter(top, 1e9), codes) == 1
        assert kc.exponent(top / 2, codes) == -1 and kc.exponent(0.0, codes) == kc.E_MIN


def test_reserve_of_the_oracle_by_hand():
    refs = np.array([1, 2, 0, 0, 0], np.int32)
    table = np.array([[0, 1, -1], [0, 1, -1]], np.int32)
    refs[0] = 2
    lens = np.array([20, 20], np.int32)
    src, dst, st = kc.reserve(refs, table, lens, [0, 1], [1, 13], 16)
    assert list(src) == [1, 1] and list(dst) == [2, 3] and list(st) == [0, 0]
    assert table.tolist() == [[0, 2, -1], [0, 3, 4]] and refs.tolist() == [2, 0, 1, 1, 1]
    assert lens.tolist() == [21, 33]
