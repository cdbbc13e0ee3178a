"""Limits of the cache's calls, as the host checks them: nothing here reaches a
GPU."""
import ctypes
import errno

import pytest
import torch

import memory_dma_descriptor_amd as dd

EINVAL = -errno.EINVAL
P = 0x1000       # never dereferenced

no_gpu_only = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                 reason="dummy-pointer probes run only without a GPU")


def cache(**kw):
    f = dict(pool=P, table=P, lens=P, npages=8, rows=2, width=4, kv_heads=2, page_tokens=32,
             dim=64, codes=0)
    f.update(kw)
    return ctypes.byref(dd._KvCache(*[f[n] for n, _ in dd._KvCache._fields_]))


def attend(cache_, total=4, heads=4, scale=0.0, tok=256, head=64):
    return dd.lib().dmadesc_kv_attend(cache_, P, tok, head, P, total, heads, 0, 1, scale, P, P, P, 1 << 40,
                                      None)


@no_gpu_only
def test_factors_that_f32_cannot_hold():
    for bad in (float("inf"), -float("inf"), 3e38, -3e38):
        assert attend(cache(), scale=bad) == EINVAL, bad
    for good in (2e38, -2e38, 1e-45):
        assert attend(cache(), scale=good) != EINVAL, good


@pytest.mark.parametrize("scale", [1e-50, -1e-46, 1e39])
def test_binding_refuses_factors_that_f32_cannot_hold(scale):
    # 1e-50 would reach the library as 0, which means 1 / sqrt(dim).
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="scale"):
        dd.kv_attend(q, None, None, None, None, 2, 16, scale=scale)


@no_gpu_only
def test_append_sizes_past_a_launch():
    # A launch holds 2^24 - 1 workgroups of 256 threads; four waves of one share a
    # workgroup, two for each block of 16 tokens and head.
    f = dd.lib().dmadesc_kv_append

    def append(rows, heads, total):
        return f(cache(rows=rows, kv_heads=heads, page_tokens=16), P, 8, 8, P, 8, 8, P, total, 0, None)

    top = (1 << 24) - 1
    for bad in ((top, 1024, 1), (top, 256, 1), (1 << 22, 8, 1), (1 << 22, 1024, 16), (1, 1024, 1 << 30),
                (1 << 23, 2, 16)):
        assert append(*bad) == EINVAL, bad
    for good in ((1 << 22, 3, 1), (1, 1024, 1 << 18), ((1 << 23) - 1, 2, 15)):
        assert append(*good) not in (0, EINVAL), good      # gets as far as a launch


@no_gpu_only
def test_attend_sizes_past_a_launch():
    size = dd.lib().dmadesc_kv_attend_workspace_bytes
    # rows, heads = kv_heads, total, width in pages of 16 tokens (256 are split, 8 not)
    for rows, heads, total, width in (((1 << 24) - 1, 1024, 16, 256), ((1 << 24) - 1, 256, 1, 256),
                                      (3 << 20, 8, 16, 256), (1 << 22, 1024, 16, 256),
                                      (1, 64, 1 << 24, 256)):
        assert size(total, rows, heads, heads, 64, width, 16) == 0
        for w in (width, 8) if rows > 1 else (width,):
            assert attend(cache(rows=rows, kv_heads=heads, page_tokens=16, width=w), total, heads) == EINVAL
    for rows, heads, total, width in ((1 << 20, 8, 16, 256), (1, 64, 1 << 20, 256),
                                      (1, 64, 1 << 24, 8)):
        assert (size(total, rows, heads, heads, 64, width, 16) > 0) == (width > 16)
        assert attend(cache(rows=rows, kv_heads=heads, page_tokens=16, width=width), total, heads) \
            not in (0, EINVAL)


@no_gpu_only
def test_strides_of_single_tokens_and_heads_mean_nothing():
    lib = dd.lib()

    def append(total, heads, tok, head):
        return lib.dmadesc_kv_append(cache(kv_heads=heads), P, tok, head, P, tok, head, P, total, 0, None)

    for f in (append, lambda total, heads, tok, head: attend(cache(kv_heads=heads), total, heads, 0.0, tok,
                                                              head)):
        for tok in (3, -8, 12):
            assert f(1, 2, tok, 64) not in (0, EINVAL)       # one token: gets as far as a launch
            assert f(2, 2, tok, 64) == EINVAL
            assert f(2, 1, 64, tok) not in (0, EINVAL)       # one head
            assert f(2, 2, 64, tok) == EINVAL
