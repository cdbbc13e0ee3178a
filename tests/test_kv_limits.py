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
