"""Calls given a stream of their own take the memory of their results and
workspaces in that stream's order: a block that the current stream has freed may
still be used by work queued there, which the other stream does not wait for."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import memory_dma_descriptor_amd as dd
from tests.test_gpu_kv import i32

pytestmark = pytest.mark.gpu


def stream_of(t):
    """The stream whose memory holds a tensor (the default stream is 0)."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not of the allocator")


def ordered(call):
    """Checks call's results, a dict or tensor, with a side stream and without one;
    returns them."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    results = []
    for stream in (None, side):
        freed = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (512, 4096, 1 << 16, 1 << 21)]
        del freed                                     # what the current stream would hand out next
        r = call(stream)
        torch.cuda.synchronize()
        for t in r.values() if isinstance(r, dict) else [r]:
            assert stream_of(t) == (0 if stream is None else stream.cuda_stream)
        results.append(r)
    return results


def cache_state():
    pool = torch.zeros((8, dd.kv_page_bytes(2, 16, 64)), dtype=torch.uint8, device="cuda")
    return pool, i32([2, 1, 1, 0, 0, 0, 0, 0]), i32([[0, 1, -1], [0, 2, -1], [-1] * 3]), i32([20, 30, 0])


def test_cache_calls():
    pool, refs, table, lens = cache_state()
    q = torch.ones((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    start = i32([0, 1, 2, 2])
    a, b = ordered(lambda s: dd.kv_attend(q, start, pool, table, lens, 2, 16, stream=s))
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    ordered(lambda s: dd.kv_check(start, 2, pool, table, lens, 2, 16, 64, stream=s))
    ordered(lambda s: dd.kv_compact(refs, table, lens, 16, stream=s))
    state = []

    def fresh(call):
        def run(s):
            state[:] = cache_state()[1:]
            torch.cuda.synchronize()
            return call(s)
        return run
    ordered(fresh(lambda s: dd.kv_free(*state, i32([1]), 16, stream=s)))
    ordered(fresh(lambda s: dd.kv_fork(*state, i32([0]), i32([2]), 16, stream=s)))
    ordered(fresh(lambda s: dd.kv_reserve(*state, i32([0, 2]), i32([20, 5]), 16, stream=s)))
