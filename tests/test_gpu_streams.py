"""Calls given a stream of their own take the memory of their results and
workspaces in that stream's order: a block that the current stream has freed may
still be used by work queued there, which the other stream does not wait for."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import memory_dma_descriptor_amd as dd
import oracle
import synth
from tests import gpu_cases as gc
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


def test_descriptor_calls():
    d = synth.generate("tiny", n=500)
    lut, off, ln, qid = gc.dev(d["lut"]), gc.dev(d["off"]), gc.dev(d["len"]), gc.dev(d["qid"])
    table = gc.dev(d["rstart"]), gc.dev(d["rend"]), gc.dev(d["rlkey"])
    bus, nq = d["list_bus_base"], d["nqueues"]
    pages = oracle.build_prp(d["lut"], d["off"], d["len"], bus, 1 << 50)["total"]
    pool = torch.zeros((pages, 512), dtype=torch.uint64, device="cuda")

    def same(results):
        for k, v in results[0].items():
            assert torch.equal(v, results[1][k]), k

    same(ordered(lambda s: dd.mr_lookup(*table, off, ln, va_base=d["va_base"], stream=s)))
    same(ordered(lambda s: dd.build_prp(lut, off, ln, bus, pool, stream=s)))
    same(ordered(lambda s: dd.partition_by_queue(qid, nq, stream=s)))
    batches = ordered(lambda s: dd.build_batch(lut, off, ln, qid, nq, bus, pool, *table,
                                               va_base=d["va_base"], stream=s))
    same(batches)
    b = batches[0]

    def emit(s):
        rings = torch.zeros((nq, 8192 * 64), dtype=torch.uint8, device="cuda")
        depth = gc.dev(np.full(nq, 8192, np.uint32))
        free = gc.dev(np.full(nq, 8191, np.uint32))
        tail, cursor = gc.dev(np.zeros(nq, np.uint32)), gc.dev(np.zeros(nq, np.uint64))
        slba = gc.dev(synth.slba("tiny", d["n"]))
        addresses = dd.ring_addresses(list(rings))
        torch.cuda.synchronize()
        r = dd.emit_sqe(b["perm"], b["qoff"], b["status"], ln, slba, b["prp1"], b["prp2"], addresses,
                        depth, free, tail, cursor, stream=s)
        torch.cuda.synchronize()
        return dict(placed=r["placed"])
    same(ordered(emit))


def test_registry_calls():
    addr = gc.dev(np.arange(64, dtype=np.uint64) * np.uint64(1 << 20))
    size = gc.dev(np.full(64, 4096, np.uint64))

    def register(s):
        reg = dd.DeviceRegistry()
        torch.cuda.synchronize()
        r = reg.register(addr, size, stream=s)           # grows from nothing
        torch.cuda.synchronize()
        status = reg.deregister(r["handle"], stream=s)
        torch.cuda.synchronize()
        assert (status == dd.DEREG_REMOVED).all() and reg.count() == 0
        return dict(handle=r["handle"], kind=r["kind"], status=status)
    a, b = ordered(register)
    assert all(torch.equal(a[k], b[k]) for k in a)
