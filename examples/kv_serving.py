"""A serving loop over the paged 8-bit key/value cache, with idle requests
spilled to NVMe through the library's descriptors.

A toy attention layer (random projections, no trained weights) serves a few
requests: their prompts are reserved, appended and attended to, then every
step each running request takes a token; one branches into two (sharing its
pages until they diverge) and one ends. Between steps, the pages of a waiting
request are written out: each page is one I/O request of its own (a multiple
of 512 bytes), looked up in the registered heap, translated to PRP entries,
split over the queues and turned into submission entries. There is no drive
here; the entries are built and counted. At the end the live pages are
gathered at the front of the heap.

    python examples/kv_serving.py [--steps 8]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import memory_dma_descriptor_amd as dd  # noqa: E402

HEADS, KV_HEADS, DIM, PAGE = 16, 4, 128, 32          # query heads, key heads, values, page tokens
ROWS, NPAGES, WIDTH = 8, 512, 64                     # request slots, heap pages, pages a request
QUEUES, DEPTH = 4, 1024


class Cache:
    """The heap of pages and the requests' state, all device tensors."""

    def __init__(self, dev):
        i32 = dict(dtype=torch.int32, device=dev)
        self.page_bytes = dd.kv_page_bytes(KV_HEADS, PAGE, DIM)
        self.pool = torch.zeros((NPAGES, self.page_bytes), dtype=torch.uint8, device=dev)
        self.refs = torch.zeros(NPAGES, **i32)
        self.table = torch.full((ROWS, WIDTH), -1, **i32)
        self.lens = torch.zeros(ROWS, **i32)

    def state(self):
        return self.refs, self.table, self.lens

    def extend(self, rows, news):
        """Pages for news[i] more tokens of rows[i]; shared pages are copied first."""
        r = dd.kv_reserve(*self.state(), rows, news, PAGE)
        dd.kv_copy_pages(self.pool, r["src"], r["dst"])


class Layer:
    """Projections of one attention layer."""

    def __init__(self, dev):
        g = torch.Generator(device=dev).manual_seed(1)
        wide = HEADS * DIM
        self.qkv = torch.randn((wide, (HEADS + 2 * KV_HEADS) * DIM), generator=g, device=dev) / wide ** 0.5
        self.out = torch.randn((wide, wide), generator=g, device=dev) / wide ** 0.5
        self.qkv, self.out = self.qkv.bfloat16(), self.out.bfloat16()

    def step(self, x, cache, rows, news):
        """New tokens x [total, HEADS * DIM] of the given rows (news[i] each)."""
        total = x.shape[0]
        y = (x @ self.qkv).view(total, HEADS + 2 * KV_HEADS, DIM)
        q, k, v = y[:, :HEADS], y[:, HEADS:HEADS + KV_HEADS], y[:, HEADS + KV_HEADS:]
        start = torch.zeros(len(news) + 1, dtype=torch.int32, device=x.device)
        start[1:] = news.cumsum(0)
        table, lens = cache.table[rows.long()], cache.lens[rows.long()]
        dd.kv_append(k, v, start, cache.pool, table, lens, PAGE)
        o = dd.kv_attend(q, start, cache.pool, table, lens, KV_HEADS, PAGE)["out"]
        return x + o.reshape(total, -1) @ self.out, start


def spill(cache, row, dev):
    """Submission entries that write the pages of one request to a drive."""
    pages = cache.table[row][cache.table[row] >= 0].long()
    n = pages.numel()
    off = (pages * cache.page_bytes).view(torch.uint64)
    length = torch.full((n,), cache.page_bytes, dtype=torch.int64, device=dev).view(torch.uint64)
    heap = NPAGES * cache.page_bytes
    # One registered region over the heap, and its (here: made-up) physical pages.
    base = 1 << 40
    region = torch.tensor([base, base + -(-heap // 4096) * 4096], dtype=torch.int64, device=dev)
    lut = (torch.arange(-(-heap // 65536), device=dev) * 65536 + (1 << 33)).view(torch.uint64)
    pool = torch.zeros((n + 1, 512), dtype=torch.uint64, device=dev)
    qid = (torch.arange(n, device=dev) % QUEUES).to(torch.uint32)
    b = dd.build_batch(lut, off, length, qid, QUEUES, 1 << 34, pool, region[:1].view(torch.uint64),
                       region[1:].view(torch.uint64),
                       torch.tensor([7], device=dev).to(torch.uint32), va_base=base)
    rings = torch.zeros((QUEUES, DEPTH * 64), dtype=torch.uint8, device=dev)
    full = torch.full((QUEUES,), DEPTH, device=dev)
    slba = (torch.arange(n, device=dev) * (cache.page_bytes // 512)).view(torch.uint64)
    e = dd.emit_sqe(b["perm"], b["qoff"], b["status"], length, slba, b["prp1"], b["prp2"],
                    dd.ring_addresses(list(rings)), full.to(torch.uint32),
                    (full - 1).to(torch.uint32), torch.zeros(QUEUES, dtype=torch.uint32, device=dev),
                    torch.zeros(QUEUES, dtype=torch.uint64, device=dev), opcode=0x01)
    return n, int(e["placed"].view(torch.int32).sum())


def main(steps: int = 8) -> dict:
    dev = torch.device("cuda", torch.cuda.current_device())
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)      # noqa: E731
    g = torch.Generator(device=dev).manual_seed(0)
    cache, layer = Cache(dev), Layer(dev)

    # Three prompts of odd lengths, written and attended to in one go.
    rows, news = i32([0, 1, 2]), i32([45, 7, 130])
    cache.extend(rows, news)
    x = torch.randn((int(news.sum()), HEADS * DIM), generator=g, device=dev).bfloat16()
    y, start = layer.step(x, cache, rows, news)
    token = {int(r): y[int(start[i + 1]) - 1] for i, r in enumerate(rows)}

    # Request 2 branches; both go on from the same pages.
    dd.kv_fork(*cache.state(), i32([2]), i32([3]), PAGE)
    token[3] = token[2] * 0.5
    running = [0, 1, 2, 3]
    for step in range(steps):
        if step == steps // 2:                        # request 1 ends
            dd.kv_free(*cache.state(), i32([1]), PAGE)
            running.remove(1)
        rows, news = i32(running), torch.ones(len(running), dtype=torch.int32, device=dev)
        cache.extend(rows, news)
        y, _ = layer.step(torch.stack([token[r] for r in running]), cache, rows, news)
        token.update({r: y[i] for i, r in enumerate(running)})

    pages, entries = spill(cache, 0, dev)
    dd.kv_free(*cache.state(), i32([0]), PAGE)        # its pages are on the drive now
    moved = dd.kv_compact(*cache.state(), PAGE)
    dd.kv_copy_pages(cache.pool, moved["src"], moved["dst"], count=moved["moves"])
    live = int((cache.refs > 0).sum())
    out = dict(lens=cache.lens.tolist(), live=live, last=int((cache.refs > 0).nonzero().max()),
               spilled=pages, entries=entries, finite=bool(torch.isfinite(torch.stack(list(token.values()))).all()))
    print(f"{steps} steps: lengths {out['lens']}, {pages} pages of request 0 in {entries} submission "
          f"entries, {live} live pages gathered at the front", flush=True)
    return out


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=8)
    main(ap.parse_args().steps)
