#!/usr/bin/env python
"""A small decoder served with adapters: every request carries its own adapter
and its own cache pages, one token of each request per step.

One step is what a serving engine runs between two samplings: pages and slots
for the new tokens (``kv_resize``), then for every layer a norm, the adapted
q, k and v projections (``linear_batch``), rotary positions and the cache write
(``kv_append``), attention over the cached tokens (``paged_attention``), the
adapted output projection, the norm that closes the sub-block
(``residual_norm``) and the adapted feed-forward block.  Lengths, tables and
slots stay on the device, so a step can be captured in a CUDA graph and
replayed while requests grow.

    python examples/decode_block.py            # 2 small layers, 64 requests
    python examples/decode_block.py --llama    # 1 layer of Llama-3-8B shapes
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import lora_normal_form_gb300 as scute  # noqa: E402
import workloads as WL  # noqa: E402

PROJ = ("q", "k", "v", "o", "gate", "up", "down")


def shapes_of(hidden: int, heads: int, kv_heads: int, dim: int, ffn: int, layers: int) -> dict:
    """Projection shapes of a decoder, by layer ("0.q", ...); (IA)^3's vectors
    on keys, values and the up projection."""
    one = {"q": (hidden, heads * dim, False), "k": (hidden, kv_heads * dim, True), "v": (hidden, kv_heads * dim, True),
           "o": (heads * dim, hidden, False), "gate": (hidden, ffn, False), "up": (hidden, ffn, True),
           "down": (ffn, hidden, False)}
    return {f"{i}.{p}": one[p] for i in range(layers) for p in PROJ}


class Decoder:
    """The stack's weights, cache and step buffers for up to ``requests`` requests."""

    def __init__(self, ctx, layer_ids, layers: int, hidden: int, heads: int, kv_heads: int, dim: int, ffn: int,
                 requests: int, pages: int, page_size: int, max_len: int, norms, theta: float = 500000.0,
                 eps: float = 1e-5):
        self.ctx, self.layer_ids, self.layers, self.eps, self.page_size = ctx, layer_ids, layers, eps, page_size
        self.dtype = torch.bfloat16 if ctx.dtype == "bf16" else torch.float32
        dev = {"device": "cuda"}
        new = lambda *s: torch.empty(*s, dtype=self.dtype, **dev)  # noqa: E731
        whole = lambda *s: torch.zeros(*s, dtype=torch.int32, **dev)  # noqa: E731
        n = requests
        self.norms = norms                          # per layer: attention, feed-forward; then the final one
        # cache bookkeeping
        self.length, self.want, self.cu, self.req = whole(n), whole(n), whole(n + 1), whole(n)
        self.table = torch.full((n, -(-max_len // page_size)), -1, dtype=torch.int32, **dev)
        self.free = torch.arange(pages, dtype=torch.int32, **dev)
        self.free_count = torch.full((1,), pages, dtype=torch.int32, **dev)
        self.slots, self.positions = whole(n), whole(n)              # of the step's rows, packed
        self.row_slots, self.row_positions = whole(n), whole(n)      # of the requests
        self.none, self.start = whole(n) - 1, whole(n)
        self.caches = [scute.KvCache(new(pages, kv_heads, page_size, dim), new(pages, kv_heads, page_size, dim), self.table)
                       for _ in range(layers)]
        self.cos_sin = torch.empty(max_len, dim, **dev)
        ctx.rope_table(self.cos_sin, theta)
        self.rope = scute.Rope(self.cos_sin, self.row_positions)
        # one step's activations
        self.ids = whole(n)
        self.x, self.h, self.a = new(n, hidden), new(n, hidden), new(n, hidden)
        self.q, self.qr, self.att = new(n, heads * dim), new(n, heads * dim), new(n, heads * dim)
        self.k, self.v = new(n, kv_heads * dim), new(n, kv_heads * dim)
        self.gate, self.up, self.out = new(n, ffn), new(n, ffn), new(n, hidden)

    def step(self):
        """Take the rows ``x`` of the requests whose ``want`` is one more than
        their ``length`` (the others keep theirs, or end where ``want`` is 0) and
        return the final hidden rows, row i for request i.

        A request that takes no token (it keeps its length, ends, or is refused
        for want of pages, which the status word says) gets slot -1: nothing of
        its row is written to the cache, and its final row means nothing."""
        ctx, io = self.ctx, self.ctx.dtype
        lid = lambda i, p: self.layer_ids[f"{i}.{p}"]  # noqa: E731
        ctx.kv_resize(self.length, self.want, self.table, self.page_size, self.free, self.free_count, self.free_count,
                      self.length, self.cu, self.slots, self.positions, self.req)
        # the new tokens' rows come packed, request r's (if it has one) at cu[r]; the
        # step's own rows stay with their requests
        took, at = self.cu[1:] > self.cu[:-1], self.cu[:-1].clamp(max=len(self.cu) - 2)
        torch.where(took, self.slots[at], self.none, out=self.row_slots)
        torch.where(took, self.positions[at], self.start, out=self.row_positions)
        self.h.copy_(self.x)
        ctx.residual_norm(self.h, self.a, pre_w=self.norms[0], eps=self.eps)
        for i in range(self.layers):
            ctx.linear_batch([(self.a, lid(i, "q"), self.q), (self.a, lid(i, "k"), self.k),
                              (self.a, lid(i, "v"), self.v)], self.ids, io)
            ctx.kv_append(self.caches[i], self.row_slots, self.k, self.v, q=self.q, q_out=self.qr, rope=self.rope)
            ctx.paged_attention(self.caches[i], self.qr, self.length, self.att)
            ctx.linear(self.att, self.ids, lid(i, "o"), self.out, io)
            ctx.residual_norm(self.out, self.a, residual=self.h, residual_out=self.h, pre_w=self.norms[2 * i + 1],
                              eps=self.eps)
            ctx.linear_batch([(self.a, lid(i, "gate"), self.gate), (self.a, lid(i, "up"), self.up)], self.ids, io)
            torch.mul(torch.nn.functional.silu(self.gate), self.up, out=self.gate)
            ctx.linear(self.gate, self.ids, lid(i, "down"), self.out, io)
            ctx.residual_norm(self.out, self.a, residual=self.h, residual_out=self.h, pre_w=self.norms[2 * i + 2],
                              eps=self.eps)
        return self.a


def build(dtype: str, hidden: int, heads: int, kv_heads: int, dim: int, ffn: int, layers: int, requests: int,
          max_len: int, page_size: int = 16, n_adapters: int = 10, rank: int = 16, rv: int = 256, seed: int = 0):
    """A decoder with random weights and mixed adapters: (decoder, workload, norm weights)."""
    shapes = shapes_of(hidden, heads, kv_heads, dim, ffn, layers)
    w = WL.decode_mixed(seed=seed, n=requests, n_adapters=n_adapters, rank=rank, rv=rv, proj=tuple(shapes), shapes=shapes,
                        dtype=dtype)
    ctx = scute.Context(dtype=dtype, max_tokens=max(64, requests), max_adapters=n_adapters + 2, max_layers=len(shapes))
    ctx.load_workload(w)
    norms = [WL.draw_vector(seed, f"norm{i}", hidden) for i in range(2 * layers + 1)]
    pages = requests * -(-max_len // page_size)
    dec = Decoder(ctx, ctx.layer_ids, layers, hidden, heads, kv_heads, dim, ffn, requests, pages, page_size, max_len,
                  [torch.from_numpy(v).cuda() for v in norms])
    dec.ids.copy_(torch.from_numpy(np.asarray(w.ids)))
    return dec, w, norms


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--llama", action="store_true", help="one layer of Llama-3-8B shapes (drawing its weights takes a while)")
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--steps", type=int, default=200)
    args = ap.parse_args()
    size = dict(hidden=4096, heads=32, kv_heads=8, dim=128, ffn=14336, layers=1) if args.llama else \
        dict(hidden=1024, heads=16, kv_heads=4, dim=64, ffn=2816, layers=2)
    max_len = args.steps + 64
    dec, w, _ = build("bf16", requests=args.requests, max_len=max_len, **size)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    dec.x.normal_(generator=g)

    def one():
        torch.add(dec.length, 1, out=dec.want)
        return dec.step()

    for _ in range(3):
        one()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = one()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(args.steps):
        graph.replay()
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t) / args.steps * 1e3
    if dec.ctx.sync_status() != 0:
        raise SystemExit("a device-side error was recorded")
    print(f"{size['layers']} layers, hidden {size['hidden']}, {args.requests} requests of {int(dec.length[0])} tokens, "
          f"{w.n_adapters} adapters: {ms:.3f} ms per step, {args.requests / ms * 1e3:.0f} tokens/s, "
          f"finite {bool(torch.isfinite(out.float()).all())}")
    dec.ctx.close()


if __name__ == "__main__":
    main()
