#!/usr/bin/env python
"""The attention half of a decoder's layers served from a paged cache.

    python examples/paged_decode.py [--batch 16] [--prompt 256] [--answer 64] [--layers 4] [--e4m3 | --int8]

Each layer is what the library runs between a layer's input and its residual sum:
the stacked q/k/v projection (affqmm_run_stacked), rotary positions with the append
to the cache (affqmm_rope_append), attention over the pages (affqmm_paged_attention)
and the o projection (affqmm_run).  A step's slots and positions are planned once
for all layers (affqmm_paged_plan).  Prompts go in chunks of equal length; the
answer's steps are one captured CUDA graph, which the lengths on the GPU drive: the
host sends nothing but the replay.  The cache is bf16, e4m3 with a scale for each
head (--e4m3), or int8 with a scale for each block of tokens and head that is made as
the cache is written (--int8, affqmm_block_append and affqmm_block_attention).  Norms
and feed-forward blocks are left out, and the weights are synthetic.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from group_affine_bit_gb300 import api, synth  # noqa: E402


class Layer:
    """q, k, v and o as affine tables, and the layer's part of the cache."""

    def __init__(self, hidden, heads, kv_heads, dim, pages, page, seed, bits=4, group=64, kv_dtype=torch.bfloat16):
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        shapes = [(heads * dim, hidden), (kv_heads * dim, hidden), (kv_heads * dim, hidden), (hidden, heads * dim)]
        self.tables = []
        for i, (n, k) in enumerate(shapes):
            codes, scales, biases = synth.affine_table(bits, group, n, k, synth.generator(seed + i))
            self.tables.append(api.pack(codes.cuda(), scales.cuda(), biases.cuda(), bits, group))
        if kv_dtype == torch.int8:
            self.cache = api.BlockCache.empty(pages, page, kv_heads, dim)
            return
        scale = [torch.full((kv_heads,), 1 / 16, device="cuda") for _ in "kv"] if kv_dtype == torch.float8_e4m3fn else [None, None]
        self.cache = api.KVCache.empty(pages, page, kv_heads, dim, kv_dtype, k_scale=scale[0], v_scale=scale[1])

    def __call__(self, x, step, table, rope, batch):
        rows = x.shape[0]
        q, k, v = api.run_stacked(self.tables[:3], x)
        q = q.view(rows, self.heads, self.dim)
        api.rope_append(q, k.view(rows, self.kv_heads, self.dim), v.view(rows, self.kv_heads, self.dim), step.positions,
                        step.slots, rope, self.cache, out=q)
        q = q.view(batch, rows // batch, self.heads, self.dim)
        a = api.paged_attention(q, self.cache, table, step.lens)
        return x + api.run(self.tables[3], a.view(rows, -1))


class Server:
    """`batch` requests over `layers` layers and one pool of pages."""

    def __init__(self, layers, batch, hidden, heads, kv_heads, dim, page, pages, longest, base=10000.0, kv_dtype=torch.bfloat16):
        self.batch = batch
        self.layers = [Layer(hidden, heads, kv_heads, dim, pages, page, 100 * i, kv_dtype=kv_dtype) for i in range(layers)]
        self.rope = api.Rope(api.rope_turns([base ** (-2 * i / dim) for i in range(dim // 2)]))
        self.page = page
        self.table = torch.full((batch, -(-longest // page)), -1, dtype=torch.int32, device="cuda")
        self.ring = torch.arange(pages, dtype=torch.int32, device="cuda")
        self.ring_state = torch.tensor([0, pages], dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.steps: dict = {}        # tokens a request -> (fresh, PagedStep), whose addresses a graph keeps

    def forward(self, x):
        """x bf16 [batch * n, hidden]: n new tokens of every request, through all layers."""
        n = x.shape[0] // self.batch
        if n not in self.steps:
            self.steps[n] = (torch.full((self.batch,), n, dtype=torch.int32, device="cuda"), api.PagedStep.empty(self.batch, x.shape[0]))
        fresh, step = self.steps[n]
        api.paged_plan(self.lens, fresh, None, self.table, self.ring, self.ring_state, self.page, out=step)
        for layer in self.layers:
            x = layer(x, step, self.table, self.rope, self.batch)
        self.lens.copy_(step.lens)
        self.ring_state.copy_(step.ring_state)
        return x

    def captured(self, x):
        """One step of x's shape as a graph: (graph, its input, its output)."""
        at_lens, at_ring = self.lens.clone(), self.ring_state.clone()
        x = x.clone()
        self.forward(x)              # sizes the workspace and the step's buffers before the capture
        self.lens.copy_(at_lens)
        self.ring_state.copy_(at_ring)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            self.forward(x)          # that stream's own workspace
        stream.synchronize()
        self.lens.copy_(at_lens)
        self.ring_state.copy_(at_ring)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            y = self.forward(x)
        return graph, x, y


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=256)
    ap.add_argument("--answer", type=int, default=64)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=5376)
    ap.add_argument("--e4m3", action="store_true", help="a cache of 8-bit floats")
    ap.add_argument("--int8", action="store_true", help="a cache of 8-bit integers with a scale for each block of tokens")
    args = ap.parse_args()
    page, longest = 32, args.prompt + args.answer
    pages = args.batch * -(-longest // page)
    server = Server(args.layers, args.batch, args.hidden, heads=32, kv_heads=8, dim=256, page=page, pages=pages, longest=longest,
                    kv_dtype=torch.int8 if args.int8 else torch.float8_e4m3fn if args.e4m3 else torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(0)
    chunk = 8
    for at in range(0, args.prompt, chunk):
        n = min(chunk, args.prompt - at)
        server.forward(torch.randn(args.batch * n, args.hidden, device="cuda", generator=g).bfloat16())
    x = torch.randn(args.batch, args.hidden, device="cuda", generator=g).bfloat16()
    graph, x, y = server.captured(x)
    torch.cuda.synchronize()
    begin = time.perf_counter()
    for _ in range(args.answer):
        graph.replay()
    torch.cuda.synchronize()
    spent = time.perf_counter() - begin
    print(f"{args.batch} requests, {args.prompt} + {args.answer} tokens, {args.layers} layers: {spent / args.answer * 1e6:.1f} us a step, "
          f"{args.batch * args.answer / spent:.0f} tokens/s; lengths {server.lens.tolist()[:4]}..., output {tuple(y.shape)}")


if __name__ == "__main__":
    main()
