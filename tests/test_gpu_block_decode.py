"""The block cache's operators and the projections together, as the example runs them: prompt chunks, then decode steps
replayed from one graph, against a 64-bit form that keeps codes and scales of its own; and what the layers left in their
caches, read back.

Tolerance: as test_gpu_paged_decode has it, 2^-6 of the row's largest value for the five bf16 roundings of each of two
layers; and as much again for the codes: one that falls to the other side of a border is off by 1/127 of its block's
largest value, less than the 2^-7 that a bf16 rounding may be."""
import os
import sys

import pytest
import torch

import blocks_ref
import paged_ref
from group_affine_bit_gb300 import api

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import paged_decode  # noqa: E402

pytestmark = pytest.mark.gpu


def bf(x):
    return x.to(torch.bfloat16).double()


class Blocks:
    """One request's k or v of a layer, [tokens, heads, dim] codes with a scale for each block and head."""

    def __init__(self, block, heads, dim):
        self.block, self.codes, self.scales = block, torch.zeros(0, heads, dim, dtype=torch.float64), []

    def add(self, x):
        """A call's tokens, all of them behind those that are there."""
        for i in range(x.shape[0]):                        # token by token, the call's part of a block at once
            at = self.codes.shape[0]
            if at % self.block == 0 or i == 0:
                part = x[i: i + self.block - at % self.block]
                need = blocks_ref.need(part.abs().amax((0, 2)), "int8")
                if at % self.block == 0:
                    self.scales.append(need)
                else:
                    old, b = self.scales[-1], at // self.block * self.block
                    new = torch.maximum(old, need)
                    self.codes[b:] = torch.where((old < new)[:, None], (self.codes[b:] * (old / new)[:, None]).round(), self.codes[b:])
                    self.scales[-1] = new
            self.codes = torch.cat([self.codes, (x[i] / self.scales[-1][:, None]).round().clamp(-127, 127)[None]])

    def values(self):
        return self.codes * torch.stack(self.scales).repeat_interleave(self.block, 0)[: self.codes.shape[0], :, None]


def reference(server, xs, steps, dim, heads, kv_heads, block):
    """xs [B, T, hidden] float64 in calls of `steps` tokens."""
    B, G = xs.shape[0], heads // kv_heads
    freqs = paged_ref.turns_of(dim)
    weights = [[api.dequant(t).cpu().double() for t in layer.tables] for layer in server.layers]
    held = [[[Blocks(block, kv_heads, dim) for _ in "kv"] for _ in range(B)] for _ in server.layers]
    outs, at = [], 0
    for n in steps:
        x = xs[:, at: at + n]
        pos = torch.arange(at, at + n)[None]
        for w, cache in zip(weights, held):
            q, k, v = (bf(x @ a.T) for a in w[:3])
            out = torch.zeros(B, n, heads * dim, dtype=torch.float64)
            for b in range(B):
                qq = bf(paged_ref.rope(q[b].view(n, heads, dim), pos, freqs, [0] * (dim // 2), False))
                cache[b][0].add(paged_ref.rope(k[b].view(n, kv_heads, dim), pos, freqs, [0] * (dim // 2), False))
                cache[b][1].add(v[b].view(n, kv_heads, dim))
                kk, vv = (c.values() for c in cache[b])
                for h in range(heads):
                    s = qq[:, h] @ kk[:, h // G].T * dim ** -0.5
                    s = s.masked_fill(torch.arange(at + n)[None] > pos[0][:, None], -float("inf"))
                    out[b, :, h * dim: (h + 1) * dim] = torch.softmax(s, 1) @ vv[:, h // G]
            x = bf(x + bf(bf(out) @ w[3].T))
        outs.append(x)
        at += n
    return torch.cat(outs, 1)


def test_prompt_chunks_and_a_captured_answer():
    B, hidden, heads, kv_heads, dim, page = 3, 256, 4, 2, 64, 8
    server = paged_decode.Server(2, B, hidden, heads, kv_heads, dim, page, pages=3 * 4 + 1, longest=30, kv_dtype=torch.int8)
    block = server.layers[0].cache.block
    assert block == page
    g = torch.Generator().manual_seed(1)
    chunks, answer = (6, 4, 1), 9
    xs = torch.randn(B, sum(chunks) + answer, hidden, generator=g).bfloat16()
    got, at = [], 0
    for n in chunks:
        y = server.forward(xs[:, at: at + n].reshape(B * n, hidden).cuda())
        got.append(y.view(B, n, hidden).cpu())
        at += n
    graph, x, y = server.captured(xs[:, at].cuda())        # runs the first answer's step beforehand: the same slots again
    for i in range(at, at + answer):
        x.copy_(xs[:, i].cuda())
        graph.replay()
        got.append(y.cpu().view(B, 1, hidden).clone())
    torch.cuda.synchronize()
    total = at + answer
    assert server.lens.tolist() == [total] * B
    got = torch.cat(got, 1).double()
    want = reference(server, xs.double(), list(chunks) + [1] * answer, dim, heads, kv_heads, block)
    room = 2.0 ** -5 * want.abs().amax(-1, keepdim=True)
    assert bool(((got - want).abs() <= room).all())

    # the last layer's cache read back, and attention over the rows: what attention over the pages gives
    cache = server.layers[-1].cache
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda") * total
    k, v = api.paged_read(cache, server.table, starts, rows=B * total)
    for b in range(B):
        pages = server.table[b, : -(-total // page)].long().cpu()
        for rows, codes, scales in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
            held = blocks_ref.values(codes.cpu(), scales.cpu())[pages].flatten(0, 1)[:total]
            assert bool(((rows[b * total: (b + 1) * total].cpu().double() - held).abs() <= held.abs() * (2.0 ** -8 + 2.0 ** -23)).all())
    q = torch.randn(B, 1, heads, dim, generator=g).bfloat16().cuda()
    pages_out = api.paged_attention(q, cache, server.table, server.lens).double().cpu()
    kk, vv = (r.double().cpu().view(B, total, kv_heads, dim) for r in (k, v))
    for b in range(B):
        for h in range(heads):
            key = kk[b, :, h // 2]
            p = torch.softmax(key @ q[b, 0, h].double().cpu() * dim ** -0.5, 0)
            want = p @ vv[b, :, h // 2]
            # rows rounded to bf16: 2^-8 of each value, and of each score's terms, besides the output's own rounding
            off = (key.abs() @ q[b, 0, h].double().cpu().abs() * dim ** -0.5).amax() * 2.0 ** -8
            assert bool(((pages_out[b, 0, h] - want).abs() <= want.abs() * 2.0 ** -8 + (p @ vv[b, :, h // 2].abs()) * (2.0 ** -8 + 2 * off + 2.0 ** -10)).all())


def test_codes_follow_the_16_bit_cache():
    """The same requests over int8 pages and bf16 ones: a value is off by half of 1/127 of its block's largest at most, and
    outputs, which average over keys, by less than 2 % of their norm."""
    B, hidden, heads, kv_heads, dim, page = 2, 256, 4, 2, 64, 16
    g = torch.Generator().manual_seed(2)
    xs = torch.randn(12, B, hidden, generator=g).bfloat16().cuda()
    outs = []
    for dt in (torch.bfloat16, torch.int8):
        server = paged_decode.Server(1, B, hidden, heads, kv_heads, dim, page, pages=4, longest=20, kv_dtype=dt)
        outs.append(torch.stack([server.forward(x) for x in xs]).float())
    a, b = outs
    assert float((a - b).norm() / a.norm()) < 0.02 and not torch.equal(a, b)
