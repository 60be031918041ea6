"""The paged cache's operators and the projections together, as the example runs
them: prompt chunks, then decode steps replayed from one graph, against a 64-bit
form without a cache that rounds to bf16 where the layers do.

Tolerance: the two differ where a value on a rounding boundary falls to either
side, one bf16 step (2^-7 of the value at most) at each of the five roundings of a
layer; 2^-6 of the row's largest value, over two layers, leaves room for those."""
import os
import sys

import pytest
import torch

import paged_ref
from group_affine_bit_gb300 import api

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import paged_decode  # noqa: E402

pytestmark = pytest.mark.gpu


def bf(x):
    return x.to(torch.bfloat16).double()


def reference(server, xs, dim, heads, kv_heads):
    """xs [B, T, hidden] float64: all tokens at once, causal, layer by layer."""
    B, T, _ = xs.shape
    G = heads // kv_heads
    freqs = paged_ref.turns_of(dim)
    pos = torch.arange(T)[None]
    x = xs
    for layer in server.layers:
        w = [api.dequant(t).cpu().double() for t in layer.tables]
        q, k, v = (bf(x @ a.T) for a in w[:3])
        out = torch.zeros(B, T, heads * dim, dtype=torch.float64)
        for b in range(B):
            qq = bf(paged_ref.rope(q[b].view(T, heads, dim), pos, freqs, [0] * (dim // 2), False))
            kk = bf(paged_ref.rope(k[b].view(T, kv_heads, dim), pos, freqs, [0] * (dim // 2), False))
            vv = v[b].view(T, kv_heads, dim)
            for h in range(heads):
                s = qq[:, h] @ kk[:, h // G].T * dim ** -0.5
                s = s.masked_fill(torch.triu(torch.ones(T, T, dtype=torch.bool), 1), -float("inf"))
                out[b, :, h * dim: (h + 1) * dim] = torch.softmax(s, 1) @ vv[:, h // G]
        x = bf(x + bf(bf(out) @ w[3].T))
    return x


def test_prompt_chunks_and_a_captured_answer():
    B, hidden, heads, kv_heads, dim, page = 3, 256, 4, 2, 64, 8
    server = paged_decode.Server(2, B, hidden, heads, kv_heads, dim, page, pages=3 * 4 + 1, longest=30)
    g = torch.Generator().manual_seed(1)
    prompt, answer = 11, 9
    xs = torch.randn(B, prompt + answer, hidden, generator=g).bfloat16()
    got = []
    at = 0
    for n in (6, 4, 1):
        y = server.forward(xs[:, at: at + n].reshape(B * n, hidden).cuda())
        got.append(y.view(B, n, hidden).cpu())
        at += n
    graph, x, y = server.captured(xs[:, at].cuda())
    for i in range(at, prompt + answer):
        x.copy_(xs[:, i].cuda())
        graph.replay()
        got.append(y.cpu().view(B, 1, hidden).clone())
    torch.cuda.synchronize()
    assert server.lens.tolist() == [prompt + answer] * B
    got = torch.cat(got, 1).double()
    want = reference(server, xs.double(), dim, heads, kv_heads)
    room = 2.0 ** -6 * want.abs().amax(-1, keepdim=True)
    assert bool(((got - want).abs() <= room).all())


def test_an_8_bit_cache_follows_the_16_bit_one():
    """The same requests over e4m3 pages: outputs differ by the cache's rounding (2^-4 of a value, averaged over
    the keys), not more than 5 % of the output's norm."""
    B, hidden, heads, kv_heads, dim, page = 2, 256, 4, 2, 64, 16
    g = torch.Generator().manual_seed(2)
    xs = torch.randn(12, B, hidden, generator=g).bfloat16().cuda()
    outs = []
    for dt in (torch.bfloat16, torch.float8_e4m3fn):
        server = paged_decode.Server(1, B, hidden, heads, kv_heads, dim, page, pages=4, longest=20, kv_dtype=dt)
        outs.append(torch.stack([server.forward(x) for x in xs]).float())
    a, b = outs
    assert float((a - b).norm() / a.norm()) < 0.05 and not torch.equal(a, b)
