"""Attention over a paged cache with a scale for each block of tokens and head, against a 64-bit form (bounds:
blocks_ref.attention_bounds)."""
import math

import pytest
import torch

import blocks_ref
from group_affine_bit_gb300 import api

pytestmark = pytest.mark.gpu


def scene(lens, hq, hk, dim, page, kv="int8", block=None, tokens=1, seed=0, layout="token", spare=2, uneven=1.0):
    """A pool whose every code that no request holds is the type's lowest (int8) or NaN (e4m3), its scales NaN or an
    infinity; `uneven`: how far the blocks' magnitudes differ (a standard deviation of their logarithm)."""
    g = torch.Generator().manual_seed(seed)
    block = min(page, 16) if block is None else block
    B = len(lens)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=g)
    table = torch.full((B, max(max(used), 1)), -1, dtype=torch.int32)
    held = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        table[b, : used[b]] = order[at: at + used[b]].to(torch.int32)
        for i in range(used[b]):
            held[order[at + i], : min(page, n - i * page)] = True
        at += used[b]
    codes, scales = [], []
    for w in "kv":
        x = torch.randn(pages, page // block, block, hk, dim, generator=g)
        x *= torch.exp(uneven * torch.randn(pages, page // block, 1, hk, 1, generator=g)) if w == "v" else 1
        c, s = blocks_ref.quantise(x, kv)
        c.view(torch.uint8)[~held] = 0x80 if kv == "int8" else 0x7f
        s[~held.view(pages, page // block, block).any(2)] = float("nan") if w == "k" else float("inf")
        codes.append(c)
        scales.append(s)
    q = torch.randn(B, tokens, hq, dim, generator=g).bfloat16()
    return dict(q=q, k=codes[0], v=codes[1], ks=scales[0], vs=scales[1], table=table, lens=torch.tensor(lens, dtype=torch.int32), layout=layout)


def cache_of(s):
    put = lambda t: t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if s["layout"] == "head" else t.cuda()  # noqa: E731
    return api.BlockCache(*(put(s[x]) for x in ("k", "v", "ks", "vs")))


def attend(s, scale=None, window=0, **kw):
    q = s["q"].cuda()
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.paged_attention(q, cache_of(s), s["table"].cuda(), s["lens"].cuda(), scale=scale, window=window, lse=lse, status=status, **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu(), int(status[0])


def check(s, scale=None, window=0):
    out, lse, status = attend(s, scale, window)
    assert status == 0
    dim = s["q"].shape[-1]
    sc = dim ** -0.5 if scale is None else scale
    want, wl, *more = blocks_ref.attention(s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"], sc, window)
    b_out, b_lse = blocks_ref.attention_bounds(want, wl, *more, dim)
    assert bool(((out.double() - want).abs() <= b_out).all())
    empty = torch.isinf(wl)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    assert bool(((lse.double() - wl).abs() <= b_lse)[~empty].all())
    assert bool((out[empty] == 0).all())
    return out, lse


EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 1000]


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 128, 192, 256, 320, 512])
def test_lengths_and_dims(dim, kv):
    check(scene(EDGES, 4, 2, dim, 16, kv, seed=dim))


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("page,block", [(1, 1), (2, 1), (2, 2), (4, 4), (8, 1), (8, 4), (32, 32), (64, 1), (64, 64), (128, 128), (256, 64), (256, 2)])
def test_pages_and_blocks(page, block, kv):
    for layout in ("token", "head"):
        check(scene([1, 70, 129, 5, 257], 6, 2, 96, page, kv, block, seed=page, layout=layout))
        check(scene([1, 70, 129, 5, 257], 6, 2, 256, page, kv, block, tokens=3, seed=page, layout=layout), window=33)


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256, 512])
@pytest.mark.parametrize("hq,hk,tokens", [(1, 1, 1), (7, 1, 1), (8, 8, 2), (16, 1, 2), (12, 2, 5), (16, 1, 4), (16, 1, 7), (40, 2, 8), (2, 2, 64)])
def test_rows_that_share_a_key_head(hq, hk, tokens, dim, kv):
    check(scene([3, 64, 150, 0, 331], hq, hk, dim, 16, kv, tokens=tokens, seed=hq + tokens))


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 63, 65, 500, 5000])
@pytest.mark.parametrize("tokens", [1, 5])
def test_windows(window, tokens):
    for kv in ("int8", "e4m3"):
        check(scene([0, 1, 3, 16, 64, 65, 130, 700], 8, 2, 128, 8, kv, tokens=tokens, seed=window), window=window)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.25, 30.0])
def test_scores_sharp_flat_and_negative(scale):
    check(scene([1, 65, 900], 8, 2, 64, 16, seed=2), scale=scale)


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("uneven", [0.0, 4.0, 12.0])
def test_blocks_of_very_different_magnitudes(uneven, kv):
    """Values whose blocks differ by factors up to 2^50 and more, within what a scale may be."""
    s = scene([40, 700, 1], 8, 2, 64, 16, kv, seed=3, uneven=uneven)
    for x in ("ks", "vs"):
        s[x] = torch.where(torch.isfinite(s[x]), s[x].clamp(blocks_ref.LEAST, blocks_ref.MOST), s[x])
    check(s)


def test_scales_at_the_ends_of_their_range():
    """Blocks at 2^-48 beside blocks at 2^48; beyond them, a scale counts as the end."""
    for lo, hi in ((2.0 ** -48, 2.0 ** 48), (0.0, 2.0 ** 48), (2.0 ** -48, math.inf), (-1.0, 2.0 ** 60), (2.0 ** -140, 1.0)):
        s = scene([200, 33], 4, 2, 64, 16, seed=4)
        s["vs"][::2], s["vs"][1::2] = lo, hi
        got = attend(s)
        s["vs"][::2], s["vs"][1::2] = max(lo, 2.0 ** -48), min(hi, 2.0 ** 48)
        want = check(s)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for bad, counts in ((0.0, 2.0 ** -48), (math.nan, 2.0 ** -48), (-5.0, 2.0 ** -48)):
        s = scene([200, 33], 4, 2, 64, 16, seed=5)
        s["ks"][::2] = bad
        got = attend(s)
        s["ks"][::2] = counts
        want = check(s)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("nats", [10, 16, 18])
def test_small_probabilities_beside_a_large_one(nats, kv):
    """One key `nats` above the others whose value is zero (and its block's scale the least there is): the others are the
    whole output."""
    s = scene([600] * 12, 8, 8, 64, 16, kv, block=1, seed=nats)
    s["q"].zero_(), s["k"].zero_()
    s["q"][..., 0], s["ks"][:] = 1, 1
    for b in range(12):
        at = (0, 300, 599)[b % 3]
        p, o = int(s["table"][b, at // 16]), at % 16
        s["k"][p, o, :, 0], s["v"][p, o], s["vs"][p, o] = 1, 0, 2.0 ** -48
    check(s, scale=float(nats))


@pytest.mark.parametrize("hq,hk,dim,lens,kv,page", [(8, 1, 128, [20011], "int8", 32), (32, 8, 256, [9000, 31], "int8", 16), (2, 2, 64, [30000, 1, 64, 7000], "e4m3", 64),
                                                    (16, 1, 512, [5000, 3001], "e4m3", 32), (24, 3, 256, [3000, 1], "int8", 128)])
def test_long_caches_are_split_and_joined(hq, hk, dim, lens, kv, page):
    check(scene(lens, hq, hk, dim, page, kv, seed=7))


def test_many_short_requests():
    check(scene([1 + (i * 37) % 90 for i in range(700)], 2, 1, 64, 16, seed=3))


@pytest.mark.parametrize("hq,hk,tokens,dim,kv", [(8, 2, 1, 128, "int8"), (8, 2, 1, 256, "e4m3"), (8, 2, 4, 192, "int8"), (8, 4, 1, 128, "e4m3"),
                                                 (12, 6, 4, 96, "int8"), (8, 8, 1, 64, "int8"), (6, 2, 2, 48, "e4m3"), (9, 3, 1, 64, "int8"), (32, 2, 2, 512, "int8")])
def test_tables_with_room_for_much_more(hq, hk, tokens, dim, kv):
    """The same requests in rows of a table that could hold half a million tokens: a coarser cut of the work, and two key
    heads to a CTA where pages and rows allow it."""
    for page, block, window in ((16, 16, 0), (4, 2, 40), (32, 32, 0), (64, 1, 100), (64, 64, 0)):
        s = scene(EDGES, hq, hk, dim, page, kv, block, tokens=tokens, seed=dim)
        wide = torch.full((len(EDGES), (1 << 19) // page), -1, dtype=torch.int32)
        wide[:, : s["table"].shape[1]] = s["table"]
        s["table"] = wide
        check(s, window=window)
    long = scene([5003, 17, 9000], hq, hk, dim, 32, kv, tokens=tokens, seed=1)
    wide = torch.full((3, 40000), -1, dtype=torch.int32)
    wide[:, : long["table"].shape[1]] = long["table"]
    long["table"] = wide
    check(long)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [1, 8, 32])
def test_two_key_heads_to_a_cta_whose_scales_lie_anywhere(block, dim):
    """The two heads' scales side by side on eight bytes or not, or apart: the same bits."""
    s = scene([5003, 17, 900], 8, 4, dim, 32, "int8", block, seed=block)
    wide = torch.full((3, 40000), -1, dtype=torch.int32)
    wide[:, : s["table"].shape[1]] = s["table"]
    s["table"] = wide
    want, wl = check(s)
    k, v, table, lens, q = s["k"].cuda(), s["v"].cuda(), wide.cuda(), s["lens"].cuda(), s["q"].cuda()
    shape = s["ks"].shape
    flat = [torch.zeros(shape.numel() + 3, device="cuda")[3:].view(shape) for _ in "kv"]       # four bytes off the boundary
    odd = [torch.zeros(shape[0], shape[1], shape[2] + 1, device="cuda")[:, :, :-1] for _ in "kv"]  # an odd stride of blocks
    apart = [torch.zeros(shape[2], shape[0], shape[1], device="cuda").permute(1, 2, 0) for _ in "kv"]
    for ks, vs in (flat, odd, apart):
        ks.copy_(s["ks"]), vs.copy_(s["vs"])
        lse = torch.empty(q.shape[:3], device="cuda")
        out = api.paged_attention(q, api.BlockCache(k, v, ks, vs), table, lens, lse=lse)
        assert torch.equal(out.cpu(), want) and torch.equal(lse.cpu(), wl)


def test_same_inputs_same_bits():
    s = scene([8000, 17, 3000, 1, 500], 8, 2, 128, 16, seed=4)
    first = attend(s)
    for _ in range(5):
        again = attend(s)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_what_a_later_token_sees_does_not_reach_an_earlier_one():
    """Five tokens; the codes of the last three are NaN: rows that do not see them are as if they were zeros."""
    for dim in (64, 256):
        s = scene([70, 5, 129], 4, 2, dim, 16, "e4m3", tokens=5, seed=11)
        clean = {**s, "k": s["k"].clone(), "v": s["v"].clone()}
        for b, n in enumerate(s["lens"].tolist()):
            for i in range(n - 3, n):
                p, o = int(s["table"][b, i // 16]), i % 16
                s["v"].view(torch.uint8)[p, o], s["k"].view(torch.uint8)[p, o] = 0x7f, 0xff
        dirty, _, _ = attend(s)
        want, _, _ = attend(clean)
        assert torch.equal(dirty[:, :2], want[:, :2])
        assert bool(torch.isnan(dirty[:, 2:]).all())


def test_entries_that_are_no_page():
    """Read as zeros, and the status says so; beyond the length they are not looked at."""
    for entry in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        for page in (2, 16):
            s = scene([100, 90], 4, 2, 64, page, seed=14)
            zeroed = {**s, "k": s["k"].clone(), "v": s["v"].clone(), "ks": s["ks"].clone(), "vs": s["vs"].clone()}
            at = int(s["table"][0, 2])
            for x in ("k", "v", "ks", "vs"):
                zeroed[x][at] = 0
            want, wl, _ = attend(zeroed)
            s["table"][0, 2] = entry
            out, lse, status = attend(s)
            assert status == 2 and torch.equal(out, want) and torch.equal(lse, wl)


def test_lengths_that_no_row_holds():
    s = scene([112, 90], 4, 2, 64, 16, seed=15)
    s["table"][s["table"] < 0] = int(s["table"][0, 0])
    s["lens"] = torch.tensor([10 ** 6, -3], dtype=torch.int32)
    out, lse, status = attend(s)
    s["lens"] = torch.tensor([112, 0], dtype=torch.int32)
    want, _, _ = attend(s)
    assert status == 2 and torch.equal(out, want) and bool((out[1] == 0).all())


def test_axes_lie_apart():
    """Codes of k and v in one allocation, key heads a slice of more, scales in another order with gaps, another stream."""
    s = scene([100, 37], 4, 2, 64, 16, block=4, seed=19)
    pages = s["k"].shape[0]
    want, _, _ = attend(s)
    big = torch.zeros(pages, 2, 16, 5, 96, dtype=torch.int8, device="cuda")
    k, v = big[:, 0, :, 1:3, :64], big[:, 1, :, 1:3, :64]
    scales = torch.zeros(2, 2, pages + 1, 6, device="cuda")
    ks, vs = (scales[i, :, 1:, 1:5].permute(1, 2, 0) for i in (0, 1))
    for to, x in ((k, "k"), (v, "v"), (ks, "ks"), (vs, "vs")):
        to.copy_(s[x])
    table, lens, q = s["table"].cuda(), s["lens"].cuda(), s["q"].cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = api.paged_attention(q, api.BlockCache(k, v, ks, vs), table, lens, stream=st)
    st.synchronize()
    assert torch.equal(out.cpu(), want)


def test_empty_batches_and_tables():
    cache = api.BlockCache.empty(2, 16, 2, 64)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert api.paged_attention(torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), cache, none.view(0, 3), none).shape == (0, 4, 64)
    q, lse = torch.randn(2, 4, 64, device="cuda").bfloat16(), torch.empty(2, 4, device="cuda")
    out = api.paged_attention(q, cache, none.view(2, 0), torch.tensor([0, 0], dtype=torch.int32, device="cuda"), lse=lse)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())


def test_offsets_beyond_32_bits():
    """Codes that begin beyond 2^32 bytes."""
    page, hk, dim = 64, 8, 512
    pages = (1 << 32) // (page * hk * dim) + 24
    k, v = (torch.zeros(pages, page, hk, dim, dtype=torch.int8, device="cuda") for _ in "kv")
    ks, vs = (torch.ones(pages, 4, hk, device="cuda") for _ in "kv")
    g = torch.Generator(device="cuda").manual_seed(1)
    for x, s in ((k, ks), (v, vs)):
        x[-8:] = torch.randint(-127, 128, (8, page, hk, dim), device="cuda", generator=g).to(torch.int8)
        s[-8:] = torch.rand(8, 4, hk, device="cuda", generator=g) / 64
    table = torch.tensor([[pages - 1, pages - 3, pages - 8]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 1, 16, dim, device="cuda", generator=g).bfloat16()
    far = api.paged_attention(q, api.BlockCache(k, v, ks, vs), table, lens)
    near = api.paged_attention(q, api.BlockCache(*(x[-8:].clone() for x in (k, v, ks, vs))), table - (pages - 8), lens)
    assert torch.equal(far, near) and bool(far.abs().sum() > 0)
    starts = torch.tensor([0, 150], dtype=torch.int32, device="cuda")
    far = api.paged_read(api.BlockCache(k, v, ks, vs), table, starts, rows=150)
    near = api.paged_read(api.BlockCache(*(x[-8:].clone() for x in (k, v, ks, vs))), table - (pages - 8), starts, rows=150)
    assert all(torch.equal(a, b) for a, b in zip(far, near)) and bool(far[0].abs().sum() > 0)
