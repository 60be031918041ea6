"""Tokens of a paged cache read back as rows, against 64 bits: one rounding to bf16 (2^-8 of the value) and one of the
product in fp32 (2^-24); a bf16 cache's values as they are."""
import pytest
import torch

import blocks_ref
from group_affine_bit_gb300 import api

pytestmark = pytest.mark.gpu


def pool(pages, page, heads, dim, kv, block, seed, layout="token"):
    """(cache, k, v float64): every code of its type but NaN."""
    g = torch.Generator().manual_seed(seed)
    shape = (pages, page, heads, dim)
    put = lambda t: t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if layout == "head" else t.cuda()  # noqa: E731
    if kv == "bf16":
        k, v = (torch.randn(shape, generator=g).bfloat16() for _ in "kv")
        return api.KVCache(put(k), put(v)), k.double(), v.double()
    codes = [torch.randint(-128, 128, shape, generator=g).to(torch.int8) for _ in "kv"]
    if kv != "int8":
        codes = [torch.where((c & 0x7f) == 0x7f, 0, c).view(torch.float8_e4m3fn) for c in codes]
    if kv == "e4m3 heads":
        scales = [torch.rand(heads, generator=g) + 0.1 for _ in "kv"]
        return (api.KVCache(*(put(c) for c in codes), *(s.cuda() for s in scales)),
                *(c.double() * s.double()[:, None] for c, s in zip(codes, scales)))
    scales = [torch.rand(pages, page // block, heads, generator=g) + 0.1 for _ in "kv"]
    return (api.BlockCache(*(put(c) for c in codes), *(put(s) for s in scales)), *(blocks_ref.values(c, s) for c, s in zip(codes, scales)))


def check(cache, k64, v64, spans, seed=0, first=True, extra=3, strided=False, bad=()):
    """spans: (first token, count) of each request; `bad`: (request, entry of its row, number) that is no page."""
    g = torch.Generator().manual_seed(seed)
    page, wide = cache.page, max([-(-(f + n) // cache.page) for f, n in spans] + [1])
    table = torch.stack([torch.randperm(cache.pages, generator=g)[:wide] for _ in spans]).to(torch.int32) if cache.pages >= wide else \
        torch.randint(0, cache.pages, (len(spans), wide), generator=g, dtype=torch.int32)
    for b, e, x in bad:
        table[b, e] = x
    rows = sum(n for _, n in spans)
    starts = torch.tensor([0] + [n for _, n in spans]).cumsum(0).to(torch.int32)
    shape = (rows + extra, cache.heads, cache.dim)
    if strided:
        k = torch.full((shape[0], cache.heads + 1, cache.dim + 8), 7.0, dtype=torch.bfloat16, device="cuda")[:, 1:, : cache.dim]
        v = torch.full((cache.heads, shape[0], cache.dim), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    else:
        k, v = (torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = torch.tensor([f for f, _ in spans], dtype=torch.int32).cuda() if first else None
    api.paged_read(cache, table.cuda(), starts.cuda(), first=at, k=k, v=v, status=status)
    torch.cuda.synchronize()
    missing = False
    for got, x in ((k.cpu().double(), k64), (v.cpu().double(), v64)):
        for b, (f, n) in enumerate(spans):
            for j in range(n):
                p = int(table[b, (f + j) // page])
                want = x[p, (f + j) % page] if 0 <= p < cache.pages else torch.zeros(shape[1:], dtype=torch.float64)
                missing |= not 0 <= p < cache.pages
                here = got[int(starts[b]) + j]
                assert bool(((here - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -23)).all()) if cache.k.dtype != torch.bfloat16 else torch.equal(here, want)
        assert bool((got[rows:] == 7).all())
    assert int(status[0]) == (2 if missing else 0)
    if strided:
        assert bool((k._base[:, 0] == 7).all()) and bool((k._base[:, :, cache.dim:] == 7).all())
    return k, v


KINDS = ["bf16", "e4m3 heads", "e4m3", "int8"]
SPANS = [(0, 5), (3, 0), (7, 30), (0, 1), (63, 66), (0, 0), (128, 9)]


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("dim", [16, 80, 128, 512])
def test_dims(dim, kv):
    check(*pool(12, 16, 3, dim, kv, 16, dim), SPANS, seed=dim)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("page,block", [(1, 1), (8, 1), (8, 8), (32, 16), (128, 128), (256, 2)])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_pages_blocks_and_orders(page, block, layout, kv):
    check(*pool(9, page, 2, 48, kv, block, page, layout), SPANS, seed=page, strided=layout == "head")


@pytest.mark.parametrize("kv", KINDS)
def test_whole_requests_from_their_first_token(kv):
    check(*pool(20, 16, 2, 64, kv, 8, 1), [(0, n) for n in (17, 0, 1, 64, 100)], first=False)
    check(*pool(20, 16, 2, 64, kv, 8, 1), [(0, 0)] * 4, first=False)


@pytest.mark.parametrize("kv", KINDS)
def test_entries_that_are_no_page_read_as_zeros(kv):
    for x in (-1, 12, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        check(*pool(12, 16, 2, 32, kv, 16, 2), SPANS, bad=[(2, 1, x), (4, 7, x)])


def test_many_requests_and_many_heads():
    check(*pool(40, 8, 1, 16, "int8", 8, 3), [(i % 5, i * 7 % 4) for i in range(1500)], seed=3)
    check(*pool(40, 8, 1, 16, "e4m3", 8, 3), [(i % 5, i * 5 % 3) for i in range(3000)], seed=5)   # more than shared memory keeps
    check(*pool(3, 2, 300, 512, "int8", 2, 4), [(0, 5), (1, 2)], seed=4)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_rows_that_do_not_fit_and_tokens_beyond_the_table(kv):
    """As many rows as there are, and the status says so; tokens outside a request's row of the table are zeros."""
    cache, k64, _ = pool(6, 16, 2, 32, kv, 16, 5)
    table = torch.tensor([[4, 1]], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    whole, _ = api.paged_read(cache, table, torch.tensor([0, 20], dtype=torch.int32, device="cuda"), rows=20)
    k, v = api.paged_read(cache, table, torch.tensor([0, 20], dtype=torch.int32, device="cuda"), rows=11, status=status)
    assert int(status[0]) == 2 and torch.equal(k, whole[:11])
    for first in (-3, 25, 2 ** 31 - 1, -2 ** 31):
        status.zero_()
        k, v = api.paged_read(cache, table, torch.tensor([0, 10], dtype=torch.int32, device="cuda"),
                              torch.tensor([first], dtype=torch.int32, device="cuda"), rows=10, status=status)
        assert int(status[0]) == 2
        for j in range(10):
            if not 0 <= first + j < 32:
                assert not bool(k[j].any()) and not bool(v[j].any())
            elif kv == "bf16":
                assert torch.equal(k[j].cpu().double(), k64[(4, 1)[(first + j) // 16], (first + j) % 16])


def test_refusals_and_made_rows():
    cache = api.BlockCache.empty(2, 16, 2, 32)
    table, starts = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    k = torch.empty(3, 2, 32, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(), dict(k=k), dict(k=k, v=k.clone(), rows=3), dict(k=k, v=k.float()), dict(k=k[:, :1], v=k[:, :1]), dict(rows=3, first=starts),
                dict(k=k.transpose(1, 2).contiguous().transpose(1, 2), v=k)):
        with pytest.raises(ValueError):
            api.paged_read(cache, table, starts, **bad)
    with pytest.raises(ValueError):
        api.paged_read(cache, table, starts[:1], rows=3)
    assert api.paged_read(cache, table, starts, rows=3)[0].shape == (3, 2, 32)
    none = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    assert api.paged_read(cache, none, starts[:1], rows=0)[0].shape == (0, 2, 32)


def test_the_same_rows_of_one_have_any_stride():
    cache, k64, _ = pool(3, 16, 1, 32, "bf16", 16, 6)
    table, starts = torch.tensor([[2]], dtype=torch.int32, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    flat = torch.zeros(64, dtype=torch.bfloat16, device="cuda")
    k, v = flat[:32].as_strided((1, 1, 32), (5, 3, 1)), flat[32:].as_strided((1, 1, 32), (5, 3, 1))
    api.paged_read(cache, table, starts, k=k, v=v)
    assert torch.equal(flat[:32].cpu().double(), k64[2, 0, 0])


def test_another_stream_and_a_captured_read():
    cache, k64, _ = pool(8, 16, 2, 64, "int8", 16, 7)
    table = torch.tensor([[4, 1, 6], [0, 2, 3]], dtype=torch.int32, device="cuda")
    starts, first = torch.tensor([0, 9, 20], dtype=torch.int32, device="cuda"), torch.tensor([3, 30], dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(40, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.paged_read(cache, table, starts, first=first, k=k, v=v)
    for counts, at in (((9, 11), (3, 30)), ((0, 18), (7, 0)), ((40, 0), (0, 0))):
        starts.copy_(torch.tensor([0, counts[0], sum(counts)], dtype=torch.int32)), first.copy_(torch.tensor(at, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        side = torch.cuda.Stream()
        want = api.paged_read(cache, table, starts, first=first, rows=sum(counts), stream=side)
        torch.cuda.synchronize()
        assert torch.equal(k[: sum(counts)], want[0]) and torch.equal(v[: sum(counts)], want[1])
