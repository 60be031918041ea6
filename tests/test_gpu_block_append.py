"""Appends to a cache with a scale for each block of tokens and head, value by value against 64 bits.

Tolerances (blocks_ref.Checker): k after its rotation is off by 2^-20 (|a| + |b|) of its pair at most (test_gpu_rope_append
says why), v not at all; a scale by that of the largest value and 2^-22 of itself (an e4m3 scale may be twice as large
where the largest value is that near to a border); a code by half a step (int8 0.5, e4m3 2^-4 of the value or half a
subnormal step, 2^-10), what the value is off, and 2^-20 of it for the product with the scale's inverse."""
import pytest
import torch

import blocks_ref
import paged_ref
from group_affine_bit_gb300 import api
from test_gpu_rope_append import parts, spread

pytestmark = pytest.mark.gpu

TYPES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


class Pool:
    """A pool on the GPU whose codes and scales are what some earlier requests left: any bytes, NaN and 0 among the scales."""

    def __init__(self, pages, page, heads, dim, kv, block, layout="token", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.kv, self.block, self.page = kv, block, page
        codes = [torch.randint(-127, 128, (pages, page, heads, dim), generator=g, dtype=torch.int8) for _ in "kv"]
        scales = [torch.rand(pages, page // block, heads, generator=g) * 0.02 for _ in "kv"]
        for s in scales:
            s[::3, 0, 0] = float("nan")
            s[1::3, 0, -1] = 0
        codes = [c.view(TYPES[kv]) for c in codes]
        if layout == "head":
            self.k, self.v = (c.transpose(1, 2).contiguous().cuda().transpose(1, 2) for c in codes)
            self.ks, self.vs = (s.permute(2, 0, 1).contiguous().cuda().permute(1, 2, 0) for s in scales)
        else:
            self.k, self.v = (c.cuda() for c in codes)
            both = torch.empty(pages, 2, page // block, heads, device="cuda")      # of k and v side by side
            self.ks, self.vs = both[:, 0], both[:, 1]
            self.ks.copy_(scales[0]), self.vs.copy_(scales[1])
        self.cache = api.BlockCache(self.k, self.v, self.ks, self.vs)

    def now(self):
        torch.cuda.synchronize()
        return [(c.float().cpu(), s.cpu()) for c, s in ((self.k, self.ks), (self.v, self.vs))]


def append(pool, qkv, pos, slots, hq, hk, dim, freqs, axis, neighbour, status=0, in_place=False):
    """One call, checked; returns how many (block, head) had to be brought to a larger scale."""
    axes = pos.shape[0]
    before = pool.now()
    dev = qkv.cuda()
    q, k, v = parts(dev, hq, hk, dim)
    rope = api.Rope(api.rope_turns(freqs), axis.cuda() if axes > 1 else None, neighbour=neighbour)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = api.rope_append(q, k, v, pos.cuda() if axes > 1 else pos[0].cuda(), slots.cuda(), rope, pool.cache, out=q if in_place else None, status=word)
    after = pool.now()
    assert int(word[0]) == status
    q64, k64, v64 = (x.double() for x in parts(qkv, hq, hk, dim))
    want, turned = (paged_ref.rope(x, pos, freqs, axis, neighbour) for x in (q64, k64))
    R = 2 * len(freqs)
    slack = [2.0 ** -20 * spread(x, R, neighbour) for x in (q64, k64)]
    assert bool(((got.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + slack[0] + 2.0 ** -134).all())
    check = blocks_ref.Checker(pool.kv, pool.block)
    return (check.check(before[0], after[0], turned, slack[1], slots) + check.check(before[1], after[1], v64, torch.zeros_like(v64), slots))


def rows_of(T, hq, hk, dim, g, size=1.0):
    gain = torch.exp(torch.randn((hq + 2 * hk) * dim, generator=g))
    return (torch.randn(T, (hq + 2 * hk) * dim, generator=g) * gain * size).bfloat16()


def places(spans, page, pages, g):
    """Slots of requests' tokens (first, count), each request on pages of its own, in any order of the pool."""
    order = torch.randperm(pages, generator=g).tolist()
    slots, positions = [], []
    for first, n in spans:
        own: dict = {}
        for i in range(first, first + n):
            if i // page not in own:
                own[i // page] = order.pop()
            slots.append(own[i // page] * page + i % page)
            positions.append(i)
    return torch.tensor(slots, dtype=torch.int32), torch.tensor(positions, dtype=torch.int32)


def run(spans, hq, hk, dim, page, block, kv, rotary=None, axes=1, neighbour=False, layout="token", seed=0, in_place=False):
    g = torch.Generator().manual_seed(seed)
    pages = sum(n // page + 2 for _, n in spans) + 1
    pool = Pool(pages, page, hk, dim, kv, block, layout, seed)
    slots, at = places(spans, page, pages, g)
    T, R = slots.numel(), dim if rotary is None else rotary
    pos = torch.stack([at + 1000 * a for a in range(axes)])
    axis = torch.tensor([i % axes for i in range(R // 2)], dtype=torch.uint8)
    return append(pool, rows_of(T, hq, hk, dim, g), pos, slots, hq, hk, dim, paged_ref.turns_of(R) if R else [], axis, neighbour, in_place=in_place)


SPANS = [(0, 1), (5, 1), (0, 37), (13, 50), (64, 16), (31, 2), (7, 130)]


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [16, 32, 64, 80, 128, 192, 256, 512])
def test_dims(dim, kv):
    assert run(SPANS, 4, 2, dim, 16, 16, kv, seed=dim) > 0


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("page,block", [(1, 1), (8, 1), (8, 2), (8, 8), (32, 16), (64, 64), (128, 4), (128, 128), (256, 128), (512, 32)])
def test_pages_and_blocks(page, block, kv):
    run(SPANS, 2, 2, 64, page, block, kv, seed=page + block)
    run(SPANS, 2, 1, 96, page, block, kv, seed=page, layout="head")


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("rotary,neighbour,axes", [(0, False, 1), (2, False, 1), (40, False, 2), (32, False, 3), (80, False, 1), (40, True, 2), (6, True, 1),
                                                   (80, True, 1), (16, True, 1), (78, False, 1), (78, True, 1)])
def test_rotations(rotary, neighbour, axes, kv):
    run(SPANS, 7, 1, 80, 8, 8, kv, rotary, axes, neighbour, seed=rotary, in_place=neighbour)


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("dim,block", [(512, 128), (256, 128), (512, 64)])
def test_blocks_whose_sines_fill_more_than_shared_memory_has_for_them(dim, block, kv):
    run([(0, 200), (100, 28), (128, 128)], 2, 1, dim, 128, block, kv, seed=dim)
    run([(0, 200), (100, 28)], 2, 1, dim, 128, block, kv, rotary=dim - 8, neighbour=True, seed=dim)


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("T,hq,hk", [(1, 1, 1), (1, 32, 8), (600, 3, 3), (2500, 2, 1)])
def test_one_token_and_many(T, hq, hk, kv):
    run([(3, T)], hq, hk, 64, 16, 16, kv, seed=T)
    run([(i * 5 % 48, 1) for i in range(T)], hq, hk, 64, 16, 16, kv, seed=T)


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("spans", [[(0, 200), (70, 60)], [(5, 1), (64, 1), (0, 30)], [(i * 9, 1 + i % 2) for i in range(40)]])
@pytest.mark.parametrize("dim,block", [(128, 64), (256, 128), (64, 128)])
def test_heads_shared_out_by_what_a_block_is_brought(dim, block, spans, kv):
    """Few tokens and large blocks: one CTA for all heads, or several, as whole blocks or single tokens come."""
    run(spans, 3, 8, dim, 128, block, kv, seed=dim + block)
    run(spans, 1, 5, dim, 128, block, kv, neighbour=True, seed=block)


@pytest.mark.parametrize("neighbour", [False, True])
def test_far_and_negative_positions(neighbour):
    """Phases are exact at any position: every quarter of a turn, from both ends of 32 bits."""
    g = torch.Generator().manual_seed(13)
    pool = Pool(8, 16, 2, 64, "int8", 8, seed=13)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (2, 40), generator=g).to(torch.int32)
    pos[0, :4] = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, -1])
    axis = torch.tensor([i % 2 for i in range(32)], dtype=torch.uint8)
    append(pool, rows_of(40, 3, 2, 64, g), pos, torch.arange(16, 56, dtype=torch.int32), 3, 2, 64, paged_ref.turns_of(64), axis, neighbour)
    # frequencies of a quarter, an eighth and three eighths of a turn, and just beside them: the borders between quarters
    freqs = [x * 2 * 3.141592653589793 for x in (0.25, 0.125, 0.375, 0.5, 0.75, 0.125 + 2.0 ** -40, 0.125 - 2.0 ** -40, 0.9999999)] * 4
    append(pool, rows_of(40, 3, 2, 64, g), torch.arange(40, dtype=torch.int32)[None], torch.arange(16, 56, dtype=torch.int32), 3, 2, 64, freqs,
           torch.zeros(32, dtype=torch.uint8), neighbour)


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("block", [1, 4, 16, 64])
def test_calls_of_many_sizes(block, kv):
    """Every way in which rows are shared out: a row to a CTA and sixteen, blocks that begin anywhere in them, none at all."""
    for T, spans in ((40, [(i, 1) for i in range(40)]), (330, [(7, 300), (0, 30)]), (1300, [(3, 1200), (60, 100)]),
                     (5000, [(5, 4000), (1, 900), (2, 100)]), (4900, [(i % 64, 1 + i % 3) for i in range(2450)])):
        run(spans, 1, 1, 32, 64, block, kv, seed=T)


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
def test_a_block_filled_token_by_token(kv):
    """The scale follows the largest value so far; what is there already is rounded again where it grows."""
    g = torch.Generator().manual_seed(1)
    pool, grown = Pool(3, 16, 2, 64, kv, 16, seed=2), 0
    axis, freqs = torch.zeros(32, dtype=torch.uint8), paged_ref.turns_of(64)
    for i in range(16):
        qkv = rows_of(2, 2, 2, 64, g, size=4.0 if i in (5, 11) else 0.01 if i == 0 else 1.0)
        slots = torch.tensor([16 + i, 32 + (i + 3) % 16], dtype=torch.int32)       # the second begins anew on its way
        grown += append(pool, qkv, torch.tensor([[i, i + 3]], dtype=torch.int32), slots, 2, 2, 64, freqs, axis, False)
    assert grown >= 8
    # and the whole block is within a few roundings of what was written: half a step of each scale that it had
    assert bool(torch.isfinite(pool.now()[0][1][1:]).all())


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
def test_tokens_written_again_do_not_shrink_a_scale(kv):
    """Drafted tokens that were refused: their slots are written once more."""
    g = torch.Generator().manual_seed(3)
    pool = Pool(2, 16, 2, 64, kv, 16, seed=4)
    axis, freqs = torch.zeros(32, dtype=torch.uint8), paged_ref.turns_of(64)
    slots = torch.arange(16, 32, dtype=torch.int32)
    pos = torch.arange(16, dtype=torch.int32)[None]
    append(pool, rows_of(16, 2, 2, 64, g), pos, slots, 2, 2, 64, freqs, axis, False)
    before = [s.clone() for _, s in pool.now()]
    append(pool, rows_of(5, 2, 2, 64, g, size=0.125), pos[:, 6:11], slots[6:11], 2, 2, 64, freqs, axis, False)
    assert all(torch.equal(a[1], s[1]) for a, (_, s) in zip(before, pool.now()))


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
def test_rows_that_are_not_kept(kv):
    g = torch.Generator().manual_seed(5)
    pool = Pool(6, 16, 2, 64, kv, 8, seed=6)
    slots = torch.tensor([3, 4, -1, -1, 40, 41, 42, 43, 44, 96, 2 ** 31 - 1, -7, 48, -1], dtype=torch.int32)   # 96 and on: no pages
    pos = torch.arange(14, dtype=torch.int32)[None]
    axis, freqs = torch.zeros(32, dtype=torch.uint8), paged_ref.turns_of(64)
    append(pool, rows_of(14, 2, 2, 64, g), pos, slots, 2, 2, 64, freqs, axis, False, status=2)
    append(pool, rows_of(3, 2, 2, 64, g), pos[:, :3], torch.full((3,), -1, dtype=torch.int32), 2, 2, 64, freqs, axis, False)


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("neighbour", [False, True])
def test_values_that_are_not_finite(kv, neighbour):
    """Infinities get the largest code and do not count for the scale; NaN is NaN in e4m3, 0 in int8; the other values of the
    block are as if they were not there."""
    g = torch.Generator().manual_seed(7)
    pool = Pool(3, 16, 1, 32, kv, 16, seed=8)
    qkv = rows_of(6, 1, 1, 32, g)
    qkv[1, 64 + 3], qkv[2, 64 + 9], qkv[4, 64 + 31] = float("inf"), float("-inf"), float("nan")      # of v
    qkv[3, 32 + 30], qkv[0, 32 + 31] = float("inf"), float("nan")                                        # of k, beside the rotation
    slots = torch.arange(16, 22, dtype=torch.int32)
    append(pool, qkv, torch.arange(6, dtype=torch.int32)[None], slots, 1, 1, 32, paged_ref.turns_of(16), torch.zeros(8, dtype=torch.uint8), neighbour)
    codes = pool.v.float().cpu()[1, :, 0]
    most = 127 if kv == "int8" else 448
    assert codes[1, 3] == most and codes[2, 9] == -most and (codes[4, 31] == 0 if kv == "int8" else torch.isnan(codes[4, 31]))


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
def test_zeros_and_the_ends_of_the_scales_range(kv):
    pool = Pool(6, 16, 1, 32, kv, 16, seed=9)
    for i, size in enumerate((0.0, 1e-30, 2.0 ** -42, 1e10, 1e20, 3e38)):
        g = torch.Generator().manual_seed(i)
        qkv = (torch.rand(4, 3 * 32, generator=g) * size).bfloat16()
        slots = torch.arange(16 * i, 16 * i + 4, dtype=torch.int32)
        append(pool, qkv, torch.arange(4, dtype=torch.int32)[None], slots, 1, 1, 32, [], torch.zeros(0, dtype=torch.uint8), False)
    s = pool.vs.cpu()[:, 0, 0]
    assert s[0] == s[1] == 2.0 ** -48 and s[4] == s[5] == 2.0 ** 48 and bool((pool.v[0, :4].float() == 0).all())


def test_powers_of_two_at_the_border():
    """e4m3: 448 times a power of two needs that power, the next bf16 number twice it."""
    pool = Pool(2, 16, 1, 16, "e4m3", 1, seed=10)
    v = torch.zeros(4, 48, dtype=torch.bfloat16)
    v[0, 32], v[1, 32], v[2, 33], v[3, 40] = 448.0, 450.0, -7.0, 1.75 * 2 ** -20
    slots = torch.arange(16, 20, dtype=torch.int32)
    append(pool, v, torch.zeros(1, 4, dtype=torch.int32), slots, 1, 1, 16, [], torch.zeros(0, dtype=torch.uint8), False)
    assert pool.vs[1, :4, 0].tolist() == [1.0, 2.0, 2.0 ** -6, 2.0 ** -28]


def test_another_stream_and_a_captured_step():
    """A step that a graph replays, on its own stream: the lengths on the GPU decide the slots."""
    g = torch.Generator().manual_seed(11)
    one, two = Pool(4, 16, 2, 64, "int8", 16, seed=12), Pool(4, 16, 2, 64, "int8", 16, seed=12)
    rope = api.Rope(api.rope_turns(paged_ref.turns_of(64)))
    rows = rows_of(3, 4, 2, 64, g).cuda()
    pos, slots = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
    out = torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        api.rope_append(*parts(rows, 4, 2, 64), pos, slots, rope, one.cache, out=out)
    for i in range(8):
        now = torch.tensor([i, 16 + i + 3, 33 + i], dtype=torch.int32)
        rows.copy_(rows_of(3, 4, 2, 64, g))
        pos.copy_(now % 16), slots.copy_(now)
        torch.cuda.synchronize()
        graph.replay()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        want = api.rope_append(*parts(rows, 4, 2, 64), pos, slots, rope, two.cache, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(torch.equal(a[0], b[0]) and torch.equal(a[1].nan_to_num(-1), b[1].nan_to_num(-1)) for a, b in zip(one.now(), two.now()))


def test_pool_beyond_32_bits():
    """Codes and rows that begin beyond 2^32 bytes."""
    page, hk, dim = 64, 8, 512
    pages = (1 << 32) // (page * hk * dim) + 24
    k, v = (torch.zeros(pages, page, hk, dim, dtype=torch.int8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros(pages, 4, hk, device="cuda") for _ in "kv")
    cache = api.BlockCache(k, v, ks, vs)
    row = torch.randn(3, hk, dim, device="cuda").bfloat16()
    slots = torch.tensor([pages * page - 1, (pages - 2) * page, (pages - 2) * page + 1], dtype=torch.int32, device="cuda")
    api.rope_append(row, row, row, torch.zeros(3, dtype=torch.int32, device="cuda"), slots, api.Rope(api.rope_turns([1.0])), cache)
    small = api.BlockCache.empty(2, page, hk, dim, block=16)
    small.k.zero_(), small.v.zero_()
    near = torch.tensor([2 * page - 1, 0, 1], dtype=torch.int32, device="cuda")
    api.rope_append(row, row, row, torch.zeros(3, dtype=torch.int32, device="cuda"), near, api.Rope(api.rope_turns([1.0])), small)
    assert torch.equal(v[-1], small.v[1]) and torch.equal(k[-2], small.k[0]) and torch.equal(vs[-1], small.v_scale[1]) and int(v[:-2].count_nonzero()) == 0
    assert bool(small.v[1, -1].any()) and int(v[-1, :-1].count_nonzero()) == 0
