"""Attention over the paged cache, against a 64-bit form (bounds: paged_ref.attention_bounds)."""
import math

import pytest
import torch

import paged_ref
from group_affine_bit_gb300 import api

pytestmark = pytest.mark.gpu


def scene(lens, hq, hk, dim, page, kv="bf16", tokens=1, seed=0, layout="token", spare=2, fill=float("nan")):
    """A pool whose every value that no request holds is `fill`."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=g)
    wide = max(max(used), 1)
    table = torch.full((B, wide), -1, dtype=torch.int32)
    shape = (pages, page, hk, dim)
    k, v = torch.randn(shape, generator=g), torch.randn(shape, generator=g)
    held = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        table[b, : used[b]] = order[at: at + used[b]].to(torch.int32)
        for i in range(used[b]):
            held[order[at + i], : min(page, n - i * page)] = True
        at += used[b]
    dt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    if kv == "e4m3":
        k, v = k * 32, v * 32
    k[~held], v[~held] = fill, fill
    scales = [torch.rand(hk, generator=g) / 32 + 0.01 for _ in "kv"] if kv == "e4m3" else [None, None]
    q = torch.randn(B, tokens, hq, dim, generator=g).bfloat16()
    return dict(q=q, k=k.to(dt), v=v.to(dt), table=table, lens=torch.tensor(lens, dtype=torch.int32), k_scale=scales[0],
                v_scale=scales[1], layout=layout, kv=kv)


def on_gpu(t, layout):
    return t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if layout == "head" else t.cuda()


def attend(s, scale=None, window=0, **kw):
    cache = api.KVCache(on_gpu(s["k"], s["layout"]), on_gpu(s["v"], s["layout"]),
                        *(x.cuda() if x is not None else None for x in (s["k_scale"], s["v_scale"])))
    q = s["q"].cuda()
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = api.paged_attention(q, cache, s["table"].cuda(), s["lens"].cuda(), scale=scale, window=window, lse=lse, status=status, **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu(), int(status[0])


def check(s, scale=None, window=0):
    out, lse, status = attend(s, scale, window)
    assert status == 0
    dim = s["q"].shape[-1]
    sc = dim ** -0.5 if scale is None else scale
    want, wl, mag, room = paged_ref.attention(s["q"], s["k"].double(), s["v"].double(), s["table"], s["lens"], sc, window,
                                              s["k_scale"], s["v_scale"])
    b_out, b_lse = paged_ref.attention_bounds(want, wl, mag, room, dim, 9 if s["kv"] == "bf16" else 12)
    assert bool(((out.double() - want).abs() <= b_out).all())
    empty = torch.isinf(wl)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    assert bool(((lse.double() - wl).abs() <= b_lse)[~empty].all())
    assert bool((out[empty] == 0).all())
    return out, lse


EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 1000]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 128, 192, 256, 320, 512])
def test_lengths_and_dims(dim, kv):
    check(scene(EDGES, 4, 2, dim, 16, kv, seed=dim))


@pytest.mark.parametrize("page", [1, 2, 4, 8, 32, 64, 256])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_pages_and_orders(page, layout):
    check(scene([1, 70, 129, 5, 257], 6, 2, 96, page, seed=page, layout=layout))
    check(scene([1, 70, 129, 5, 257], 6, 2, 96, page, "e4m3", tokens=3, seed=page, layout=layout), window=33)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256, 512])
@pytest.mark.parametrize("hq,hk,tokens", [(1, 1, 1), (7, 1, 1), (8, 8, 2), (10, 1, 1), (16, 1, 2), (12, 2, 5), (16, 1, 4),
                                          (5, 1, 13), (16, 1, 7), (40, 2, 8), (2, 2, 64)])
def test_rows_that_share_a_key_head(hq, hk, tokens, dim, kv):
    check(scene([3, 64, 150, 0, 331], hq, hk, dim, 16, kv, tokens=tokens, seed=hq + tokens))


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 63, 64, 65, 500, 5000])
@pytest.mark.parametrize("tokens", [1, 5])
def test_windows(window, tokens):
    check(scene([0, 1, 3, 16, 64, 65, 130, 700], 8, 2, 128, 8, tokens=tokens, seed=window), window=window)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 4, 2 ** 31 - 64])
@pytest.mark.parametrize("tokens", [1, 5, 64])
def test_windows_that_hide_nothing(window, tokens):
    s = scene([0, 1, 2, 3, 4, 5, 6, 63, 64, 130], 2, 2, 64, 8, tokens=tokens, seed=tokens)
    got, want = check(s, window=window), check(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_window_beyond_32_bits_is_refused():
    s = scene([5], 2, 2, 64, 8)
    for window in (2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1):
        with pytest.raises(ValueError):
            attend(s, window=window)
    with pytest.raises(api.AffqmmError):
        attend(s, window=-1)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.25, 30.0])
def test_scales(scale):
    """Sharp, flat and negative scores; at 30 the running maximum moves many times."""
    check(scene([1, 65, 900], 8, 2, 64, 16, seed=2), scale=scale)


def test_rising_scores():
    """Keys whose scores rise along the cache: every tile has a new maximum."""
    s = scene([1500], 2, 1, 64, 16, seed=1)
    s["q"] = torch.ones(1, 1, 2, 64).bfloat16()
    order = s["table"][0].long()
    ramp = (torch.arange(1504, dtype=torch.float32) / 50).reshape(94, 16, 1, 1)
    s["k"][order] = (ramp + torch.zeros(94, 16, 1, 64)).bfloat16()
    check(s, scale=0.5)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,dim", [(8, 64), (24, 128), (128, 256)])
@pytest.mark.parametrize("nats", [10, 15, 16, 17, 18])
def test_small_probabilities_beside_a_large_one(nats, hq, dim, kv):
    """One key `nats` above the others, whose value is zero: the others are the whole output, and all alike, so that
    what their probabilities lose does not average out.  Requests enough that a run takes whole ones."""
    s = scene([600] * 40, hq, 8, dim, 16, kv, seed=nats)
    k, v = s["k"].float(), s["v"].float().abs()
    k[torch.isfinite(k)] = 0
    for b in range(40):
        at = (0, 300, 599)[b % 3]
        p, o = int(s["table"][b, at // 16]), at % 16
        k[p, o, :, 0], v[p, o] = 1, 0
    s["k"], s["v"] = k.to(s["k"].dtype), v.to(s["v"].dtype)
    s["q"] = torch.zeros_like(s["q"])
    s["q"][..., 0] = 1
    if kv == "e4m3":
        s["k_scale"] = torch.ones(8)
    check(s, scale=float(nats))


@pytest.mark.parametrize("hq,hk,dim,lens,kv", [(8, 1, 128, [20011], "bf16"), (32, 8, 256, [9000, 31], "bf16"), (2, 2, 64, [30000, 1, 64, 7000], "e4m3"),
                                              (16, 1, 512, [5000, 3001], "e4m3")])
def test_long_caches_are_split_and_joined(hq, hk, dim, lens, kv):
    check(scene(lens, hq, hk, dim, 32, kv, seed=7))


def test_many_short_requests():
    check(scene([1 + (i * 37) % 90 for i in range(700)], 2, 1, 64, 16, seed=3))


def test_same_inputs_same_bits():
    s = scene([8000, 17, 3000, 1, 500], 8, 2, 128, 16, seed=4)
    first = attend(s)
    for _ in range(5):
        again = attend(s)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_what_a_later_token_sees_does_not_reach_an_earlier_one(bad, kv):
    """Five tokens; the values and keys of the last three are not finite: rows
    that do not see them are as if they were zeros, rows that do are NaN."""
    if kv == "e4m3" and not math.isnan(bad):
        pytest.skip("e4m3 has no infinities")
    for dim in (64, 256):
        s = scene([70, 5, 129], 4, 2, dim, 16, kv, tokens=5, seed=11)
        clean = {**s, "k": s["k"].clone(), "v": s["v"].clone()}
        for b, n in enumerate(s["lens"].tolist()):
            for i in range(n - 3, n):
                p, o = int(s["table"][b, i // 16]), i % 16
                v, k = s["v"].float(), s["k"].float()
                v[p, o], k[p, o] = bad, float("nan")
                s["v"], s["k"] = v.to(s["v"].dtype), k.to(s["k"].dtype)
        dirty, _, _ = attend(s)
        want, _, _ = attend(clean)
        assert torch.equal(dirty[:, :2], want[:, :2])
        assert bool(torch.isnan(dirty[:, 2:]).all())


def test_a_window_leaves_what_it_drops():
    """Values that are not finite behind the window, seen by the first tokens only."""
    s = scene([100, 40], 4, 2, 128, 16, tokens=5, seed=12)
    clean = {**s, "v": s["v"].clone()}
    for b, n in enumerate(s["lens"].tolist()):
        for i in range(n - 5 + 1 - 20, n - 5 + 1 - 20 + 2):      # the oldest keys of tokens 0 and 1
            s["v"][int(s["table"][b, i // 16]), i % 16] = float("nan")
    dirty, _, _ = attend(s, window=20)
    want, _, _ = attend(clean, window=20)
    assert torch.equal(dirty[:, 2:], want[:, 2:]) and bool(torch.isnan(dirty[:, :2]).all())


def test_nan_and_infinite_scores():
    """As the formula has them: a NaN key or an infinite score makes its rows NaN, others not."""
    s = scene([100, 90], 4, 2, 64, 16, seed=13)
    s["k"][int(s["table"][0, 2]), 3, 0] = float("nan")
    s["q"][1, 0, 3] = float("inf")
    out, lse, _ = attend(s)
    assert bool(torch.isnan(out[0, 0, :2]).all()) and bool(torch.isfinite(out[0, 0, 2:]).all())
    assert bool(torch.isfinite(out[1, 0, :3]).all()) and bool(torch.isnan(out[1, 0, 3]).all())


@pytest.mark.parametrize("tokens", [1, 3])
@pytest.mark.parametrize("dim", [64, 128, 256, 512])
def test_infinite_values_stay_infinite(dim, tokens):
    """As the formula has them: a row that sees an infinite value has it in that place, and NaN where both signs meet;
    other rows and places are as if it were zero."""
    s = scene([100, 6000, 5], 4, 2, dim, 16, tokens=tokens, seed=dim)
    clean = {**s, "v": s["v"].clone()}
    hit = []                                     # (request, token from which it is seen, key head, value, what is there)
    for b, n in enumerate(s["lens"].tolist()):
        for key, h, d, x in ((0, 0, 3, math.inf), (n - 1, 1, 5, -math.inf), (n // 3, 1, 9, math.inf), (n // 2, 1, 9, -math.inf)):
            p, o = int(s["table"][b, key // 16]), key % 16
            s["v"][p, o, h, d], clean["v"][p, o, h, d] = x, 0
            hit.append((b, max(0, key - (n - tokens)), h, d, x if d != 9 else math.nan))
    out, lse, _ = attend(s)
    want, wl, _ = attend(clean)
    for b, j, h, d, x in hit:
        want[b, j:, 2 * h: 2 * h + 2, d] = x
    assert torch.equal(lse, wl)
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.equal(out.nan_to_num(7), want.nan_to_num(7))


def test_entries_that_are_no_page():
    """Read as zeros, and the status says so; beyond the length they are not looked at."""
    for entry in (-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1):
        s = scene([100, 90], 4, 2, 64, 16, seed=14)
        zeroed = {**s, "k": s["k"].clone(), "v": s["v"].clone()}
        page = int(s["table"][0, 2])
        zeroed["k"][page], zeroed["v"][page] = 0, 0
        want, _, _ = attend(zeroed)
        s["table"][0, 2] = entry
        out, _, status = attend(s)
        assert status == 2 and torch.equal(out, want)


def test_lengths_that_no_row_holds():
    s = scene([100, 90], 4, 2, 64, 16, seed=15, fill=0.5)
    s["table"][s["table"] < 0] = 0
    s["lens"] = torch.tensor([10 ** 6, -3], dtype=torch.int32)
    out, lse, status = attend(s)
    s["lens"] = torch.tensor([7 * 16, 0], dtype=torch.int32)
    want, _, _ = attend(s)
    assert status == 2 and torch.equal(out, want) and bool((out[1] == 0).all())


def test_views_streams_and_one_token_shape():
    """q as a view of the stacked projection's rows, a strided out, a strided table, another stream."""
    s = scene([100, 1, 345], 8, 2, 128, 16, seed=16)
    want, wl, _ = attend(s)
    rows = torch.zeros(3, 12 * 128 + 64, dtype=torch.bfloat16, device="cuda")
    q = rows[:, 64: 64 + 8 * 128].view(3, 8, 128)
    q.copy_(s["q"][:, 0].cuda())
    wide = torch.full((3, 40), -9, dtype=torch.int32, device="cuda")
    table = wide[:, 3: 3 + s["table"].shape[1]]
    table.copy_(s["table"].cuda())
    cache = api.KVCache(s["k"].cuda(), s["v"].cuda())
    big = torch.full((3, 8, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    lens = s["lens"].cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = api.paged_attention(q, cache, table, lens, out=big[:, :, 64:192], stream=st)
    st.synchronize()
    assert torch.equal(out.cpu(), want[:, 0])
    assert bool((big[:, :, :64] == 5).all()) and bool((big[:, :, 192:] == 5).all())


def test_axes_of_one_have_any_stride():
    s = scene([100], 2, 1, 64, 16, seed=20)
    want, _, _ = attend(s)
    cache, table, lens = api.KVCache(s["k"].cuda(), s["v"].cuda()), s["table"].cuda(), s["lens"].cuda()
    rows = torch.zeros(3, 2 * 64 + 3, dtype=torch.bfloat16, device="cuda")
    q = rows.as_strided((3, 2, 64), (131, 64, 1))[:1]     # the first of rows whose pitch is odd
    q.copy_(s["q"][:, 0].cuda())
    assert q.stride(0) % 8 != 0
    assert torch.equal(api.paged_attention(q, cache, table, lens).cpu(), want[:, 0])
    flat = s["q"][0, 0].cuda()
    q4 = flat.as_strided((1, 1, 2, 64), (3, 5, 64, 1))
    assert torch.equal(api.paged_attention(q4, cache, table, lens, out=torch.empty_like(flat).as_strided((1, 1, 2, 64), (7, 1, 64, 1))).cpu(), want)
    rope, i = api.Rope(api.rope_turns([0.5] * 32)), torch.tensor([3], dtype=torch.int32, device="cuda")
    plain = api.rope_append(q.contiguous(), q[:, :1].contiguous(), q[:, :1].contiguous(), i, i, rope, cache)
    k1 = flat.as_strided((1, 1, 64), (9, 11, 1))
    assert torch.equal(api.rope_append(q, k1, k1, i, i, rope, cache), plain)


def test_offsets_beyond_32_bits():
    """A pool whose last pages begin beyond 2^31 elements (and 2^32 bytes)."""
    pages, page, hk, dim = (1 << 31) // (64 * 2 * 256) + 40, 64, 2, 256
    k, v = (torch.zeros(pages, page, hk, dim, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    g = torch.Generator(device="cuda").manual_seed(1)
    k[-8:] = torch.randn(8, page, hk, dim, device="cuda", generator=g).bfloat16()
    v[-8:] = torch.randn(8, page, hk, dim, device="cuda", generator=g).bfloat16()
    assert (pages - 8) * k.stride(0) > 2 ** 31
    table = torch.tensor([[pages - 1, pages - 3, pages - 8]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([150], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 1, 4, dim, device="cuda", generator=g).bfloat16()
    far = api.paged_attention(q, api.KVCache(k, v), table, lens)
    near = api.paged_attention(q, api.KVCache(k[-8:].clone(), v[-8:].clone()), table - (pages - 8), lens)
    assert torch.equal(far, near) and bool(far.abs().sum() > 0)
    # and the append reaches them
    row = torch.randn(2, 2, dim, device="cuda", generator=g).bfloat16()
    slots = torch.tensor([pages * page - 1, (pages - 2) * page], dtype=torch.int32, device="cuda")
    api.rope_append(row, row, row, torch.zeros(2, dtype=torch.int32, device="cuda"), slots, api.Rope(api.rope_turns([1.0])), api.KVCache(k, v))
    assert torch.equal(v[-1, -1], row[0]) and torch.equal(k[-2, 0], row[1])


def test_a_captured_step_follows_the_lengths():
    """One captured graph, replayed as the lengths on the GPU grow."""
    s = scene([64, 200, 1], 8, 2, 128, 16, seed=17, spare=40, fill=0.25)
    used = set(s["table"][s["table"] >= 0].tolist())
    free = [p for p in range(s["k"].shape[0]) if p not in used]
    wide = torch.full((3, 16), -1, dtype=torch.int32)
    wide[:, : s["table"].shape[1]] = s["table"]
    for b in range(3):
        for i in range(16):
            if wide[b, i] < 0 and free:
                wide[b, i] = free.pop()
    s["table"] = wide
    cache = api.KVCache(s["k"].cuda(), s["v"].cuda())
    q, table, lens = s["q"].cuda(), wide.cuda(), s["lens"].cuda()
    ws = api.Workspace()
    out = torch.empty_like(q)
    api.paged_attention(q, cache, table, lens, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.paged_attention(q, cache, table, lens, out=out, workspace=ws)
    for step in range(4):
        now = torch.tensor([64 + 13 * step, 200 + step, 1 + 40 * step], dtype=torch.int32)
        lens.copy_(now.cuda())
        graph.replay()
        torch.cuda.synchronize()
        want = api.paged_attention(q, cache, table, now.cuda())
        assert torch.equal(out, want)
    assert api.workspace_status(ws.buf) == 0


def test_the_workspace_serves_projections_and_attention():
    """One stream's default workspace: its counters are zero again after each call."""
    from group_affine_bit_gb300 import synth
    x, codes, sc, bi = synth.problem(4, 64, 1, 512, 2048, seed=1)
    w = api.pack(codes.cuda(), sc.cuda(), bi.cuda(), 4, 64)
    y0 = api.run(w, x.cuda()).cpu()
    s = scene([9000], 8, 2, 128, 16, seed=18)
    a0 = attend(s)[0]
    for _ in range(3):
        assert torch.equal(api.run(w, x.cuda()).cpu(), y0) and torch.equal(attend(s)[0], a0)
    ws = api.default_workspace(torch.device("cuda", 0))
    assert bool((ws.buf[: api.WORKSPACE_ZEROED] == 0).all())


@pytest.mark.parametrize("hq,hk,tokens,dim,kv", [(8, 2, 1, 128, "bf16"), (6, 2, 3, 128, "bf16"), (4, 2, 1, 80, "bf16"), (8, 2, 1, 256, "e4m3"),
                                                 (8, 2, 4, 192, "e4m3"), (8, 2, 1, 128, "e4m3"), (12, 6, 4, 96, "e4m3"), (8, 8, 1, 64, "bf16"),
                                                 (6, 2, 2, 48, "e4m3"), (9, 3, 1, 64, "bf16"), (32, 4, 1, 64, "e4m3")])
def test_tables_with_room_for_much_more(hq, hk, tokens, dim, kv):
    """The same requests in rows of a table that could hold half a million tokens: a coarser cut of the work."""
    for page, window in ((16, 0), (4, 40), (32, 0), (64, 100)):
        s = scene(EDGES, hq, hk, dim, page, kv, tokens=tokens, seed=dim)
        wide = torch.full((len(EDGES), (1 << 19) // page), -1, dtype=torch.int32)
        wide[:, : s["table"].shape[1]] = s["table"]
        s["table"] = wide
        check(s, window=window)
    long = scene([5003, 17, 9000], hq, hk, dim, 32, kv, tokens=tokens, seed=1)
    wide = torch.full((3, 40000), -1, dtype=torch.int32)
    wide[:, : long["table"].shape[1]] = long["table"]
    long["table"] = wide
    check(long)


@pytest.mark.parametrize("page", [1, 2, 4, 512])
@pytest.mark.parametrize("dim", [32, 64])
def test_short_rows_in_small_and_large_pages(page, dim):
    """Rows of 64 bytes and less (e4m3), page by page of one token."""
    for kv in ("e4m3", "bf16"):
        check(scene([1, 70, 129, 5, 257], 6, 2, dim, page, kv, tokens=2, seed=page))


@pytest.mark.parametrize("hq,tokens,dim,kv", [(16, 9, 64, "bf16"), (16, 9, 128, "e4m3"), (24, 3, 256, "bf16"), (24, 2, 512, "bf16"), (33, 4, 512, "e4m3")])
def test_row_tiles_of_long_requests(hq, tokens, dim, kv):
    """More rows than a tile holds, over requests that several runs share."""
    check(scene([3000, 1, 777], hq, 1, dim, 16, kv, tokens=tokens, seed=dim))


def test_more_requests_than_a_warp_scans():
    """Beyond 256 requests the threads of a CTA share the prefix sum; some of the requests are long enough to be split."""
    lens = [(i * 7919) % 300 for i in range(290)]
    lens[5], lens[100], lens[289] = 6000, 4001, 5000
    check(scene(lens, 2, 1, 64, 16, seed=9))


def test_a_pool_whose_axes_lie_apart():
    """K and V in one allocation, pages padded, key heads a slice of more."""
    s = scene([100, 37], 4, 2, 64, 16, seed=19, fill=0.125)
    pages = s["k"].shape[0]
    big = torch.zeros(pages, 2, 16, 5, 96, dtype=torch.bfloat16, device="cuda")
    k, v = big[:, 0, :, 1:3, :64], big[:, 1, :, 1:3, :64]
    k.copy_(s["k"])
    v.copy_(s["v"])
    want, _, _ = attend(s)
    out = api.paged_attention(s["q"].cuda(), api.KVCache(k, v), s["table"].cuda(), s["lens"].cuda())
    assert torch.equal(out.cpu(), want)


def test_empty_batches_and_tables():
    cache = api.KVCache.empty(2, 16, 2, 64)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    out = api.paged_attention(torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), cache, none.view(0, 3), none)
    assert out.shape == (0, 4, 64)
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    lse = torch.empty(2, 4, device="cuda")
    out = api.paged_attention(q, cache, none.view(2, 0), torch.tensor([0, 0], dtype=torch.int32, device="cuda"), lse=lse)
    assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
