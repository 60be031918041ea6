"""Rotary positions with the append to the paged cache, against a 64-bit form.

Tolerance, per value x of a pair (a, b): one rounding to bf16, 2^-9 of the value
(doubled for a binade's edge), and fp32 arithmetic: the phase in 2^-25 of a turn
and the sines and products in a few 2^-24, together under 2^-20 (|a| + |b|).  In
an e4m3 cache the rounding is 2^-4 of the value or half a subnormal step, 2^-10."""
import numpy as np
import pytest
import torch

import paged_ref
from group_affine_bit_gb300 import api

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def case(T, hq, hk, dim, rotary, axes, neighbour, page, kv, seed, layout="token", high=300000):
    g = gen(seed)
    qkv = torch.randn(T, (hq + 2 * hk) * dim, generator=g).bfloat16()
    pos = torch.randint(-5, high, (axes, T), generator=g, dtype=torch.int32)
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    freqs = paged_ref.turns_of(rotary) if rotary else []
    axis = torch.tensor([i % axes for i in range(rotary // 2)], dtype=torch.uint8)
    shape = (pages, page, hk, dim) if layout == "token" else (pages, hk, page, dim)
    dt = torch.bfloat16 if kv == "bf16" else torch.float8_e4m3fn
    raw = [torch.randn(shape, generator=g).to(dt) for _ in "kv"]
    if layout == "head":
        raw = [r.transpose(1, 2) for r in raw]
    scales = [torch.rand(hk, generator=g) * 0.1 + 0.01 for _ in "kv"] if kv == "e4m3" else [None, None]
    return qkv, pos, slots, freqs, axis, raw, scales


def parts(qkv, hq, hk, dim):
    T = qkv.shape[0]
    return (qkv[:, : hq * dim].view(T, hq, dim), qkv[:, hq * dim: (hq + hk) * dim].view(T, hk, dim),
            qkv[:, (hq + hk) * dim:].view(T, hk, dim))


def keep_layout(t, layout):
    return t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if layout == "head" else t.cuda()


def spread(x, rotary, neighbour):
    """|a| + |b| of each value's pair."""
    y = torch.zeros_like(x)
    R = rotary
    a = x.abs()
    if neighbour:
        s = a[..., 0:R:2] + a[..., 1:R:2]
        y[..., 0:R:2] = s
        y[..., 1:R:2] = s
    else:
        s = a[..., : R // 2] + a[..., R // 2: R]
        y[..., : R // 2] = s
        y[..., R // 2: R] = s
    return y


def run_and_check(T, hq, hk, dim, rotary, axes, neighbour, page, kv, seed=0, layout="token", in_place=False, padded=False, high=300000):
    qkv, pos, slots, freqs, axis, raw, scales = case(T, hq, hk, dim, rotary, axes, neighbour, page, kv, seed, layout, high)
    if padded:
        slots[:: 3] = -1
    dev = qkv.cuda()
    q, k, v = parts(dev, hq, hk, dim)
    kc, vc = (keep_layout(r, layout) for r in raw)
    cache = api.KVCache(kc, vc, *(s.cuda() if s is not None else None for s in scales))
    rope = api.Rope(api.rope_turns(freqs), axis.cuda() if axes > 1 else None, neighbour=neighbour)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    positions = pos.cuda() if axes > 1 else pos[0].cuda()
    got = api.rope_append(q, k, v, positions, slots.cuda(), rope, cache, out=q if in_place else None, status=status)
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    hq_, hk_, hv_ = (x.double() for x in parts(qkv, hq, hk, dim))
    want_q, want_k = (paged_ref.rope(x, pos, freqs, axis, neighbour) for x in (hq_, hk_))
    err = (got.cpu().double() - want_q).abs()
    assert bool((err <= 2.0 ** -8 * want_q.abs() + 2.0 ** -20 * spread(hq_, rotary, neighbour)).all())
    for stored, before, want, src, scale in ((kc, raw[0], want_k, hk_, scales[0]), (vc, raw[1], hv_, None, scales[1])):
        stored = stored.cpu()
        flat = stored.reshape(-1, hk, dim)
        old = before.reshape(-1, hk, dim)
        keep = slots >= 0
        s = 1.0 if scale is None else scale.double()[None, :, None]
        w = want / s
        room = 0 if src is None else 2.0 ** -20 * spread(src, rotary, neighbour) / s
        e = (flat.double()[slots[keep].long()] - (w[keep].clamp(-448, 448) if kv == "e4m3" else w[keep])).abs()
        # a value within `room` of a rounding boundary may fall on its other side: one more step
        tol = (2.0 ** -4 * w.abs() + 2.0 ** -10 if kv == "e4m3" else 2.0 ** -8 * w.abs()) + room
        assert bool((e <= tol[keep]).all())
        if src is None and kv == "bf16":
            assert torch.equal(flat[slots[keep].long()], parts(qkv, hq, hk, dim)[2][keep])   # v as it is
        others = torch.ones(flat.shape[0], dtype=torch.bool)
        others[slots[keep].long()] = False
        bits = torch.int16 if kv == "bf16" else torch.uint8
        assert torch.equal(flat.contiguous().view(bits)[others], old.contiguous().view(bits)[others])   # other slots untouched
    if in_place:   # the rest of the projection's rows is as it was
        assert torch.equal(dev[:, hq * dim:].cpu(), qkv[:, hq * dim:])


@pytest.mark.parametrize("T,hq,hk,dim,rotary,axes,neighbour,page,kv", [
    (1, 32, 8, 256, 256, 1, False, 16, "bf16"), (1, 1, 1, 16, 16, 1, True, 1, "bf16"), (4, 32, 8, 256, 256, 1, False, 16, "bf16"),
    (37, 32, 8, 128, 128, 3, False, 64, "bf16"), (129, 28, 4, 80, 40, 2, True, 8, "e4m3"), (65, 6, 2, 80, 80, 2, False, 16, "e4m3"),
    (17, 16, 16, 64, 32, 1, False, 32, "bf16"), (33, 5, 1, 512, 512, 4, False, 128, "e4m3"), (9, 3, 3, 48, 20, 1, False, 2, "bf16"),
    (9, 3, 3, 48, 20, 2, True, 2, "e4m3"), (12, 4, 2, 96, 0, 1, False, 16, "bf16"), (700, 8, 2, 64, 64, 1, True, 16, "bf16"),
    (5, 2, 2, 48, 2, 1, False, 4, "bf16"), (300, 7, 1, 112, 56, 3, True, 32, "bf16")])
def test_against_64_bits(T, hq, hk, dim, rotary, axes, neighbour, page, kv):
    run_and_check(T, hq, hk, dim, rotary, axes, neighbour, page, kv, seed=T)


@pytest.mark.parametrize("rotary,neighbour", [(128, False), (128, True), (20, False), (20, True)])
def test_in_place_head_major_and_padded(rotary, neighbour):
    run_and_check(40, 8, 2, 128, rotary, 2, neighbour, 16, "bf16", seed=3, layout="head", in_place=True, padded=True)
    run_and_check(40, 8, 2, 128, rotary, 2, neighbour, 16, "e4m3", seed=4, layout="head", in_place=True, padded=True)


def test_positions_up_to_the_last_integer():
    """The phase is exact at any position: no tolerance grows with it."""
    run_and_check(64, 4, 2, 128, 128, 1, False, 16, "bf16", seed=5, high=2 ** 31 - 1)


def test_an_axis_beyond_the_positions_is_the_last():
    """A rope of three axes with the positions of text, and with two axes."""
    g = gen(7)
    q = torch.randn(9, 4, 64, generator=g).bfloat16().cuda()
    k, v = (torch.randn(9, 2, 64, generator=g).bfloat16().cuda() for _ in "kv")
    pos = torch.randint(0, 5000, (2, 9), generator=g, dtype=torch.int32).cuda()
    slots, turns = torch.arange(9, dtype=torch.int32, device="cuda"), api.rope_turns(paged_ref.turns_of(64))
    axis = torch.tensor([i % 3 for i in range(32)], dtype=torch.uint8, device="cuda")
    for positions, same in ((pos[0], None), (pos[:1], None), (pos, axis.clamp(max=1))):
        got, want = (api.KVCache.empty(1, 16, 2, 64) for _ in "ab")
        for c in (got, want):
            c.k.zero_(), c.v.zero_()
        a = api.rope_append(q, k, v, positions, slots, api.Rope(turns, axis), got)
        b = api.rope_append(q, k, v, positions, slots, api.Rope(turns, same), want)
        assert torch.equal(a, b) and torch.equal(got.k, want.k) and torch.equal(got.v, want.v)


def test_a_frequency_of_zero_turns_nothing():
    g = gen(6)
    q = torch.randn(7, 4, 64, generator=g).bfloat16().cuda()
    k, v = (torch.randn(7, 2, 64, generator=g).bfloat16().cuda() for _ in "kv")
    cache = api.KVCache.empty(2, 16, 2, 64)
    out = api.rope_append(q, k, v, torch.arange(7, dtype=torch.int32, device="cuda") * 999983,
                          torch.arange(7, dtype=torch.int32, device="cuda"), api.Rope(api.rope_turns([0.0] * 32)), cache)
    assert torch.equal(out, q) and torch.equal(cache.k.reshape(-1, 2, 64)[:7], k)


def test_slots_outside_the_pool():
    q = torch.ones(6, 2, 32, dtype=torch.bfloat16, device="cuda")
    k = torch.full((6, 1, 32), 3.0, dtype=torch.bfloat16, device="cuda")
    rope = api.Rope(api.rope_turns([1.0] * 16))
    pos = torch.zeros(6, dtype=torch.int32, device="cuda")
    guard = torch.zeros(5, 4, 1, 32, dtype=torch.bfloat16, device="cuda")
    for slots, flag in (([0, 5, -1, 11, -1, 3], 0), ([0, 12, 1, 2, 3, 4], 2), ([-2, 0, 1, 2, 3, 4], 2),
                        ([2 ** 31 - 1, 0, 1, 2, 3, 4], 2), ([-2 ** 31, 0, 1, 2, 3, 4], 2)):
        guard.zero_()
        cache = api.KVCache(guard[1:4], guard[1:4].clone())
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = api.rope_append(q, k, k, pos, torch.tensor(slots, dtype=torch.int32, device="cuda"), rope, cache, status=status)
        assert int(status[0]) == flag and bool((out == 1).all())
        flat = guard.reshape(-1, 32)
        written = sorted(set((flat != 0).any(1).nonzero()[:, 0].tolist()))
        assert written == sorted(4 + s for s in slots if 0 <= s < 12)


def test_infinities_and_saturation():
    """e4m3: beyond +-448 saturates, an infinity too; a NaN stays one."""
    cache = api.KVCache.empty(1, 16, 1, 16, dtype=torch.float8_e4m3fn, v_scale=torch.tensor([0.5], device="cuda"))
    v = torch.tensor([1.0, -2.0, 448.0, 500.0, -1e30, float("inf"), float("-inf"), float("nan")] * 2).bfloat16().reshape(1, 1, 16).cuda()
    zero = torch.zeros_like(v)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.rope_append(zero, zero, v, one, one, api.Rope(api.rope_turns([1.0])), cache)
    got = cache.v[0, 0, 0].float().cpu()
    want = torch.tensor([2.0, -4.0, 448.0, 448.0, -448.0, 448.0, -448.0, float("nan")] * 2)
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(7), want.nan_to_num(7))


def test_no_tokens():
    cache = api.KVCache.empty(1, 16, 2, 32)
    e = lambda h: torch.empty(0, h, 32, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    assert api.rope_append(e(4), e(2), e(2), i, i, api.Rope(api.rope_turns([1.0] * 16)), cache).shape == (0, 4, 32)
