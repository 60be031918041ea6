"""The paged cache's entry points without a GPU: refusals by name before
anything is launched, the binding's own checks, and rope_turns."""
import ctypes
import math

import pytest
import torch

import paged_ref
from group_affine_bit_gb300 import api, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def cache(type=0, page=16, heads=2, dim=128, pages=4, ps=4096, ts=256, hs=128, k=0x100000, v=0x200000, ks=None, vs=None):
    return api.CCache(type, page, heads, dim, pages, ps, ts, hs, k, v, ks, vs)


def name(rc):
    return api.STATUS_NAMES[rc]


CACHE_REFUSALS = [
    (dict(type=2), "AFFQMM_E_ARG"), (dict(page=0), "AFFQMM_E_ARG"), (dict(page=24), "AFFQMM_E_ARG"), (dict(page=1 << 17), "AFFQMM_E_ARG"),
    (dict(ks=0x1000), "AFFQMM_E_ARG"), (dict(heads=0), "AFFQMM_E_SHAPE"), (dict(dim=0), "AFFQMM_E_SHAPE"), (dict(dim=72), "AFFQMM_E_SHAPE"),
    (dict(dim=528), "AFFQMM_E_SHAPE"), (dict(pages=-1), "AFFQMM_E_SHAPE"), (dict(pages=1 << 27), "AFFQMM_E_SHAPE"), (dict(ps=-8), "AFFQMM_E_SHAPE"),
    (dict(k=None), "AFFQMM_E_NULL"), (dict(v=None), "AFFQMM_E_NULL"), (dict(k=0x100008), "AFFQMM_E_ALIGN"), (dict(ts=252), "AFFQMM_E_ALIGN"),
    (dict(type=1, hs=136), "AFFQMM_E_ALIGN"), (dict(ps=4104), "AFFQMM_E_ALIGN"), (dict(hs=384), "AFFQMM_E_ALIGN"), (dict(ts=64), "AFFQMM_E_SHAPE"), (dict(type=1, vs=0x1002), "AFFQMM_E_ALIGN")]


def attend(L, c, batch=1, tokens=1, hq=8, q=0x300000, out=0x400000, qs=1024, table=0x500000, stride=8, wide=8, lens=0x600000,
           scale=1.0, window=0, lse=None, status=None, ws=None, nbytes=0):
    lanes = lambda p, s: ctypes.byref(api.CLanes(p, s, 0, 128))  # noqa: E731
    return name(L.affqmm_paged_attention(ctypes.byref(c) if c is not None else None, lanes(q, qs), lanes(out, qs), lse, batch, tokens, hq,
                                         table, stride, wide, lens, scale, window, status, ws, nbytes, None))


def append(L, c, rope=None, tokens=1, hq=8, q=0x300000, k=0x310000, v=0x320000, out=0x400000, qs=1024, os=1024, pos=0x500000, ps=0,
           slots=0x600000, status=None):
    rope = api.CRope(0x700000, None, 128, 0, 1) if rope is None else rope
    rows = lambda p, s: ctypes.byref(api.CRows(p, s, 128))  # noqa: E731
    return name(L.affqmm_rope_append(ctypes.byref(c) if c is not None else None, ctypes.byref(rope), rows(q, qs), rows(k, 256), rows(v, 256),
                                     rows(out, os), tokens, hq, pos, ps, slots, status, None))


@pytest.mark.parametrize("change,status", CACHE_REFUSALS)
def test_caches_are_refused_by_name(L, change, status):
    assert attend(L, cache(**change)) == status
    assert append(L, cache(**change)) == status


def test_attention_refusals(L):
    assert attend(L, None) == "AFFQMM_E_NULL"
    for kw, status in [(dict(tokens=0), "AFFQMM_E_ARG"), (dict(tokens=65), "AFFQMM_E_ARG"), (dict(hq=7), "AFFQMM_E_SHAPE"), (dict(hq=0), "AFFQMM_E_SHAPE"),
                       (dict(batch=-1), "AFFQMM_E_SHAPE"), (dict(batch=16385), "AFFQMM_E_SHAPE"), (dict(wide=-1), "AFFQMM_E_SHAPE"),
                       (dict(wide=1 << 27), "AFFQMM_E_SHAPE"), (dict(scale=math.nan), "AFFQMM_E_ARG"), (dict(scale=math.inf), "AFFQMM_E_ARG"),
                       (dict(window=-1), "AFFQMM_E_ARG"), (dict(lens=None), "AFFQMM_E_NULL"), (dict(table=None), "AFFQMM_E_NULL"),
                       (dict(q=None), "AFFQMM_E_NULL"), (dict(out=None), "AFFQMM_E_NULL"), (dict(q=0x300008), "AFFQMM_E_ALIGN"),
                       (dict(qs=1028), "AFFQMM_E_ALIGN"), (dict(qs=-8), "AFFQMM_E_SHAPE"), (dict(lse=0x800002), "AFFQMM_E_ALIGN"),
                       (dict(lens=0x600002), "AFFQMM_E_ALIGN")]:
        assert attend(L, cache(), **kw) == status, kw
    assert attend(L, cache(), batch=0) == "AFFQMM_OK"
    n = ctypes.c_size_t(0)
    assert name(L.affqmm_paged_attention_workspace_bytes(None, 1, 8, ctypes.byref(n))) == "AFFQMM_E_NULL"
    assert name(L.affqmm_paged_attention_workspace_bytes(ctypes.byref(cache()), 1, 8, None)) == "AFFQMM_E_NULL"
    assert name(L.affqmm_paged_attention_workspace_bytes(ctypes.byref(cache()), 1, 9, ctypes.byref(n))) == "AFFQMM_E_SHAPE"


def test_the_most_tiles_of_a_call(L):
    """Below the documented bound a call gets as far as the device or the workspace; at it, it is refused."""
    def edge(batch, c, **kw):
        return attend(L, c, batch=batch, **kw) == "AFFQMM_E_SHAPE"

    c = cache(pages=1 << 26)                             # 2 key heads x (2^30 / 128 + 2) tiles
    big = dict(wide=1 << 26, stride=0)
    assert not edge(127, c, **big) and edge(128, c, **big)
    wide = cache(pages=1 << 16, heads=8, dim=512, ps=65536, ts=4096, hs=512)
    rows = dict(wide=1 << 16, stride=0, hq=64, tokens=64)    # 8 x 32 row tiles x (2^20 / 64 + 2)
    assert not edge(511, wide, **rows) and edge(512, wide, **rows)
    rows["window"] = 64                                  # 128 keys that a window sees: two tiles and two more
    assert not edge(16384, wide, **rows)


def test_append_refusals(L):
    assert append(L, None) == "AFFQMM_E_NULL"
    R = api.CRope
    for kw, status in [(dict(rope=R(0x700000, None, 130, 0, 1)), "AFFQMM_E_SHAPE"), (dict(rope=R(0x700000, None, 3, 0, 1)), "AFFQMM_E_SHAPE"),
                       (dict(rope=R(0x700000, None, 64, 2, 1)), "AFFQMM_E_ARG"), (dict(rope=R(0x700000, None, 64, 0, 0)), "AFFQMM_E_ARG"),
                       (dict(rope=R(None, None, 64, 0, 1)), "AFFQMM_E_NULL"), (dict(rope=R(0x700004, None, 64, 0, 1)), "AFFQMM_E_ALIGN"),
                       (dict(tokens=-1), "AFFQMM_E_SHAPE"), (dict(hq=0), "AFFQMM_E_SHAPE"), (dict(pos=None), "AFFQMM_E_NULL"),
                       (dict(slots=None), "AFFQMM_E_NULL"), (dict(q=None), "AFFQMM_E_NULL"), (dict(v=0x320004), "AFFQMM_E_ALIGN"),
                       (dict(out=0x300000, os=2048), "AFFQMM_E_ARG"), (dict(ps=-1), "AFFQMM_E_SHAPE")]:
        assert append(L, cache(), **kw) == status, kw
    assert append(L, cache(), tokens=0) == "AFFQMM_OK"


def test_plan_refusals(L):
    def plan(batch=2, lens=0x1000, fresh=0x2000, table=0x3000, stride=8, wide=8, ring=0x4000, pool=16, state=0x5000, page=16, capacity=8,
             starts=0x6000, lens_out=0x7000, state_out=0x8000, slots=0x9000, positions=0xA000, requests=0xB000, status=0xC000, step=True):
        s = api.CStep(capacity, starts, lens_out, state_out, slots, positions, requests, status)
        return name(L.affqmm_paged_plan(batch, lens, fresh, None, table, stride, wide, ring, pool, state, page, ctypes.byref(s) if step else None, None))

    for kw, status in [(dict(step=False), "AFFQMM_E_NULL"), (dict(batch=-1), "AFFQMM_E_SHAPE"), (dict(batch=16385), "AFFQMM_E_SHAPE"),
                       (dict(wide=-1), "AFFQMM_E_SHAPE"), (dict(stride=7), "AFFQMM_E_SHAPE"), (dict(pool=-1), "AFFQMM_E_SHAPE"),
                       (dict(pool=1 << 28), "AFFQMM_E_SHAPE"), (dict(wide=1 << 28, stride=1 << 28), "AFFQMM_E_SHAPE"), (dict(page=12), "AFFQMM_E_ARG"),
                       (dict(capacity=-1), "AFFQMM_E_ARG"), (dict(lens=None), "AFFQMM_E_NULL"), (dict(table=None), "AFFQMM_E_NULL"),
                       (dict(ring=None), "AFFQMM_E_NULL"), (dict(state=None), "AFFQMM_E_NULL"), (dict(slots=None), "AFFQMM_E_NULL"),
                       (dict(status=None), "AFFQMM_E_NULL"), (dict(slots=0x9004), "AFFQMM_E_ALIGN"), (dict(lens=0x1002), "AFFQMM_E_ALIGN"),
                       (dict(lens_out=0x1000), "AFFQMM_E_ARG"), (dict(state_out=0x5000), "AFFQMM_E_ARG")]:
        assert plan(**kw) == status, kw


def test_the_binding_refuses_host_tensors():
    k = torch.zeros(2, 16, 2, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.KVCache(k, k.clone())
    with pytest.raises(ValueError):
        api.Rope(torch.zeros(4, dtype=torch.int64))
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.PagedStep(i, i, i, i, i, i, i)


def test_a_status_word_must_be_on_the_calls_device():
    assert api._status_ptr(None, 0) is None
    for t in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64), torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(ValueError):
            api._status_ptr(t, 0)


def test_rope_turns_are_the_frequencies_fractions():
    f = paged_ref.turns_of(64) + [0.0, 2 * math.pi, 7.5]
    got = [x % (1 << 64) for x in api.rope_turns(f, "cpu").tolist()]
    for x, g in zip(f, got):
        t = x / (2 * math.pi)
        assert abs(g / 2.0 ** 64 - (t - math.floor(t))) <= 2.0 ** -52
