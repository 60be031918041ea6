"""The entry points of a cache with a scale for each block of tokens and head, and of reading a cache back, without a
GPU: refusals by name before anything is launched."""
import ctypes
import math

import pytest
import torch

import test_paged_host as plain
from group_affine_bit_gb300 import api, build


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


name = plain.name


def cache(type=2, page=16, heads=2, dim=128, pages=4, ps=4096, ts=256, hs=128, k=0x100000, v=0x200000, ks=None, vs=None, block=16, sps=2, sbs=1,
          shs=1, k_scales=0x1000, v_scales=0x2000):
    return api.CBlockCache(api.CCache(type, page, heads, dim, pages, ps, ts, hs, k, v, ks, vs), block, sps, sbs, shs, k_scales, v_scales)


class Blocks:
    """The library with the block cache's entry points in the places of the others, for the tests of those."""

    def __init__(self, lib):
        self.affqmm_rope_append, self.affqmm_paged_attention = lib.affqmm_block_append, lib.affqmm_block_attention


def read(f, c, batch=2, rows=8, k=0x300000, v=0x400000, ts=256, hs=128, table=0x500000, stride=8, wide=8, starts=0x600000, first=None, status=None):
    at = lambda p: ctypes.byref(api.CRows(p, ts, hs)) if p is not False else None  # noqa: E731
    return name(f(ctypes.byref(c) if c is not None else None, at(k), at(v), rows, batch, table, stride, wide, starts, first, status, None))


REFUSALS = [
    (dict(type=0), "AFFQMM_E_ARG"), (dict(type=3), "AFFQMM_E_ARG"), (dict(page=24), "AFFQMM_E_ARG"), (dict(ks=0x1000), "AFFQMM_E_ARG"),
    (dict(vs=0x1000), "AFFQMM_E_ARG"), (dict(type=1, ks=0x1000), "AFFQMM_E_ARG"), (dict(heads=0), "AFFQMM_E_SHAPE"), (dict(dim=72), "AFFQMM_E_SHAPE"),
    (dict(pages=0), "AFFQMM_E_SHAPE"), (dict(k=None), "AFFQMM_E_NULL"), (dict(k=0x100008), "AFFQMM_E_ALIGN"), (dict(hs=136), "AFFQMM_E_ALIGN"),
    (dict(block=0), "AFFQMM_E_ARG"), (dict(block=3), "AFFQMM_E_ARG"), (dict(block=32), "AFFQMM_E_ARG"), (dict(block=-16), "AFFQMM_E_ARG"),
    (dict(page=256, block=256, ps=65536), "AFFQMM_E_ARG"), (dict(sps=0), "AFFQMM_E_SHAPE"), (dict(sps=1), "AFFQMM_E_SHAPE"), (dict(shs=0), "AFFQMM_E_SHAPE"),
    (dict(shs=-1), "AFFQMM_E_SHAPE"), (dict(sps=1 << 31), "AFFQMM_E_SHAPE"), (dict(block=8, sbs=1), "AFFQMM_E_SHAPE"), (dict(block=8, sps=2, sbs=2), "AFFQMM_E_SHAPE"),
    (dict(k_scales=None), "AFFQMM_E_NULL"), (dict(v_scales=None), "AFFQMM_E_NULL"), (dict(v_scales=0x2002), "AFFQMM_E_ALIGN")]


@pytest.mark.parametrize("change,status", REFUSALS)
def test_caches_are_refused_by_name(L, change, status):
    c = cache(**change)
    assert plain.attend(Blocks(L), c) == status
    assert plain.append(Blocks(L), c) == status
    assert read(L.affqmm_block_read, c) == status


def test_scales_in_any_order_that_does_not_overlap(L):
    """Accepted as far as the device or the workspace."""
    for kw in (dict(), dict(block=8, sps=4, sbs=2), dict(block=8, sps=4, sbs=1, shs=2), dict(block=8, sps=1, sbs=4, shs=8), dict(sbs=-7),
               dict(heads=1, shs=0, sps=1), dict(pages=1, sps=-3)):
        assert plain.attend(Blocks(L), cache(**kw), hq=8) in ("AFFQMM_E_WORKSPACE", "AFFQMM_E_DEVICE", "AFFQMM_E_CUDA"), kw


def test_attention_refusals(L):
    B = Blocks(L)
    assert plain.attend(B, None) == "AFFQMM_E_NULL"
    for kw, status in [(dict(tokens=0), "AFFQMM_E_ARG"), (dict(tokens=65), "AFFQMM_E_ARG"), (dict(hq=7), "AFFQMM_E_SHAPE"), (dict(batch=-1), "AFFQMM_E_SHAPE"),
                       (dict(batch=16385), "AFFQMM_E_SHAPE"), (dict(wide=1 << 27), "AFFQMM_E_SHAPE"), (dict(scale=math.nan), "AFFQMM_E_ARG"),
                       (dict(window=-1), "AFFQMM_E_ARG"), (dict(lens=None), "AFFQMM_E_NULL"), (dict(table=None), "AFFQMM_E_NULL"),
                       (dict(q=0x300008), "AFFQMM_E_ALIGN"), (dict(lse=0x800002), "AFFQMM_E_ALIGN")]:
        assert plain.attend(B, cache(), **kw) == status, kw
    assert plain.attend(B, cache(), batch=0) == "AFFQMM_OK"
    n = ctypes.c_size_t(0)
    size = L.affqmm_block_attention_workspace_bytes
    assert name(size(None, 1, 8, ctypes.byref(n))) == "AFFQMM_E_NULL" and name(size(ctypes.byref(cache()), 1, 8, None)) == "AFFQMM_E_NULL"
    assert name(size(ctypes.byref(cache()), 1, 9, ctypes.byref(n))) == "AFFQMM_E_SHAPE"
    assert name(size(ctypes.byref(cache(block=5)), 1, 8, ctypes.byref(n))) == "AFFQMM_E_ARG"


def test_append_refusals(L):
    B, R = Blocks(L), api.CRope
    assert plain.append(B, None) == "AFFQMM_E_NULL"
    for kw, status in [(dict(rope=R(0x700000, None, 130, 0, 1)), "AFFQMM_E_SHAPE"), (dict(rope=R(0x700000, None, 64, 2, 1)), "AFFQMM_E_ARG"),
                       (dict(rope=R(None, None, 64, 0, 1)), "AFFQMM_E_NULL"), (dict(tokens=-1), "AFFQMM_E_SHAPE"), (dict(slots=None), "AFFQMM_E_NULL"),
                       (dict(v=0x320004), "AFFQMM_E_ALIGN"), (dict(out=0x300000, os=2048), "AFFQMM_E_ARG")]:
        assert plain.append(B, cache(), **kw) == status, kw
    assert plain.append(B, cache(), tokens=0) == "AFFQMM_OK"


def test_read_refusals(L):
    for f, c in ((L.affqmm_block_read, cache()), (L.affqmm_paged_read, plain.cache())):
        assert read(f, None) == "AFFQMM_E_NULL"
        for kw, status in [(dict(batch=-1), "AFFQMM_E_SHAPE"), (dict(batch=16385), "AFFQMM_E_SHAPE"), (dict(rows=-1), "AFFQMM_E_SHAPE"),
                           (dict(rows=1 << 30), "AFFQMM_E_SHAPE"), (dict(wide=-1), "AFFQMM_E_SHAPE"), (dict(wide=1 << 27), "AFFQMM_E_SHAPE"),
                           (dict(wide=1 << 62), "AFFQMM_E_SHAPE"), (dict(stride=-1), "AFFQMM_E_SHAPE"), (dict(starts=None), "AFFQMM_E_NULL"),
                           (dict(table=None), "AFFQMM_E_NULL"), (dict(k=None), "AFFQMM_E_NULL"), (dict(v=False), "AFFQMM_E_NULL"),
                           (dict(k=0x300008), "AFFQMM_E_ALIGN"), (dict(ts=260), "AFFQMM_E_ALIGN"), (dict(hs=-8), "AFFQMM_E_SHAPE"),
                           (dict(starts=0x600002), "AFFQMM_E_ALIGN"), (dict(first=0x600001), "AFFQMM_E_ALIGN"), (dict(status=0x600003), "AFFQMM_E_ALIGN")]:
            assert read(f, c, **kw) == status, kw
        assert read(f, c, batch=0) == read(f, c, rows=0) == "AFFQMM_OK"
    for change, status in plain.CACHE_REFUSALS:
        assert read(L.affqmm_paged_read, plain.cache(**change)) == status


def test_the_binding_refuses_host_tensors_and_odd_blocks():
    k = torch.zeros(2, 16, 2, 32, dtype=torch.int8)
    s = torch.ones(2, 2, 2)
    with pytest.raises(ValueError):
        api.BlockCache(k, k.clone(), s, s)
    with pytest.raises(ValueError):
        api.BlockCache.empty(2, 16, 2, 32, block=3, device="cpu")
    with pytest.raises(ValueError):
        api.KVCache(k, k.clone())


def test_the_binding_hands_over_the_headers_structure():
    """Offsets of affqmm_block_cache on a 64-bit machine."""
    want = [("kv", 0), ("block", 80), ("s_page_stride", 88), ("s_block_stride", 96), ("s_head_stride", 104), ("k_scales", 112), ("v_scales", 120)]
    assert [(n, getattr(api.CBlockCache, n).offset) for n, _ in want] == want and ctypes.sizeof(api.CBlockCache) == 128
