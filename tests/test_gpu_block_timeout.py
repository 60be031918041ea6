"""Bounded waits of attention over a cache with scales of blocks, made to run out by the test hook, as
test_gpu_paged_timeout has it: the call ends, the status says so, and the next call is as if it had not been."""
import pytest
import torch

from group_affine_bit_gb300 import api
from test_gpu_block_attention import cache_of, scene
from test_gpu_paged_timeout import LIMIT_CYCLES

pytestmark = pytest.mark.gpu

CASES = {
    "one request in many parts": dict(lens=[20011], hq=8, hk=1, dim=128, page=32),
    "many whole units, a scale for every token": dict(lens=[1 + (i * 37) % 90 for i in range(700)], hq=2, hk=1, dim=64, page=16, block=1),
    "whole units, parts and empty requests": dict(lens=[3000, 0, 17, 5000, 1], hq=8, hk=8, dim=256, page=16, kv="e4m3"),
    "two groups of consumers": dict(lens=[5000, 331], hq=16, hk=1, dim=128, page=16, tokens=4),
    "pairs of key heads": dict(lens=[5000, 17, 331], hq=8, hk=4, dim=128, page=32, room=1 << 19),
    "one q buffer": dict(lens=[3000, 777], hq=16, hk=1, dim=512, page=16),
}


@pytest.mark.parametrize("name", CASES)
def test_a_wait_runs_out_then_the_next_call_is_right(name):
    kw = dict(CASES[name])
    room = kw.pop("room", 0)
    s = scene(seed=21, **kw)
    if room:                                  # tables with room for many tiles
        wide = torch.full((len(kw["lens"]), room // kw["page"]), -1, dtype=torch.int32)
        wide[:, : s["table"].shape[1]] = s["table"]
        s["table"] = wide
    cache, q, table, lens = cache_of(s), s["q"].cuda(), s["table"].cuda(), s["lens"].cuda()
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device="cuda")
    want = api.paged_attention(q, cache, table, lens, lse=lse, workspace=api.Workspace())
    want_lse = lse.clone()
    ws, out = api.Workspace(), torch.full_like(q, 7.0)
    lse.fill_(7.0)
    api.test_fault_wait(LIMIT_CYCLES)
    try:
        api.paged_attention(q, cache, table, lens, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
    finally:
        api.test_fault_wait(0)
    assert api.STATUS_NAMES[api.workspace_status(ws.buf)] == "AFFQMM_E_TIMEOUT"
    assert int(ws.buf[: api.WORKSPACE_ZEROED].count_nonzero()) == 0
    assert bool((out == 7).all()) and bool((lse == 7).all())
    for _ in range(2):
        api.paged_attention(q, cache, table, lens, out=out, lse=lse, workspace=ws)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert api.workspace_status(ws.buf) == 0
