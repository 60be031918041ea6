"""Block tables and slot maps built on the GPU, against a request-by-request
allocator: every value equal."""
import numpy as np
import pytest
import torch

import paged_ref
from group_affine_bit_gb300 import api

pytestmark = pytest.mark.gpu


def cuda(a, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=dtype, device="cuda")


def scene(rng, batch, page, wide, spare, most, done=0.1, pool=None, head=None):
    lens = rng.integers(0, wide * page + 1 - min(most, wide * page), batch)
    fresh = rng.integers(0, most + 1, batch)
    finished = rng.random(batch) < done
    used = -(-lens // page)
    total = int(used.sum())
    pool = total + spare if pool is None else pool
    order = rng.permutation(max(pool, total)).astype(np.int32)
    table = np.full((batch, wide), -1, np.int32)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = order[at: at + u]
        at += u
    left = order[total:]
    ring = np.full(pool, -7, np.int32)
    head = int(rng.integers(0, pool)) if head is None else head
    ring[(head + np.arange(left.size)) % pool] = left
    return dict(lens=lens.astype(np.int32), fresh=fresh.astype(np.int32), finished=finished, table=table, ring=ring,
                ring_state=np.array([head, left.size], np.int32))


def check(sc, page, capacity, stream=None):
    want = paged_ref.plan(sc["lens"], sc["fresh"], sc["finished"], sc["table"], sc["ring"], sc["ring_state"], page, capacity)
    table, ring = cuda(sc["table"]), cuda(sc["ring"])
    step = api.PagedStep.empty(sc["lens"].size, capacity)
    args = (cuda(sc["lens"]), cuda(sc["fresh"]), cuda(sc["finished"], torch.bool), table, ring, cuda(sc["ring_state"]), page)
    for _ in range(2):          # the same call on the same inputs writes the same values
        api.paged_plan(*args, out=step)
        torch.cuda.synchronize()
        got = dict(starts=step.starts, lens=step.lens, slots=step.slots, positions=step.positions, requests=step.requests,
                   ring_state=step.ring_state, status=step.status, table=table, ring=ring)
        for name, t in got.items():
            assert np.array_equal(t.cpu().numpy(), want[name]), name
    return want


@pytest.mark.parametrize("batch,page,wide,most,capacity", [
    (1, 16, 8, 1, 1), (1, 1, 40, 5, 7), (2, 64, 3, 64, 200), (33, 16, 20, 1, 33), (64, 16, 20, 40, 3001),
    (257, 8, 30, 3, 1024), (1024, 32, 12, 20, 20000), (1025, 16, 12, 9, 9001), (5000, 16, 6, 2, 12003), (16384, 16, 3, 1, 16384)])
def test_steps(batch, page, wide, most, capacity):
    rng = np.random.default_rng(batch * 7 + page)
    want = check(scene(rng, batch, page, wide, spare=batch * (most // page + 1) + 3, most=most), page, capacity)
    assert want["status"][0] & ~4 == 0


@pytest.mark.parametrize("spare", [0, 1, 5, 20])
def test_a_pool_that_runs_out(spare):
    rng = np.random.default_rng(spare)
    want = check(scene(rng, 70, 8, 16, spare, most=16, done=0.0), 8, 2000)
    assert want["status"][0] & 1


def test_tokens_beyond_the_capacity():
    rng = np.random.default_rng(3)
    sc = scene(rng, 50, 16, 10, 200, most=16)
    for capacity in (0, 1, 2, 63, 64, 65, 200):
        want = check(sc, 16, capacity)
        assert want["status"][0] & 4


def test_a_request_that_outgrows_its_row():
    rng = np.random.default_rng(4)
    sc = scene(rng, 20, 16, 4, 60, most=8, done=0.0)
    sc["lens"][5], sc["fresh"][5] = 64, 1
    sc["table"][5] = np.arange(4)
    assert check(sc, 16, 500)["status"][0] == 2


def test_counts_that_cannot_be():
    rng = np.random.default_rng(5)
    sc = scene(rng, 20, 16, 4, 60, most=8, done=0.0)
    sc["lens"][2], sc["fresh"][3], sc["lens"][4] = -5, -1, 65
    sc["finished"][4] = True
    assert check(sc, 16, 500)["status"][0] == 8
    for bad in ([-1, 3], [0, 10 ** 6], [10 ** 6, 2]):
        sc["ring_state"] = np.array(bad, np.int32)
        assert check(sc, 16, 500)["status"][0] & 8
    # huge numbers of new tokens saturate instead of wrapping around
    sc = scene(rng, 6, 16, 4, 60, most=8, done=0.0)
    sc["fresh"][:] = 2 ** 31 - 1
    step = api.PagedStep.empty(6, 100)
    api.paged_plan(cuda(sc["lens"]), cuda(sc["fresh"]), None, cuda(sc["table"]), cuda(sc["ring"]), cuda(sc["ring_state"]), 16, out=step)
    assert int(step.status[0]) == 6 and bool((step.slots == -1).all()) and np.array_equal(step.lens.cpu().numpy(), sc["lens"])


@pytest.mark.parametrize("capacity", [2 ** 30, 2 ** 30 - 1])
def test_sums_beyond_the_largest_capacity(capacity):
    """More tokens than 2^30 in a step that could hold 2^30: the request that lies beyond is not served."""
    page, wide = 1 << 16, 1 << 14
    pool = wide + 7
    table = torch.full((3, wide), -1, dtype=torch.int32, device="cuda")
    ring = torch.arange(pool, dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    fresh = torch.tensor([capacity - 3, 10, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    step = api.PagedStep.empty(3, capacity)
    api.paged_plan(lens, fresh, None, table, ring, torch.tensor([5, pool], dtype=torch.int32, device="cuda"), page, out=step)
    assert int(step.status[0]) == 4 + 2 and step.lens.tolist() == [capacity - 3, 0, 0]
    assert step.starts[:3].tolist() == [0, capacity - 3, capacity + 7]
    assert step.ring_state.tolist() == [(5 + wide) % pool, 7]
    assert step.slots[-5:].tolist() == [(4 + wide) % pool * page + page - 5 - (2 ** 30 - capacity), (4 + wide) % pool * page + page - 4 - (2 ** 30 - capacity), -1, -1, -1]
    assert step.positions[-4:].tolist() == [capacity - 4, 0, 1, 2] and step.requests[-4:].tolist() == [0, 1, 1, 1]


def test_more_pages_back_than_the_ring_holds():
    rng = np.random.default_rng(6)
    sc = scene(rng, 10, 16, 4, 4, most=4)
    sc["finished"][:] = True
    sc["ring_state"][1] = sc["ring"].size
    assert check(sc, 16, 100)["status"][0] == 8


def test_no_requests():
    step = api.PagedStep.empty(0, 10)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    ring = torch.arange(5, dtype=torch.int32, device="cuda")
    api.paged_plan(none, none, None, torch.empty(0, 4, dtype=torch.int32, device="cuda"), ring,
                   torch.tensor([1, 4], dtype=torch.int32, device="cuda"), 16, out=step)
    assert step.starts.tolist() == [0] and step.slots.tolist() == [-1] * 10 and step.ring_state.tolist() == [1, 4]


def test_a_strided_table_and_another_stream():
    rng = np.random.default_rng(8)
    sc = scene(rng, 40, 16, 6, 100, most=20)
    want = paged_ref.plan(*(sc[k] for k in ("lens", "fresh", "finished", "table", "ring", "ring_state")), 16, 900)
    wide = torch.full((40, 11), -3, dtype=torch.int32, device="cuda")
    table = wide[:, 2:8]
    table.copy_(cuda(sc["table"]))
    ring = cuda(sc["ring"])
    step = api.PagedStep.empty(40, 900)
    args = (cuda(sc["lens"]), cuda(sc["fresh"]), cuda(sc["finished"], torch.bool), table, ring, cuda(sc["ring_state"]), 16)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    api.paged_plan(*args, out=step, stream=st)
    st.synchronize()
    assert np.array_equal(table.cpu().numpy(), want["table"]) and np.array_equal(step.slots.cpu().numpy(), want["slots"])
    assert bool((wide[:, :2] == -3).all()) and bool((wide[:, 8:] == -3).all())


@pytest.mark.parametrize("pool", [300, 100])
def test_pages_are_never_held_twice(pool):
    """Sixty steps of requests that come, grow and finish: every page of the pool
    is free or held by one request, and what the slots say is what the tables say."""
    rng = np.random.default_rng(9)
    batch, page, wide, capacity = 48, 8, 12, 400
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    table = torch.full((batch, wide), -1, dtype=torch.int32, device="cuda")
    ring = cuda(rng.permutation(pool).astype(np.int32))
    state = torch.tensor([0, pool], dtype=torch.int32, device="cuda")
    steps = [api.PagedStep.empty(batch, capacity) for _ in range(2)]
    ran_out = 0
    for i in range(60):
        n = lens.cpu().numpy()
        finished = (n > 0) & (rng.random(batch) < 0.15)
        fresh = np.where(rng.random(batch) < 0.2, rng.integers(0, 40, batch), 1)
        fresh = np.where(n + fresh > wide * page, 0, fresh)
        step = api.paged_plan(lens, cuda(fresh.astype(np.int32)), cuda(finished, torch.bool), table, ring, state, page, out=steps[i % 2])
        lens, state = step.lens, step.ring_state
        ran_out |= int(step.status[0])
        held = [int(x) for r, k in zip(table.cpu().numpy(), lens.tolist()) for x in r[: -(-k // page)]]
        head, count = state.tolist()
        free = ring.cpu().numpy()[(head + np.arange(count)) % pool].tolist()
        assert sorted(held + free) == list(range(pool))
        slots = step.slots.cpu().numpy()
        kept = slots[slots >= 0]
        assert len(set(kept.tolist())) == kept.size and set((kept // page).tolist()) <= set(held)
    assert ran_out & 1 == (pool == 100)   # the small one does not hold all of them at times
