"""Appends whose tokens do not come block by block, or that bring a block more than it has: the status word says so, and
everything but the blocks concerned is as it should be.  Orders that are allowed leave it as it was."""
import pytest
import torch

import paged_ref
from group_affine_bit_gb300 import api
from test_gpu_block_append import Pool, parts, rows_of

pytestmark = pytest.mark.gpu

HQ, HK, DIM, PAGE = 2, 1, 32, 32


def append(pool, slots, rows, status=True, rotary=DIM):
    word = torch.zeros(1, dtype=torch.int32, device="cuda") if status else None
    rope = api.Rope(api.rope_turns(paged_ref.turns_of(rotary) if rotary else []))
    pos = torch.arange(len(slots), dtype=torch.int32, device="cuda")
    q = api.rope_append(*parts(rows.cuda(), HQ, HK, DIM), pos, torch.tensor(slots, dtype=torch.int32, device="cuda"), rope, pool.cache, status=word)
    torch.cuda.synchronize()
    return q, int(word[0]) if status else None


def pools(pages, kv, block):
    return [Pool(pages, PAGE, HK, DIM, kv, block, seed=5) for _ in range(2)]


def step_by_step(requests, tokens):
    """Token by token across the requests, each on a page of its own."""
    return [r * PAGE + t for t in range(tokens) for r in range(requests)]


BROKEN = {
    "-1 between": (8, [0, 1, -1, 2, 64, 65], [0]),
    "another block between": (8, [64, 0, 8, 9, 1], [0]),
    "a slot beyond the pool between": (8, [64, 0, 1, 1 << 20, 2], [0]),
    "two requests in turn": (16, step_by_step(2, 3), [0, 2]),
    "forty requests in turn": (16, step_by_step(40, 3), [2 * r for r in range(40)]),
    "far behind": (32, [5] + list(range(PAGE, PAGE + 6000)) + [6], [0]),
    "a slot twice": (1, [64, 65, 3, 3], [3]),
    "a slot twice, far behind": (1, [3] + list(range(PAGE, PAGE + 3000)) + [3], [3]),
    "more tokens than a block has": (4, [64, 65, 0, 1, 2, 3, 3, 3, 2, 1, 0], [0]),
    "one token more than a block has": (16, [64] + list(range(16)) + [3, 80], [0]),
}


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("name", BROKEN)
def test_broken_orders_are_reported(name, kv):
    block, slots, blocks = BROKEN[name]
    pages = (max(s for s in slots if s < 1 << 20) // PAGE) + 2
    one, two = pools(pages, kv, block)
    rows = rows_of(len(slots), HQ, HK, DIM, torch.Generator().manual_seed(1))
    q, status = append(one, slots, rows)
    assert status == (6 if name.startswith("a slot beyond") else 4)
    # the same rows without those of the blocks concerned
    kept = [s if s // block not in blocks and s < 1 << 20 else -1 for s in slots]
    want, status = append(two, kept, rows)
    assert status == 0 and torch.equal(q, want)
    for (c1, s1), (c2, s2) in zip(one.now(), two.now()):
        each = PAGE // block
        other = torch.ones(pages * each, dtype=torch.bool)
        other[blocks] = False
        a, b = (c.reshape(pages * each, block, HK, DIM)[other].nan_to_num(1e9) for c in (c1, c2))
        assert torch.equal(a, b) and torch.equal(*(s.reshape(pages * each, HK)[other].nan_to_num(-1) for s in (s1, s2)))


@pytest.mark.parametrize("rotary", [DIM, 0])
@pytest.mark.parametrize("block", [1, 2, 16, 32])
def test_allowed_orders_are_not(block, rotary):
    """Blocks in any order, their tokens in any order within; numbers that a table of names holds close together."""
    g = torch.Generator().manual_seed(2)
    for T in (1, 2, 31, 33, 64, 500, 2049, 9000):
        pages = 3 * T // PAGE + 4
        pool = Pool(pages, PAGE, HK, DIM, "int8", block, seed=6)
        slots = []
        for b in torch.randperm(pages * PAGE // block, generator=g).tolist():
            n = int(torch.randint(1, block + 1, (1,), generator=g))
            slots += (b * block + torch.randperm(block, generator=g)[:n]).tolist()
        slots = slots[:T]
        assert append(pool, slots, rows_of(T, HQ, HK, DIM, g), rotary=rotary)[1] == 0
        assert len(slots) == T
        if block == 1:
            slots[T // 2] = -1
            assert append(pool, slots, rows_of(T, HQ, HK, DIM, g), rotary=rotary)[1] == 0


def test_each_of_many_tokens_is_looked_at():
    """One slot of a long call named twice, wherever the two are."""
    T, g = 20000, torch.Generator().manual_seed(3)
    pool = Pool(T // PAGE + 2, PAGE, HK, DIM, "int8", 1, seed=7)
    rows = rows_of(T, HQ, HK, DIM, g)
    assert append(pool, list(range(T)), rows)[1] == 0
    for i, j in ((0, T - 1), (1, 2), (7000, 15000), (T - 2, T - 1), (255, 256)):
        slots = list(range(T))
        slots[j] = slots[i]
        assert append(pool, slots, rows)[1] == 4


def test_the_status_word_changes_nothing_else():
    g = torch.Generator().manual_seed(4)
    slots = list(range(5, 900))
    rows = rows_of(len(slots), HQ, HK, DIM, g)
    one, two = pools(40, "int8", 16)
    a, b = append(one, slots, rows)[0], append(two, slots, rows, status=False)[0]
    assert torch.equal(a, b)
    assert all(torch.equal(x[0], y[0]) and torch.equal(x[1].nan_to_num(-1), y[1].nan_to_num(-1)) for x, y in zip(one.now(), two.now()))
