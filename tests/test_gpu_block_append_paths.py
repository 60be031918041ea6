"""Every way of the block cache's append through prompt chunks: pairings and lengths that choose kernels, blocks whose
sines pass what shared memory has for them, and the roundings that a block has gathered once it is full.

Tolerances of single calls: blocks_ref.Checker, as test_gpu_block_append.py derives them."""
import pytest
import torch

import paged_ref
from group_affine_bit_gb300 import api
from test_gpu_block_append import Pool, places, rows_of, run

pytestmark = pytest.mark.gpu

TABLE = 136 << 10     # bytes that hold sines, 8 to a token and pair of the 8 * ceil(rotary / 16) that a row of them has


def tokens_of(rows):
    """Tokens from which on a CTA takes so many rows of a call."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return {1: 1, 2: 2, 8: 8, 16: 32}[rows] * sms


def chunks(total, block, requests=9):
    """Requests' tokens (first, count), `total` in all, whose blocks begin anywhere in a CTA's rows."""
    spans, left = [], total
    for i in range(requests):
        n = left if i == requests - 1 else left // (requests - i) - 7 * i % 5
        spans.append(((i * 37 + 3 * i * i) % (2 * block), n))
        left -= n
    return spans


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("dim,block,rotary,neighbour,rows", [
    (256, 128, 256, False, 16), (256, 128, 256, True, 16), (256, 128, 248, False, 16), (256, 128, 254, False, 16),
    (512, 64, 512, False, 16), (512, 64, 512, True, 8), (512, 64, 504, False, 8), (512, 64, 510, False, 8),
    (512, 128, 512, False, 8), (512, 128, 504, False, 1), (512, 128, 510, False, 1), (512, 128, 504, False, 8), (512, 128, 510, False, 2)])
def test_blocks_whose_sines_pass_the_table(dim, block, rotary, neighbour, rows, kv):
    """Rows within the table beside rows beyond it, in all pairings: half pairs in runs of eight, four and one value, and
    neighbours; one row of the call to a CTA, and several, at any of which a block begins."""
    assert TABLE // (64 * -(-rotary // 16)) < block + rows - 1, "the table holds all of them"
    total = tokens_of(rows) + 11
    spans = chunks(total, block, 9) if rows > 1 else [(0, 2 * block), (block - 5, block + 9), (3, 1)]
    run(spans, 1, 1, dim, 128, block, kv, rotary=rotary, neighbour=neighbour, seed=rotary + rows)


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("times", [9, 17, 33])
@pytest.mark.parametrize("rotary,neighbour,axes", [(80, False, 1), (40, False, 2), (78, False, 1), (0, False, 1), (80, True, 3), (38, True, 1), (0, True, 1)])
def test_prompt_chunks_in_every_pairing(rotary, neighbour, axes, times, kv):
    """Two and four tokens of q to a CTA, four chunks of k and v to a thread."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    run(chunks(times * sms + 5, 16), 3, 2, 80, 32, 16, kv, rotary, axes, neighbour, seed=rotary + times, in_place=times != 17)


@pytest.mark.parametrize("kv", ["int8", "e4m3"])
@pytest.mark.parametrize("steps", ["slow", "random", "falling"])
def test_what_a_block_has_gathered_when_it_is_full(steps, kv):
    """A block filled token by token: each value is off by half a step of every scale that the block had since it was written.

    int8: a rounding is off by half a step of the scale that it is for, and 2^-16 of one for the product in fp32 (|code| <=
    127, two roundings of 2^-24).  e4m3: the first by 2^-4 of the value, or half a subnormal step (2^-10) of the scale where
    that is more; scales are powers of two, so that a later one is exact but for codes that fall below the normal ones,
    off by half a subnormal step."""
    block, heads, dim = 128, 2, 32
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(block, heads, dim, generator=g) * 0.4).clamp(-0.99, 0.99).bfloat16()
    if steps == "slow":        # each token's largest is the next number of its type: the scale grows with every one of them
        x[:, :, 5] = torch.arange(0x3f80, 0x3f80 + block, dtype=torch.int16).view(torch.bfloat16)[:, None]
    if steps == "falling":     # and with none
        x[:, :, 5] = torch.arange(0x4000, 0x4000 - block, -1, dtype=torch.int16).view(torch.bfloat16)[:, None]
    pool = Pool(3, 128, heads, dim, kv, block, seed=4)
    rope = api.Rope(api.rope_turns([]))
    rows = x.cuda()
    room, scales = torch.zeros(block, heads, dim, dtype=torch.float64), []
    for i in range(block):
        row = rows[i: i + 1]
        api.rope_append(row, row, row, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([128 + i], dtype=torch.int32, device="cuda"), rope, pool.cache)
        scale = pool.vs[1, 0].double().cpu()
        grown = scale > scales[-1] if scales else torch.ones(heads, dtype=torch.bool)
        assert not scales or bool((scale >= scales[-1]).all())
        scales.append(scale)
        rounded = scale[None, :, None] * (0.5 + 2.0 ** -16 if kv == "int8" else 2.0 ** -10)
        room[:i] += torch.where(grown[None, :, None], rounded, 0.0)
        room[i] = rounded[0] if kv == "int8" else torch.maximum(rounded[0], 2.0 ** -4 * x[i].double().abs())
    if kv == "int8":
        distinct = len({float(s[0]) for s in scales})
        assert distinct == (block if steps == "slow" else 1) or steps == "random"
    for codes, held in ((pool.k, pool.ks), (pool.v, pool.vs)):
        assert torch.equal(held[1, 0].double().cpu(), scales[-1])
        got = codes[1].double().cpu() if kv == "int8" else codes[1].float().double().cpu()
        assert bool(((got * scales[-1][:, None] - x.double()).abs() <= room).all())
