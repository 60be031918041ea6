"""Reading a paged cache back where there is little to read: what the status word says."""
import pytest
import torch

from group_affine_bit_gb300 import api
from test_gpu_paged_read import pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_no_room_at_all_is_reported_too(kv):
    cache, _, _ = pool(3, 16, 2, 32, kv, 16, 8)
    table = torch.tensor([[2], [0]], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, _ = api.paged_read(cache, table, torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda"), rows=0, status=status)
    assert k.shape == (0, 2, 32) and int(status[0]) == 0
    api.paged_read(cache, table, torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda"), rows=0, status=status)
    assert int(status[0]) == 2
    status.zero_()
    api.paged_read(cache, table[:0], torch.tensor([0], dtype=torch.int32, device="cuda"), rows=0, status=status)
    assert int(status[0]) == 0


def test_codes_and_rows_beyond_32_bits():
    """Pages whose codes begin beyond 2^32 bytes of the pool, read to rows that begin beyond 2^32 bytes of the output."""
    page, heads, dim = 64, 8, 512
    pages = (1 << 32) // (page * heads * dim) + 3
    k, v = (torch.zeros(pages, page, heads, dim, dtype=torch.int8, device="cuda") for _ in "kv")
    ks, vs = (torch.ones(pages, 4, heads, device="cuda") for _ in "kv")
    last = torch.randint(-127, 128, (2, page, heads, dim), device="cuda", dtype=torch.int8)
    k[-1], v[-1], vs[-1] = last[0], last[1], 0.5
    rows = (1 << 32) // (heads * dim * 2) + page
    out = [torch.full((rows, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    # one request of no page's tokens but the last's, behind one whose entries are all page 0
    wide = -(-rows // page)
    table = torch.zeros(2, wide, dtype=torch.int32, device="cuda")
    table[1, 0] = pages - 1
    starts = torch.tensor([0, rows - page, rows], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    api.paged_read(api.BlockCache(k, v, ks, vs), table, starts, k=out[0], v=out[1], status=status)
    assert int(status[0]) == 0
    assert torch.equal(out[0][-page:], last[0].bfloat16()) and torch.equal(out[1][-page:], last[1].bfloat16() * 0.5)
    assert not bool(out[0][:-page].any()) and not bool(out[1][:-page].any())
