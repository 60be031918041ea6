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
