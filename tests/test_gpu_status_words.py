"""Status words that are not the device's are refused before anything is launched."""
import pytest
import torch

from group_affine_bit_gb300 import api, synth

pytestmark = pytest.mark.gpu


def test_status_words_are_checked():
    cache = api.KVCache.empty(2, 16, 2, 64)
    x = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    rope = api.Rope(api.rope_turns([1.0] * 32))
    _, codes, sc, bi = synth.problem(4, 64, 1, 64, 128, seed=1)
    w = api.pack(codes.cuda(), sc.cuda(), bi.cuda(), 4, 64)
    rows = api.pack_rows(w)
    calls = (lambda s: api.paged_attention(x, cache, i.view(1, 1), i, status=s),
             lambda s: api.rope_append(x, k, k, i, i, rope, cache, status=s),
             lambda s: api.embed_rows(w, i, status=s), lambda s: api.embed_rows_copy(w, rows, i, status=s))
    for call in calls:
        for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64, device="cuda"),
                    torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda")):
            with pytest.raises(ValueError):
                call(bad)
        for dtype in (torch.int32, torch.uint32):
            good = torch.zeros(1, dtype=dtype, device="cuda")
            call(good)
            assert int(good.view(torch.int32)[0]) == 0
