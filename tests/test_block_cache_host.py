"""What api.BlockCache refuses when it is made, with a word on what is wrong, rather than in every call."""
import pytest
import torch

from group_affine_bit_gb300 import api


def cache(page, scales, heads=2, pages=3, dtype=torch.int8):
    k = torch.zeros(pages, page, heads, 32, dtype=dtype)
    return api.BlockCache(k, k.clone(), scales, scales.clone() if scales.is_contiguous() else scales)


@pytest.mark.parametrize("page,blocks", [(256, 1), (512, 2), (48, 1), (96, 2), (24, 1), (65536, 256)])
def test_blocks_that_no_call_takes(page, blocks):
    with pytest.raises(ValueError, match="power of two"):
        cache(page, torch.ones(3, blocks, 2))


@pytest.mark.parametrize("block", [0, -16, 3, 24, 256])
def test_empty_takes_no_such_block(block):
    with pytest.raises(ValueError, match="power of two"):
        api.BlockCache.empty(3, 512, 2, 32, block=block, device="cpu")
    with pytest.raises(ValueError, match="divide"):
        api.BlockCache.empty(3, 16, 2, 32, block=32, device="cpu")


def test_scales_that_share_a_place():
    for scales in (torch.ones(1, 4, 2).expand(3, 4, 2), torch.ones(3, 4, 1).expand(3, 4, 2), torch.ones(3, 1, 2).expand(3, 4, 2),
                   torch.ones(40).as_strided((3, 4, 2), (4, 2, 1)), torch.ones(40).as_strided((3, 4, 2), (1, 3, 6))):
        with pytest.raises(ValueError, match="share a place"):
            cache(64, scales)


def test_what_is_taken_fails_only_for_want_of_a_gpu():
    for page, scales in ((128, torch.ones(3, 1, 2)), (256, torch.ones(3, 2, 2)), (64, torch.ones(3, 64, 2)), (64, torch.ones(2, 3, 4).permute(1, 2, 0)),
                         (64, torch.ones(60).as_strided((3, 4, 2), (17, 2, 1))), (64, torch.ones(60).as_strided((3, 4, 2), (1, 3, 12))),
                         (16, torch.ones(1).expand(3, 1, 1).contiguous())):
        with pytest.raises(ValueError, match="CUDA"):
            cache(page, scales, heads=scales.shape[2])
