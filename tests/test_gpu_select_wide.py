"""Lists as wide as their type allows: the places behind the last kept block."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("keep", [2 ** 31 - 1, 2 ** 31 - 33])
def test_the_widest_list(keep, cuda_dev):
    """One row of nearly 2^31 places, one block in it: -1 in all the others, and nothing in front of or behind the row."""
    from video_dit_quantized_b200 import sparse
    q = torch.randn((1, 1, 100, 64), device=cuda_dev).to(torch.bfloat16)
    pad = torch.full((keep + 128,), 7, dtype=torch.int32, device=cuda_dev)
    lists, counts = sparse.select_blocks(q, q, keep, lists=pad[64:64 + keep].view(1, 1, 1, keep))
    assert counts.item() == 1 and lists[0, 0, 0, 0].item() == 0
    row = lists.view(-1)
    assert row[1:].max().item() == -1 and row[1:].min().item() == -1
    assert (pad[:64] == 7).all() and (pad[64 + keep:] == 7).all()
