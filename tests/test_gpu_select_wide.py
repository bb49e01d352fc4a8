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


@pytest.mark.parametrize("d", [64, 128])
def test_sums_of_values_too_far_apart_keep_their_order(d, cuda_dev):
    """1e20 and 1 in one channel: no fp64 sum holds both, so the mean is that of the documented order (rows r, r + 8,
    r + 16, .. for each r < 8, then the eight sums).  Block 0: (1e20 + 1) - 1e20 = 0 within one r.  Block 1:
    (1e20 - 1e20) + 1 = 1.  Block 2: 0 from r = 0 and 1 from r = 1 give 1, where rows in a row would give 0."""
    from video_dit_quantized_b200 import sparse
    q = torch.zeros((1, 1, 384, d), dtype=torch.bfloat16, device=cuda_dev)
    k = torch.zeros_like(q)
    q[..., 3] = 1
    for block, rows in enumerate(({0: 1e20, 8: 1, 16: -1e20}, {0: 1e20, 8: -1e20, 16: 1}, {0: 1e20, 1: 1, 8: -1e20})):
        for r, x in rows.items():
            k[0, 0, block * 128 + r, 3] = x
    lists, counts = sparse.select_blocks(q, k, 2, window=-1)
    assert lists[0, 0].tolist() == [[1, 2]] * 3 and (counts == 2).all()
