"""Block-sparse attention with both query blocks of a CTA at work: more items than two per SM, lists of several blocks.

The kernel hands item i < SMs to the first lane of CTA i, item SMs + i to its second, and the others by a counter, so
smaller calls run one lane a CTA.  Every case is checked against the dense kernel's bits or the formula in 64 bits
(the bounds of test_gpu_sparse.py), on heads from everywhere in the call.
"""
import pytest
import torch

from test_gpu_sparse import MODES, all_blocks, bits, expect, inputs, random_lists

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def check_heads(q, k, v, mode, lists, counts, heads):
    """One call over all heads; the given ones against the formula, the empty rows of all of them against 0."""
    from video_dit_quantized_b200 import sage, sparse
    B, H, N, d = q.shape
    ws = sage.alloc_workspace(B, H, N, d, mode, q.device)
    o = torch.full_like(q, 9.0)
    for rep in range(2):                                    # the second call finds the counter used
        sparse.attn_fwd_sparse(q, k, v, mode, lists, counts, o=o, workspace=ws)
        assert sage.status(ws) == sage.OK and torch.isfinite(o).all()
    pick = lambda t: t[:, heads].contiguous()
    val, tol = expect(pick(q), pick(k), pick(v), mode, pick(lists), pick(counts))
    err = (pick(o).double() - val).abs()
    assert (err <= tol).all(), (float((err - tol).max()), int((err > tol).sum()))
    nT = lists.shape[2]
    empty = (counts == 0)[..., None].expand(-1, -1, -1, 128).reshape(B, H, nT * 128)[:, :, :N]
    assert not o[empty].any()
    return o


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("B,H,N,d", [(1, 90, 1500, 128), (2, 45, 1601, 64), (1, 60, 2560, 64), (3, 37, 1025, 128)])
def test_all_blocks_of_many_items_are_the_dense_call(B, H, N, d, mode, cuda_dev):
    from video_dit_quantized_b200 import sage, sparse
    nT = -(-N // 128)
    assert B * H * nT > 3 * sms()
    q, k, v, _ = inputs(B, H, N, d, 200 + N, cuda_dev)
    lists, counts = all_blocks(B, H, nT, cuda_dev)
    ref = sage.attn_fwd(q, k, v, mode)
    for rep in range(3):
        got = sparse.attn_fwd_sparse(q, k, v, mode, lists, counts)
        assert torch.equal(bits(got), bits(ref)), rep


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("B,H,N,d,width", [(1, 90, 1500, 128, 12), (1, 70, 2300, 64, 18), (2, 40, 1900, 128, 9), (1, 130, 1100, 64, 5)])
def test_ragged_lists_of_many_items(B, H, N, d, width, mode, cuda_dev):
    nT = -(-N // 128)
    assert B * H * nT > 3 * sms()
    q, k, v, g = inputs(B, H, N, d, 300 + N + mode, cuda_dev)
    lists, counts = random_lists(B, H, nT, width, g, cuda_dev)
    check_heads(q, k, v, mode, lists, counts, [0, 1, H // 3, H // 2, H - 17, H - 2, H - 1])


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("c0,c1", [(0, 9), (9, 0), (1, 9), (9, 1), (2, 3), (9, 9), (5, 6)])
def test_two_lanes_of_any_two_lengths(c0, c1, d, mode, cuda_dev):
    """Every CTA gets one list of c0 blocks and one of c1, at the same time; what is behind them is empty."""
    n, nT = sms(), 9
    H = -(-2 * n // nT)
    q, k, v, g = inputs(1, H, nT * 128 - 52, d, 10 * c0 + c1, cuda_dev)
    lists, _ = random_lists(1, H, nT, 9, g, cuda_dev, lo=9)
    item = torch.arange(H * nT, device=cuda_dev)
    counts = torch.where(item < n, c0, torch.where(item < 2 * n, c1, 0)).to(torch.int32).view(1, H, nT)
    edge = n // nT                                          # the head where c0 turns into c1
    check_heads(q, k, v, mode, lists, counts, [0, 1, edge - 1, edge, edge + 1, H - 2, H - 1])


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("d", [64, 128])
def test_long_short_and_empty_lists_in_turn(d, mode, cuda_dev):
    """Items of 0, 1 and 11 blocks in patterns that give a lane one kind after another, its neighbour another."""
    n, nT = sms(), 11
    H = -(-4 * n // nT)
    q, k, v, g = inputs(1, H, nT * 128 - 3, d, 77, cuda_dev)
    lists, _ = random_lists(1, H, nT, 11, g, cuda_dev, lo=11)
    item = torch.arange(H * nT, device=cuda_dev)
    length = torch.tensor([11, 0, 1], device=cuda_dev)
    for kind in (item % 3, item // n % 3, item // (2 * n) % 3, (item * 7 // 5) % 3):
        counts = length[kind].to(torch.int32).view(1, H, nT)
        check_heads(q, k, v, mode, lists, counts, [0, H // 4, H // 2, H - 1])
