"""sage_select_blocks against the scores in 64 bits: the same sets, exactly."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def want(q, k, keep, first, window):
    """lists, counts of one [N, d] head in numpy fp64, ranked by (forced, score, -index)."""
    N, d = q.shape
    nT = -(-N // 128)
    pool = lambda x: np.stack([x[i * 128:(i + 1) * 128].astype(np.float64).sum(0) / min(128, N - i * 128)
                               for i in range(nT)]).astype(np.float32).astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        s = pool(q) @ pool(k).T
    n = min(keep, nT)
    lists = np.full((nT, keep), -1, np.int32)
    for i in range(nT):
        key = [(-(j < first or (window >= 0 and abs(i - j) <= window)), np.isnan(s[i, j]), -s[i, j], j) for j in range(nT)]
        key = sorted((f, bad, 0.0 if bad else v, j) for f, bad, v, j in key)
        lists[i, :n] = sorted(j for _, _, _, j in key[:n])
    return lists, np.full(nT, n, np.int32)


def check(q, k, keep, first, window):
    from video_dit_quantized_b200 import sparse
    B, H, N, d = q.shape
    lists, counts = sparse.select_blocks(q, k, keep, first=first, window=window)
    ql, kl = q.float().cpu().numpy(), k.float().cpu().numpy()
    for b in range(B):
        for h in range(H):
            wl, wc = want(ql[b, h], kl[b, h], keep, first, window)
            assert np.array_equal(lists[b, h].cpu().numpy(), wl), (b, h)
            assert np.array_equal(counts[b, h].cpu().numpy(), wc)


@pytest.mark.parametrize("B,H,N,d,keep,first,window", [
    (1, 1, 1, 64, 1, 0, 0), (1, 2, 127, 128, 3, 1, 0), (2, 3, 129, 64, 1, 0, -1), (1, 2, 1000, 128, 3, 0, 0),
    (1, 2, 1000, 128, 8, 0, 0), (1, 1, 1000, 64, 20, 30, 30), (2, 2, 4500, 64, 5, 2, 1), (1, 3, 8200, 128, 7, 0, -1),
    (1, 1, 40000, 64, 33, 1, 2), (1, 1, 128 * 257, 128, 256, 0, 0)])
def test_sets(B, H, N, d, keep, first, window, cuda_dev):
    g = torch.Generator(device=cuda_dev)
    g.manual_seed(N + keep)
    q, k = (torch.randn((B, H, N, d), generator=g, device=cuda_dev).to(torch.bfloat16) for _ in range(2))
    check(q, k, keep, first, window)


def test_long_rows(cuda_dev):
    """More blocks than a sixteen-row CTA holds (four rows a CTA), and the most that are allowed."""
    from video_dit_quantized_b200 import sparse
    g = torch.Generator(device=cuda_dev)
    g.manual_seed(3)
    for nT in (1600, sparse.SELECT_MAX_BLOCKS):
        N = nT * 128 - 5
        q, k = (torch.randn((1, 1, N, 64), generator=g, device=cuda_dev).to(torch.bfloat16) for _ in range(2))
        lists, counts = sparse.select_blocks(q, k, 40, first=1, window=1)
        pool = lambda x: (torch.nn.functional.pad(x[0, 0].double(), (0, 0, 0, 5)).view(nT, 128, 64).sum(1) /
                          torch.tensor([128.0] * (nT - 1) + [123.0], device=cuda_dev, dtype=torch.float64)[:, None])
        s = pool(q).float().double() @ pool(k).float().double().T
        i = torch.arange(nT, device=cuda_dev)
        s[((i[:, None] - i).abs() <= 1) | (i < 1)[None].expand(nT, nT)] = float("inf")
        ref = s.sort(dim=1, descending=True, stable=True).indices[:, :40].sort(dim=1).values
        assert torch.equal(lists[0, 0].long(), ref) and (counts == 40).all()


def test_ties_go_to_the_lowest_index(cuda_dev):
    """Equal blocks have equal scores to the last bit; all-zero inputs tie everywhere."""
    x = torch.randn((1, 2, 4, 128, 64), device=cuda_dev).to(torch.bfloat16)
    k = x[:, :, [0, 1, 1, 2, 1, 3, 0, 1, 2, 2]].reshape(1, 2, 1280, 64).contiguous()
    q = torch.randn((1, 2, 1280, 64), device=cuda_dev).to(torch.bfloat16)
    for keep in (1, 2, 3, 4, 5, 7, 9):
        check(q, k, keep, 0, -1)
        check(q, k, keep, 0, 0)
    z = torch.zeros((1, 1, 5000, 128), dtype=torch.bfloat16, device=cuda_dev)
    check(z, z, 6, 0, -1)
    check(z, -z, 6, 1, 1)


def test_scores_that_share_their_high_half(cuda_dev):
    """Scores that differ only far behind the leading bits are still told apart."""
    q = torch.ones((1, 1, 128 * 40, 64), dtype=torch.bfloat16, device=cuda_dev)
    k = torch.ones((1, 1, 40, 128, 64), dtype=torch.float32, device=cuda_dev) * 128
    g = torch.Generator(device=cuda_dev)
    g.manual_seed(11)
    k[..., 4] = 0
    # the mean of channel 4 is r * 2^-21 beside 63 channels of 128: below the 20 leading bits, exact in fp64
    k[0, 0, :, 0, 4] = 2.0 ** -14 * torch.randint(0, 20, (40,), generator=g, device=cuda_dev)
    k = k.view(1, 1, 128 * 40, 64).to(torch.bfloat16)
    for keep in (1, 7, 20):
        check(q, k, keep, 0, -1)


def test_scores_that_are_not_numbers_rank_last(cuda_dev):
    q, k = (torch.randn((1, 1, 1280, 64), device=cuda_dev).to(torch.bfloat16) for _ in range(2))
    k[0, 0, 130, 3] = float("nan")
    k[0, 0, 700, 1] = float("nan")
    check(q, k, 8, 0, -1)
    check(q, k, 9, 0, -1)
    check(q, k, 3, 0, 0)
