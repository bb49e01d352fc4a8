"""The sparse calls at their edges: values at the ends of the types' ranges, neighbouring items with and without
blocks, memory that was in use before, and tensors and lists whose offsets pass 2^31 elements."""
import math

import numpy as np
import pytest
import torch

from test_gpu_norm_rope import ALL, HALVES, RMS, close, want as norm_want
from test_gpu_select import check as check_select

pytestmark = pytest.mark.gpu

BF16, I8, QTOK = 0, 1, 2


def draw(shape, seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)


@pytest.mark.parametrize("q_mul,k_mul,k_off", [
    (1e-38, 1e10, 0.0), (1e10, 1e-38, 0.0), (1e-20, 1e18, 1e20), (1e-36, 1e-36, 0.0), (1e30, 1e30, 0.0),
    (1.0, 50.0, 1e4), (0.0, 1.0, 0.0)])
@pytest.mark.parametrize("d", [64, 128])
def test_block_scores_over_the_range_of_the_type(d, q_mul, k_mul, k_off, cuda_dev):
    """Means whose squares or reciprocals leave the normal range of fp32, and keys with an offset far above their
    spread: the sets are still those of the scores in 64 bits."""
    q = (draw((1, 2, 3900, d), d, cuda_dev).float() * q_mul).to(torch.bfloat16)
    k = (draw((1, 2, 3900, d), d + 1, cuda_dev).float() * k_mul + k_off).to(torch.bfloat16)
    check_select(q, k, 5, 1, 0)


def test_block_scores_with_infinite_tokens(cuda_dev):
    """One infinite value makes its block's mean infinite; the other blocks rank as ever.  Token 0 is among them."""
    for at in (0, 700):
        q, k = draw((1, 2, 1500, 64), 3, cuda_dev), draw((1, 2, 1500, 64), 4, cuda_dev)
        k[0, 0, at, 5] = math.inf
        k[0, 1, at, 6] = -math.inf
        q[0, 1, 300, 6] = math.inf
        check_select(q, k, 4, 0, -1)


@pytest.mark.parametrize("nT,d,keep", [(128, 64, 12), (129, 128, 128), (640, 64, 64), (641, 128, 1), (641, 64, 640)])
def test_block_rows_at_the_borders_of_their_forms(nT, d, keep, cuda_dev):
    """Rows that just fit a lane's registers or a power of blocks, and one more; lists that keep one and all but one."""
    q, k = (draw((1, 1, nT * 128 - 77, d), s, cuda_dev) for s in (17, 18))
    check_select(q, k, keep, 0, -1)


@pytest.mark.parametrize("mode", [BF16, I8, QTOK])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_a_bad_index_adds_nothing_whatever_block_0_holds(mode, value, cuda_dev):
    """V of block 0 is not a finite number; rows that do not list it are those without the bad index."""
    from video_dit_quantized_b200 import sage, sparse
    q, k, v = (draw((1, 2, 600, 128), s, cuda_dev) for s in (1, 2, 3))
    v[:, :, 5, :64] = value
    if mode == BF16:
        k[:, :, 7] = value
    nT = 5
    good = torch.tensor([[1, 2], [3, 4], [2, 2], [4, 1], [3, 2]], dtype=torch.int32, device=cuda_dev)
    good = good.expand(1, 2, nT, 2).contiguous()
    two = torch.full((1, 2, nT), 2, dtype=torch.int32, device=cuda_dev)
    ref = sparse.attn_fwd_sparse(q, k, v, mode, good, two)
    ws = sage.alloc_workspace(1, 2, 600, 128, mode, cuda_dev)
    for at in range(3):
        bad = torch.cat((good[..., :at], torch.full_like(good[..., :1], nT), good[..., at:]), -1).contiguous()
        got = sparse.attn_fwd_sparse(q, k, v, mode, bad, two + 1, workspace=ws)
        assert sage.status(ws) == sage.EINVAL
        same = (got == ref) | (got.isnan() & ref.isnan())
        assert same.all(), (at, int((~same).sum()))
        if mode == BF16:
            assert torch.isfinite(got).all()


@pytest.mark.parametrize("mode", [BF16, I8, QTOK])
@pytest.mark.parametrize("d", [64, 128])
def test_items_of_other_heads_with_empty_ones_between(d, mode, cuda_dev):
    """One query block a head, so that each item of a CTA has another head's V scales; empty lists between them, at
    random and in turn.  A list of the one block is the dense call's bits, an empty one zeros."""
    from video_dit_quantized_b200 import sage, sparse
    H, N = 4000, 128
    q, k, v = (draw((1, H, N, d), s, cuda_dev) for s in (5, 6, 7))
    v *= torch.linspace(0.01, 50, H, device=cuda_dev)[torch.randperm(H, device=cuda_dev)][None, :, None, None].to(torch.bfloat16)
    ref = sage.attn_fwd(q, k, v, mode)
    lists = torch.zeros((1, H, 1, 1), dtype=torch.int32, device=cuda_dev)
    g = torch.Generator(device=cuda_dev)
    g.manual_seed(8)
    i = torch.arange(H, device=cuda_dev)
    for counts in (torch.randint(0, 2, (H,), generator=g, device=cuda_dev), i // 148 % 2, i // 296 % 2, i % 2,
                   (torch.rand(H, generator=g, device=cuda_dev) < 0.1)):
        counts = counts.to(torch.int32).view(1, H, 1)
        for rep in range(5):
            got = sparse.attn_fwd_sparse(q, k, v, mode, lists, counts)
            assert torch.equal(got.view(torch.int16), torch.where(counts[..., None] > 0, ref, 0).view(torch.int16)), rep


@pytest.mark.parametrize("mode", [BF16, I8, QTOK])
def test_memory_of_the_call_s_own_was_in_use(mode, cuda_dev):
    """Scratch and workspace that a call allocates itself may hold anything."""
    from video_dit_quantized_b200 import sage, sparse
    q, k, v = (draw((1, 3, 1300, 128), s, cuda_dev) for s in (9, 10, 11))
    ws = sage.alloc_workspace(1, 3, 1300, 128, mode, cuda_dev)
    lists, counts = sparse.select_blocks(q, k, 3)
    ref = sparse.attn_fwd_sparse(q, k, v, mode, lists, counts, workspace=ws)
    for fill in (0xFF, 0x7F, 0x80):
        dirty = [torch.full((n,), fill, dtype=torch.uint8, device=cuda_dev) for n in (ws.numel(), sparse.select_scratch_bytes(1, 3, 1300, 128))]
        del dirty
        l2, c2 = sparse.select_blocks(q, k, 3)
        got = sparse.attn_fwd_sparse(q, k, v, mode, l2, c2)
        assert torch.equal(l2, lists) and torch.equal(c2, counts)
        assert torch.equal(got.view(torch.int16), ref.view(torch.int16)), fill


def test_norm_of_more_than_2_31_elements(cuda_dev):
    """The last tokens of a tensor whose offsets pass 2^31 elements, in both kinds of layout."""
    from video_dit_quantized_b200 import sparse
    B, N, H, d = 2, 210001, 40, 128
    x = torch.empty((B, N, H, d), dtype=torch.bfloat16, device=cuda_dev)
    part = draw((1, 2000, H, d), 12, cuda_dev)
    for b in range(B):
        for n in range(0, N, 2000):
            x[b, n:n + 2000] = part[0, :min(2000, N - n)] * (1 + b)
    w = draw((H * d,), 13, cuda_dev)
    angle = torch.arange(N, device=cuda_dev, dtype=torch.float32)[:, None] * (0.001 / (1 + torch.arange(d // 2, device=cuda_dev)))
    cos, sin = angle.cos(), angle.sin()
    assert x.numel() > 2 ** 31
    for ranks in (0, 2):
        y = sparse.qk_norm_rope(x, wq=w, scope=ALL, cos=cos, sin=sin, rope=HALVES, ranks=ranks)[0]
        for b, n0 in ((0, 0), (1, N - 300)):
            ref, mag = norm_want(x[b:b + 1, n0:n0 + 300], w, None, cos[n0:n0 + 300], sin[n0:n0 + 300], RMS, ALL, 1e-6, HALVES, 0, ranks)
            got = y[b:b + 1, :, n0:n0 + 300] if ranks == 0 else y[:, b:b + 1, n0:n0 + 300]
            close(got, ref, mag)
        del y


def test_lists_of_more_than_2_31_entries(cuda_dev):
    """Rows wider than the number of blocks, -1 behind, over more than 2^31 entries."""
    from video_dit_quantized_b200 import sparse
    H, N, d, keep = 60, 128 * 4000, 64, 9000
    q = draw((1, H, N, d), 14, cuda_dev)
    lists, counts = sparse.select_blocks(q, q, keep)
    assert lists.numel() > 2 ** 31 and (counts == 4000).all()
    row = torch.full((keep,), -1, dtype=torch.int32, device=cuda_dev)
    row[:4000] = torch.arange(4000, dtype=torch.int32, device=cuda_dev)
    for h in (0, H // 2, H - 1):
        assert (lists[0, h] == row).all(), h


@pytest.mark.parametrize("mode", [BF16, QTOK])
def test_attention_over_the_longest_sequence(mode, cuda_dev):
    """2^31 elements a tensor but for one block: the first and last query blocks attend to the first and last keys.
    Rows against the formula in 64 bits on the same 512 keys, with the rounding of every operand (half steps):
    fp32 scores (d + 8) * 2^-24 of sum |q||k|, bf16 P 2^-8; INT8 codes of q (a token) and k (a block, smoothed by a
    mean below 0.1 here) 1/254 of the largest; e4m3 P and V 2^-4 of the value or 2^-10 / 448 of the largest."""
    from video_dit_quantized_b200 import sage, sparse
    nT, d = 131071, 128
    N = nT * 128
    part = draw((3, 1, 1, 128 * 1000, d), 15, cuda_dev)
    q, k, v = (torch.empty((1, 1, N, d), dtype=torch.bfloat16, device=cuda_dev) for _ in range(3))
    for x, p in zip((q, k, v), part):
        for n in range(0, N, 128000):
            x[:, :, n:n + 128000] = p[:, :, :min(128000, N - n)]
    tail = draw((3, 512, d), 16, cuda_dev)
    for x, p in zip((q, k, v), tail):
        x[0, 0, -512:] = p
    want = torch.tensor([0, nT - 1, nT - 2, 1], dtype=torch.int32, device=cuda_dev)
    lists = want.expand(1, 1, nT, 4).contiguous()
    counts = torch.zeros((1, 1, nT), dtype=torch.int32, device=cuda_dev)
    rows = [0, 1, 77777, nT - 2, nT - 1]
    counts[0, 0, rows] = 4
    ws = sage.alloc_workspace(1, 1, N, d, mode, cuda_dev)
    o = sparse.attn_fwd_sparse(q, k, v, mode, lists, counts, workspace=ws)
    assert sage.status(ws) == sage.OK
    keys = torch.cat([torch.arange(int(b) * 128, int(b) * 128 + 128) for b in want]).to(cuda_dev)
    kk, vv = k[0, 0, keys].double(), v[0, 0, keys].double()
    for r in rows:
        qq = q[0, 0, r * 128:r * 128 + 128].double()
        s = qq @ kk.T / math.sqrt(d)
        p = torch.softmax(s, -1)
        ref = p @ vv
        kmax = kk.abs().max() + 0.1
        if mode == BF16:
            ds = (d + 8) * 2 ** -24 * (qq.abs() @ kk.abs().T)
            p_rel, p_abs, dv = 2 ** -8, 0.0, 0.0 * vv
        else:
            q_step = qq.abs().amax(1, keepdim=True) / 254
            ds = q_step * (kk.abs() + 0.1).sum(1)[None] + (qq.abs().sum(1, keepdim=True) + d * q_step) * kmax / 254
            p_rel, p_abs = 2 ** -4, 2 ** -10 / 448
            dv = 2 ** -4 * vv.abs() + v[0, 0].abs().amax(0).double() * 2 ** -10 / 448
        # scores off by ds move p, and the sum it is divided by, by exp(ds) each
        grow = torch.expm1(2 * ds.amax(1, keepdim=True) / math.sqrt(d)) + 2 ** -16
        dp = p * (grow + p_rel * (1 + grow)) + p.amax(1, keepdim=True) * (1 + grow) * p_abs
        tol = dp @ vv.abs() + (p + dp) @ dv
        tol = tol + 2 ** -8 * (ref.abs() + tol)
        err = (o[0, 0, r * 128:r * 128 + 128].double() - ref).abs()
        assert (err <= tol).all(), (r, float((err - tol).max()))
    empty = counts[0, 0] == 0
    assert not o.view(nT, -1)[empty].any()
