"""The test hooks of the bounded waits with limits about as long as a load or a step takes, so that waits run out
while their barriers are about to complete: each call reports the timeout and returns, and the next one is right."""
import pytest
import torch

pytestmark = pytest.mark.gpu

LIMITS = [1000, 1400, 1900, 2600, 3600, 5000, 8000, 20000, 100000]


def bits(t):
    return t.view(torch.int16)


def draw(shape, seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mode", [0, 1, 2])
def test_block_sparse_attention(mode, d, cuda_dev):
    from video_dit_quantized_b200 import sage, sparse
    B, H, N, nT = 1, 50, 1500, 12                 # 600 items: four or five per CTA
    q, k, v = (draw((B, H, N, d), s, cuda_dev) for s in (1, 2, 3))
    lists = torch.arange(nT, dtype=torch.int32, device=cuda_dev).expand(B, H, nT, nT).contiguous()
    counts = (torch.arange(B * H * nT, device=cuda_dev) % (nT + 1)).to(torch.int32).view(B, H, nT)
    ws = sage.alloc_workspace(B, H, N, d, mode, cuda_dev)
    ref = sparse.attn_fwd_sparse(q, k, v, mode, lists, counts, workspace=ws).clone()
    assert sage.status(ws) == sage.OK
    for limit in LIMITS:
        sparse.dbg_sparse_forced_timeout(q, k, v, mode, lists, counts, ws, limit)
        assert sage.status(ws) == sage.ETIMEOUT, limit
        got = sparse.attn_fwd_sparse(q, k, v, mode, lists, counts, workspace=ws)
        assert sage.status(ws) == sage.OK and torch.equal(bits(got), bits(ref)), limit


@pytest.mark.parametrize("d", [64, 128])
def test_dense_attention(d, cuda_dev):
    from video_dit_quantized_b200 import sage
    q, k, v = (draw((1, 20, 1500, d), s, cuda_dev) for s in (4, 5, 6))
    pre = sage.quantize_qk(q, k, v)
    status = torch.zeros(64, dtype=torch.int32, device=cuda_dev)
    ref = sage.attn_quantized(pre, 1500, status=status).clone()
    for limit in LIMITS:
        sage.dbg_attn_forced_timeout(pre, 1500, status, timeout_cycles=limit)
        assert sage.status(status) == sage.ETIMEOUT, limit
        got = sage.attn_quantized(pre, 1500, status=status)
        assert sage.status(status) == sage.OK and torch.equal(bits(got), bits(ref)), limit


def test_linear_layers(cuda_dev):
    from video_dit_quantized_b200 import sage
    x, w = draw((2000, 1024), 7, cuda_dev), draw((1024, 1024), 8, cuda_dev)
    xq, sx = sage.quantize_blocks_2d(x)
    wq, sw = sage.quantize_blocks_2d(w)
    status = torch.zeros(64, dtype=torch.int32, device=cuda_dev)
    ref8 = sage.linear_w8a8(xq, sx, wq, sw, status=status).clone()
    ref16 = sage.linear_bf16(x, w, status=status).clone()
    assert sage.status(status) == sage.OK
    for limit in LIMITS:
        sage.dbg_linear_forced_timeout(xq, sx, wq, sw, status, limit)
        assert sage.status(status) == sage.ETIMEOUT, limit
        sage.dbg_linear_bf16_forced_timeout(x, w, status, limit)
        assert sage.status(status) == sage.ETIMEOUT, limit
        assert torch.equal(bits(sage.linear_w8a8(xq, sx, wq, sw, status=status)), bits(ref8)), limit
        assert torch.equal(bits(sage.linear_bf16(x, w, status=status)), bits(ref16)), limit
        assert sage.status(status) == sage.OK
