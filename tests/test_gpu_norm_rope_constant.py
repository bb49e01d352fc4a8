"""Layer norm of vectors whose channels are all equal: exactly 0 before the bias, whatever the value, the width and eps.

A sum of n <= 16384 equal bf16 values (8 significant bits) is exact in fp32 in any order, and the mean is the value
itself, so the centred vector is 0 without an error.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

HEAD, ALL, LAYER = 0, 1, 2


def values(dev):
    """One token for each of the 128 bf16 significands, exponents and signs mixed."""
    m = 1 + torch.arange(128, device=dev) / 128
    e = torch.arange(128, device=dev) * 7 % 40 - 20
    return (m * torch.exp2(e) * (1 - 2 * (torch.arange(128, device=dev) % 2))).to(torch.bfloat16)


# widths over all heads that are no powers of two, in every form of the kernel
@pytest.mark.parametrize("H,d", [(7, 64), (7, 128), (15, 128), (30, 64), (41, 128), (40, 128), (65, 128), (127, 128), (8, 128)])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-5])
def test_constant_vectors_are_zero(H, d, eps, cuda_dev):
    from video_dit_quantized_b200 import sparse
    v = values(cuda_dev)
    x = v[None, :, None, None].expand(1, 128, H, d).contiguous()
    heads = v[(torch.arange(128, device=cuda_dev)[:, None] + torch.arange(H, device=cuda_dev)) % 128]
    y = heads[None, :, :, None].expand(1, 128, H, d).contiguous()          # equal within a head only
    angle = torch.arange(128 * (d // 2), device=cuda_dev, dtype=torch.float32).view(128, d // 2)
    for scope, t, width in ((ALL, x, H * d), (HEAD, x, d), (HEAD, y, d)):
        for rope in (1, 2):
            out, _ = sparse.qk_norm_rope(t, norm=LAYER, scope=scope, eps=eps, cos=angle.cos(), sin=angle.sin(), rope=rope)
            assert not out.any(), (scope, rope, int((out != 0).sum()))
        w = torch.linspace(-3, 3, width, device=cuda_dev).to(torch.bfloat16)
        b = torch.linspace(5, -5, width, device=cuda_dev).to(torch.bfloat16)
        out, _ = sparse.qk_norm_rope(t, wq=w, bq=b, norm=LAYER, scope=scope, eps=eps, ranks=1)
        assert torch.equal(out.view(128, H * d), b.view(1, -1).expand(128, width).repeat(1, H * d // width)), scope
