"""sage_qk_norm_rope against the formulas in 64 bits.

Tolerance, derived: the output is rounded once to bf16, half a step = 2^-8 of the value.  Before that, in fp32
(half a step 2^-24): a sum over at most 16384 channels in a thread's 128 terms and a tree of 10 is off by at most
138 * 2^-24 of the sum of magnitudes; the root halves that, adds 2 steps; the centring adds 138 * 2^-24 of
mean |x|; weight, bias and rotation add 6 steps.  Together below 256 * 2^-24 = 2^-16 of
  S = r * |w| * (|x| + mean |x|) + |b|   (summed over the two channels of a rotated pair).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

NONE, RMS, LAYER = 0, 1, 2
HEAD, ALL = 0, 1
OFF, PAIRS, HALVES = 0, 1, 2


def want(x, w, b, cos, sin, norm, scope, eps, rope, begin, ranks):
    """(value, magnitude) in fp64, in the output layout."""
    B, N, H, d = x.shape
    y = x.double()
    dims = (-2, -1) if scope == ALL else (-1,)
    shape = (H, d) if scope == ALL else (d,)
    mag = y.abs()
    if norm == LAYER:
        y = y - y.mean(dims, keepdim=True)
        mag = mag + mag.mean(dims, keepdim=True)
    if norm != NONE:
        v = y.square().mean(dims, keepdim=True) + eps
        r = torch.where(v == 0, 0.0, v.rsqrt())
        y, mag = y * r, mag * r
    if w is not None:
        y, mag = y * w.double().view(shape), mag * w.double().abs().view(shape)
    if b is not None:
        y, mag = y + b.double().view(shape), mag + b.double().abs().view(shape)
    if rope != OFF and cos is not None and cos.shape[0]:
        n = cos.shape[0]
        ia = torch.arange(0, d, 2) if rope == PAIRS else torch.arange(d // 2)
        ib = ia + (1 if rope == PAIRS else d // 2)
        a, c = y[:, begin:begin + n][..., ia], y[:, begin:begin + n][..., ib]
        co, si = cos.double()[None, :, None], sin.double()[None, :, None]
        s = mag[:, begin:begin + n][..., ia] + mag[:, begin:begin + n][..., ib]
        y, mag = y.clone(), mag.clone()
        y[:, begin:begin + n, :, ia] = a * co - c * si
        y[:, begin:begin + n, :, ib] = a * si + c * co
        mag[:, begin:begin + n, :, ia] = s
        mag[:, begin:begin + n, :, ib] = s
    lay = (lambda t: t.permute(0, 2, 1, 3)) if ranks == 0 else (
        lambda t: t.reshape(B, N, ranks, H // ranks, d).permute(2, 0, 1, 3, 4))
    return lay(y), lay(mag)


def close(got, ref, mag):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    assert (err <= 2 ** -8 * ref.abs() + 2 ** -16 * mag + 1e-38).all(), float((err - 2 ** -8 * ref.abs()).max())


def tables(n, d, g, dev):
    a = torch.rand((n, d // 2), generator=g, device=dev, dtype=torch.float64) * 500
    return a.cos().float(), a.sin().float()


CASES = [
    # B, N, H, d, norm, scope, w dtype, rope, begin, len, fused, ranks
    (1, 1, 40, 128, RMS, ALL, "bf16", PAIRS, 0, 1, True, 0),
    (1, 1, 1, 64, RMS, HEAD, "bf16", HALVES, 0, 1, False, 0),
    (2, 130, 30, 64, LAYER, HEAD, "bf16", PAIRS, 100, 30, False, 0),
    (1, 257, 12, 128, RMS, ALL, "f32", HALVES, 0, 257, True, 4),
    (3, 77, 5, 128, LAYER, ALL, "f32", PAIRS, 7, 60, True, 0),
    (2, 33, 16, 64, RMS, HEAD, None, HALVES, 33, 0, False, 2),
    (1, 200, 3, 64, LAYER, ALL, None, OFF, 0, 0, False, 3),
    (2, 65, 7, 128, NONE, HEAD, None, PAIRS, 1, 63, True, 7),
    (1, 9, 128, 128, RMS, ALL, "bf16", HALVES, 0, 9, False, 1),          # the widest token
    (1, 9, 65, 128, LAYER, ALL, "f32", PAIRS, 2, 5, False, 0),           # just past 8192 channels
    (1, 50, 33, 64, RMS, HEAD, "f32", PAIRS, 0, 50, True, 0),            # just past 2048 channels
    (2, 40, 64, 128, LAYER, HEAD, "bf16", HALVES, 0, 40, False, 8),
    (1, 1025, 2, 128, RMS, HEAD, "bf16", PAIRS, 0, 1025, True, 0),
    (1, 8, 41, 128, LAYER, ALL, "bf16", HALVES, 0, 8, True, 0),          # just past 5120 channels
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_the_formula(case, cuda_dev):
    from video_dit_quantized_b200 import sparse
    B, N, H, d, norm, scope, wt, rope, begin, length, fused, ranks = case
    g = torch.Generator(device=cuda_dev)
    g.manual_seed(hash(case) % 1000003)
    rnd = lambda *s: torch.randn(s, generator=g, device=cuda_dev)
    qkv = (rnd(B, N, 3, H, d) * 2 + 0.5).to(torch.bfloat16)
    q, k = qkv[:, :, 0], qkv[:, :, 1]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    width = d if scope == HEAD else H * d
    ws = [None] * 4
    if wt is not None:
        dt = torch.bfloat16 if wt == "bf16" else torch.float32
        ws = [(1 + 0.3 * rnd(width)).to(dt), (1 + 0.3 * rnd(width)).to(dt), None, None]
        if norm == LAYER:
            ws[2:] = [rnd(width).to(dt), rnd(width).to(dt)]
    cos, sin = tables(length, d, g, cuda_dev) if rope != OFF else (None, None)
    kw = dict(norm=norm, scope=scope, eps=1e-6, cos=cos, sin=sin, rope=rope, rope_begin=begin, ranks=ranks)
    shape = (ranks, B, N, H // ranks, d) if ranks else (B, H, N, d)
    n = B * N * H * d
    pads = [torch.full((n + 512,), 7.0, dtype=torch.bfloat16, device=cuda_dev) for _ in range(2)]
    outs = [p[256:256 + n].view(shape) for p in pads]
    keep = qkv.clone()
    got = sparse.qk_norm_rope(q, k, *ws, **kw, q_out=outs[0], k_out=outs[1])
    for x, w, b, y, pad in zip((q, k), ws[:2], ws[2:], got, pads):
        close(y, *want(x, w, b, cos, sin, norm, scope, 1e-6, rope, begin, ranks))
        assert (pad[:256] == 7).all() and (pad[256 + n:] == 7).all()          # nothing behind or before
    assert torch.equal(qkv.view(torch.int16), keep.view(torch.int16))
    # one tensor at a time gives the same bits
    only_q = sparse.qk_norm_rope(q, None, ws[0], None, ws[2], None, **kw)
    only_k = sparse.qk_norm_rope(None, k, None, ws[1], None, ws[3], **kw)
    assert only_q[1] is None and only_k[0] is None
    assert torch.equal(only_q[0].view(torch.int16), got[0].view(torch.int16))
    assert torch.equal(only_k[1].view(torch.int16), got[1].view(torch.int16))


def test_in_place_zero_rows_and_large_means(cuda_dev):
    from video_dit_quantized_b200 import sparse
    g = torch.Generator(device=cuda_dev)
    g.manual_seed(5)
    x = (torch.randn((2, 70, 6, 128), generator=g, device=cuda_dev) + 300).to(torch.bfloat16)   # var << mean^2
    x[0, 3] = 0
    x[1, 9] = 1.5                                                                              # no variance
    cos, sin = tables(70, 128, g, cuda_dev)
    for norm in (RMS, LAYER):
        for scope in (HEAD, ALL):
            kw = dict(norm=norm, scope=scope, eps=0.0, cos=cos, sin=sin, ranks=1)
            y = x.clone()
            out, _ = sparse.qk_norm_rope(y, q_out=y.view(1, 2, 70, 6, 128), **kw)
            assert out.data_ptr() == y.data_ptr()
            ref, mag = want(x, None, None, cos, sin, norm, scope, 0.0, PAIRS, 0, 1)
            if norm == LAYER and scope == HEAD:
                ref[0, 1, 9], mag[0, 1, 9] = 0, 0
            close(out, ref, mag)
            assert (out[0, 0, 3] == 0).all()
            if norm == LAYER:
                assert (out[0, 1, 9] == 0).all()


def test_a_bad_token_stays_a_bad_token(cuda_dev):
    """NaN and infinity reach only their own token (their own head)."""
    from video_dit_quantized_b200 import sparse
    x = torch.randn((1, 20, 4, 64), device=cuda_dev).to(torch.bfloat16)
    cos, sin = tables(20, 64, torch.Generator(device=cuda_dev), cuda_dev)
    y = x.clone()
    y[0, 3, 1, 5] = float("nan")
    y[0, 8, 2, 7] = float("inf")
    for scope in (HEAD, ALL):
        a, _ = sparse.qk_norm_rope(x, norm=RMS, scope=scope, cos=cos, sin=sin)
        b, _ = sparse.qk_norm_rope(y, norm=RMS, scope=scope, cos=cos, sin=sin)
        same = (a.view(torch.int16) == b.view(torch.int16)).all(-1)              # [1, H, N]
        hit = torch.zeros_like(same)
        if scope == ALL:
            hit[:, :, 3] = hit[:, :, 8] = True
        else:
            hit[0, 1, 3] = hit[0, 2, 8] = True
        assert same[~hit].all() and b[0, 1, 3].isnan().all() and b[0, 2, 8].isnan().any()


def test_exchange_layout_is_the_send_copy(cuda_dev):
    from video_dit_quantized_b200 import sage, sparse
    B, N, H, d = 2, 50, 8, 64
    x = torch.randn((B, N, H, d), device=cuda_dev).to(torch.bfloat16)
    flat, _ = sparse.qk_norm_rope(x, ranks=1)
    for P in (2, 4, 8):
        out, _ = sparse.qk_norm_rope(x, ranks=P)
        ref = torch.empty_like(out)
        sage.ulysses_permute(flat.view(B, N, H, d), ref, B, N, H, d, P, sage.ULYSSES_SEND)
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
